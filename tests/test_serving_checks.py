"""Refusals of the serving operators (no GPU): the binding checks shapes and
types before any call, and the C entry points return an argument error before
any launch."""
import ctypes
import math

import pytest
import torch

import bit_level_weight_gb300 as cas

P = ctypes.c_void_p
GOOD = 0x10000  # a 16-byte aligned address that no refused call touches
ODD = GOOD + 2


@pytest.fixture(scope="module")
def L():
    from bit_level_weight_gb300 import build
    build.build()
    return cas.lib()


# ------------------------------------------------------------------ C entry points
def call_qk(L, qkv=GOOD, kind=0, rows=2, hq=4, hkv=2, gq=None, gk=None, eps=1e-6, pos=None, pos0=0, rps=1, theta=1e4,
            q=GOOD, k=GOOD, ks=256, v=GOOD, vs=256):
    return L.cas_qk_norm_rope(qkv, kind, rows, hq, hkv, gq, gk, eps, pos, pos0, rps, theta, q, k, ks, v, vs, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(kind=2), dict(hq=0), dict(hkv=0), dict(hq=5000), dict(theta=1.0), dict(theta=math.nan),
    dict(theta=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(pos0=-1), dict(rps=0), dict(qkv=None),
    dict(qkv=ODD), dict(gq=ODD), dict(gk=ODD), dict(q=None), dict(q=ODD), dict(k=None), dict(v=ODD), dict(ks=248),
    dict(vs=250 + 8 + 1),
])
def test_qk_norm_rope_refuses(L, bad):
    assert call_qk(L, **bad) == -1


def test_qk_norm_rope_no_rows_does_nothing(L):
    assert call_qk(L, rows=0, qkv=None, q=None) == 0


def paged(**bad):
    kv = dict(n_kv_heads=2, page_size=16, n_pages=8, k=GOOD, v=GOOD, page_stride=4096, token_stride=256,
              head_stride=128)
    b = dict(batch=1, rows=2, max_pages=3, reserved0=0, row_start=GOOD, kv_len=GOOD, pages=GOOD)
    for key, x in bad.items():
        (kv if key in kv else b)[key] = x
    return cas.cas_paged_kv(*kv.values()), cas.cas_paged_batch(*b.values())


PAGED_BAD = [
    dict(n_kv_heads=0), dict(page_size=0), dict(page_size=4), dict(page_size=48), dict(page_size=2048),
    dict(n_pages=0), dict(n_pages=1 << 31), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD),
    dict(page_stride=120), dict(page_stride=4100), dict(token_stride=64), dict(head_stride=129),
    dict(head_stride=1 << 38), dict(batch=-1), dict(rows=-1), dict(max_pages=0), dict(row_start=None),
    dict(kv_len=None), dict(pages=None),
]


@pytest.mark.parametrize("bad", PAGED_BAD)
def test_paged_descriptors_refused(L, bad):
    kv, b = paged(**bad)
    assert L.cas_paged_append(ctypes.byref(kv), ctypes.byref(b), GOOD, 0, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged_attn(ctypes.byref(kv), ctypes.byref(b), GOOD, 4, GOOD, GOOD, 1 << 40, None) == -1


def test_paged_calls_refuse(L):
    kv, b = paged()
    kv, b = ctypes.byref(kv), ctypes.byref(b)
    assert L.cas_paged_append(None, b, GOOD, 0, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged_append(kv, None, GOOD, 0, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged_append(kv, b, GOOD, 0, 4, None, None, 1e-6, 1e4, None, None) == -1
    assert L.cas_paged_append(kv, b, GOOD, 3, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged_append(kv, b, GOOD, 0, 4, None, None, 1e-6, 0.5, GOOD, None) == -1
    for q, hq, o, ws, n, want in ((GOOD, 3, GOOD, GOOD, 1 << 40, -1), (GOOD, 0, GOOD, GOOD, 1 << 40, -1),
                                  (None, 4, GOOD, GOOD, 1 << 40, -1), (ODD, 4, GOOD, GOOD, 1 << 40, -1),
                                  (GOOD, 4, None, GOOD, 1 << 40, -1), (GOOD, 4, ODD, GOOD, 1 << 40, -1),
                                  (GOOD, 4, GOOD, None, 1 << 40, -6), (GOOD, 4, GOOD, ODD, 1 << 40, -6),
                                  (GOOD, 4, GOOD, GOOD, 0, -6)):
        assert L.cas_paged_attn(kv, b, q, hq, o, ws, n, None) == want
    # o over a part of q is refused (rows 2 x 4 heads x 256 bytes); q itself and what lies beside it pass on
    for far, want in ((0, -6), (16, -1), (-16, -1), (2047 & ~15, -1), (-2032, -1), (2048, -6), (-2048, -6)):
        assert L.cas_paged_attn(kv, b, GOOD, 4, GOOD + far, GOOD, 0, None) == want


@pytest.mark.parametrize("none", [dict(rows=0), dict(batch=0)])
def test_paged_nothing_to_do(L, none):
    kv, b = paged(row_start=None, kv_len=None, pages=None, **none)
    assert L.cas_paged_append(ctypes.byref(kv), ctypes.byref(b), None, 0, 4, None, None, 1e-6, 1e4, None, None) == 0
    assert L.cas_paged_attn(ctypes.byref(kv), ctypes.byref(b), None, 4, None, None, 0, None) == 0


def call_spec(L, t=GOOD, ts=100, d=GOOD, ds=100, x=GOOD, u=GOOD, nd=None, batch=2, gamma=3, vocab=100, temp=1.0, n=GOOD,
              tok=GOOD, ratio=None, ws=GOOD, wn=1 << 40):
    return L.cas_spec_verify(t, ts, d, ds, x, u, nd, batch, gamma, vocab, temp, n, tok, ratio, ws, wn, None)


@pytest.mark.parametrize("bad,want", [
    (dict(batch=-1), -1), (dict(batch=65536), -1), (dict(gamma=-1), -1), (dict(gamma=65), -1), (dict(vocab=0), -1),
    (dict(vocab=1 << 31), -1), (dict(ts=99), -1), (dict(ds=99), -1), (dict(temp=-1.0), -1), (dict(temp=math.nan), -1),
    (dict(temp=math.inf), -1), (dict(temp=1e-7), -1), (dict(t=None), -1), (dict(d=None), -1), (dict(x=None), -1),
    (dict(u=None), -1), (dict(n=None), -1), (dict(tok=None), -1), (dict(ws=None), -6), (dict(ws=ODD), -6),
    (dict(wn=0), -6),
])
def test_spec_verify_refuses(L, bad, want):
    assert call_spec(L, **bad) == want


def test_spec_verify_nothing_to_do(L):
    assert call_spec(L, batch=0, t=None, n=None, ws=None) == 0


def test_struct_layout(L):
    assert ctypes.sizeof(cas.cas_paged_kv) == 56 and cas.cas_paged_kv.page_stride.offset == 32
    assert ctypes.sizeof(cas.cas_paged_batch) == 40 and cas.cas_paged_batch.row_start.offset == 16


# ------------------------------------------------------------------ binding
def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


BF = torch.bfloat16


@pytest.mark.parametrize("args,kw,what", [
    ((torch.zeros(2, 1000), 4, 2), {}, "qkv"),
    ((torch.zeros(2, 1024, dtype=torch.float64), 4, 2), {}, "qkv"),
    ((torch.zeros(2, 1024), 4, 2), {"gamma_q": z(64, dtype=BF)}, "gamma_q"),
    ((torch.zeros(2, 1024), 4, 2), {"pos": z(3)}, "pos"),
    ((torch.zeros(2, 1024), 4, 2), {"pos": z(2, dtype=torch.int64)}, "pos"),
    ((torch.zeros(2, 1024), 4, 2), {"q": z(2, 3, 128, dtype=BF)}, "q"),
    ((torch.zeros(2, 1024), 4, 2), {"k": z(2, 4, 128, dtype=BF)}, "k"),
    ((torch.zeros(2, 1024), 4, 2), {}, "device tensors"),
])
def test_qk_norm_rope_binding(args, kw, what):
    with pytest.raises(ValueError, match=what):
        cas.qk_norm_rope(*args, **kw)


POOL = z(8, 16, 2, 128, dtype=BF)


@pytest.mark.parametrize("kw,what", [
    (dict(k_pages=z(8, 16, 2, 64, dtype=BF)), "k_pages"),
    (dict(v_pages=z(7, 16, 2, 128, dtype=BF)), "k_pages"),
    (dict(v_pages=POOL.transpose(1, 2).contiguous().transpose(1, 2)), "strides"),
    (dict(row_start=z(3)), "row_start"),
    (dict(row_start=z(2, dtype=torch.int64)), "row_start"),
    (dict(kv_len=z(1, dtype=torch.int64)), "kv_len"),
    (dict(pages=z(2, 3)), "pages"),
    (dict(pages=z(1, 3, dtype=torch.int64)), "pages"),
    (dict(), "device tensors"),
])
def test_paged_binding(kw, what):
    a = dict(k_pages=POOL, v_pages=POOL, row_start=z(2), kv_len=z(1), pages=z(1, 3)) | kw
    with pytest.raises(ValueError, match=what):
        cas.paged_append(torch.zeros(2, 1024), 4, **a)
    with pytest.raises(ValueError, match=what):
        cas.paged_attn(z(2, 4, 128, dtype=BF), workspace=z(256, dtype=torch.uint8), **a)


@pytest.mark.parametrize("n,heads", [(1, 2), (8, 1), (1, 1)])
def test_paged_strides_over_one_do_not_matter(n, heads):
    """One page or one head: torch's stride over it may be any, and differ between the pools."""
    k = z(n, 16, heads, 128, dtype=BF)
    v = k.as_strided(k.shape, [s if e > 1 else 7 * s + 1 for s, e in zip(k.stride(), k.shape)])
    assert v.stride() != k.stride()
    kv, _ = cas._paged(2, k, v, z(2), z(1), z(1, 3), -1)
    assert (kv.page_stride, kv.token_stride, kv.head_stride) == (16 * heads * 128 if n > 1 else 128, heads * 128, 128)


@pytest.mark.parametrize("kw,what", [
    (dict(x=z(2, 3, dtype=torch.int64)), "x"),
    (dict(u=None), "draft and u"),
    (dict(draft=None), "draft and u"),
    (dict(u=torch.zeros(2, 3)), "u"),
    (dict(u=torch.zeros(2, 4, dtype=torch.float64)), "u"),
    (dict(n_draft=z(3)), "n_draft"),
    (dict(n_draft=z(2, dtype=torch.int64)), "n_draft"),
    (dict(target=torch.zeros(2, 3, 10)), "target"),
    (dict(target=torch.zeros(2, 4, 10, dtype=BF)), "target"),
    (dict(), "device tensors"),
])
def test_spec_binding(kw, what):
    a = dict(target=torch.zeros(2, 4, 10), draft=torch.zeros(2, 3, 10), x=z(2, 3), u=torch.zeros(2, 4)) | kw
    with pytest.raises(ValueError, match=what):
        cas.spec_verify(**a)


@pytest.mark.parametrize("B,G", [(1, 3), (2, 0), (2, 3)])
def test_spec_binding_refuses_expanded_rows(B, G):
    """Rows that share memory have a stride below the vocabulary: read at any
    other stride they would run past the tensor's end."""
    a = dict(draft=torch.zeros(B, G, 10), x=z(B, G), u=torch.zeros(B, G + 1))
    with pytest.raises(ValueError, match="evenly spaced"):
        cas.spec_verify(torch.zeros(1, 1, 10).expand(B, G + 1, 10), **a)
    if G > 1 or B > 1 and G:
        a["draft"] = torch.zeros(1, 1, 10).expand(B, G, 10)
        with pytest.raises(ValueError, match="evenly spaced"):
            cas.spec_verify(torch.zeros(B, G + 1, 10), **a)


def test_workspace_bytes_of_refused_sizes(L):
    for rows, hq, hkv in ((-1, 4, 2), (0, 4, 2), (2, 0, 2), (2, -8, 2), (2, 4, 0), (2, 4, -1)):
        assert L.cas_paged_attn_workspace_bytes(rows, hq, hkv) == 16
    for b, g, n in ((0, 3, 10), (65536, 3, 10), (2, 65, 10), (2, -1, 10), (2, 3, 0), (2, 3, 1 << 31)):
        assert L.cas_spec_verify_workspace_bytes(b, g, n) == 16
    assert L.cas_paged_attn_workspace_bytes(1, 4, 2) > 1000 and L.cas_spec_verify_workspace_bytes(65535, 64, 10) > 1 << 20
