"""GPU parity of the serving operators against float64 definitions
(oracle/serving.py).

Tolerances. A bf16 rounding is off by at most 2^-8 relative. Norm + rotation:
one rounding of a value formed in fp32 from a rotated pair, whose fp32 error is
below 2^-19 of the pair's magnitude (sine and cosine of an angle held in 32
bits of a turn and 24 bits of mantissa: 2^-21; norm, gamma and two products:
a few 2^-24). Attention: probabilities rounded to bf16 before the product
with V (2^-8 of sum p |v|), the output's rounding, and fp32 scores, whose
error of 128 products and their exponential stays below 2^-12 relative.
Acceptance: ratios relative to the exponent's size, counts and tokens exact."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
D = 128


@pytest.fixture(scope="module")
def cas():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_level_weight_gb300 as cas
    from bit_level_weight_gb300 import build
    build.build()
    return cas


def f64(bits):
    return bits.view(BF).double().cpu().numpy()


def near_rotated(got, ref, normed):
    mag = np.sqrt(normed[..., :64] ** 2 + normed[..., 64:] ** 2)
    mag = np.concatenate([mag, mag], -1)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * mag + 1e-30).all()


# ------------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("rows,Hq,Hkv,dtype,norm", [
    (1, 32, 8, torch.float32, "qk"), (14, 32, 8, torch.float32, "qk"), (3, 5, 1, BF, "q"), (129, 8, 8, BF, "k"),
    (1, 1, 1, torch.float32, ""), (700, 7, 2, BF, "qk"), (33, 40, 4, torch.float32, "qk"), (2500, 32, 8, BF, "qk"),
])
@pytest.mark.parametrize("positions", ["given", "counted"])
def test_qk_norm_rope(cas, rows, Hq, Hkv, dtype, norm, positions):
    g = torch.Generator().manual_seed(rows + Hq)
    qkv = (3 * torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g)).to(dtype)
    gq = (1 + 0.2 * torch.randn(D, generator=g)).to(BF) if "q" in norm else None
    gk = (1 + 0.2 * torch.randn(D, generator=g)).to(BF) if "k" in norm else None
    if positions == "given":
        pos = torch.randint(-5, 200000, (rows,), generator=g, dtype=torch.int32)
        pos[-1] = 2 ** 31 - 1
        kw, p = dict(pos=pos.cuda()), pos.numpy()
    else:
        kw, p = dict(pos0=131000, rows_per_seq=7), 131000 + np.arange(rows) % 7
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    q, k, v = cas.qk_norm_rope(qkv.cuda(), Hq, Hkv, dev(gq), dev(gk), 1e-6, theta=1e6, **kw)
    num = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    rq, rk, rv, qn, kn = serving.qk_norm_rope(qkv.double().numpy(), Hq, Hkv, num(gq), num(gk), 1e-6, p, 1e6)
    near_rotated(f64(q), rq, qn)
    near_rotated(f64(k), rk, kn)
    assert (np.abs(f64(v) - rv) <= 2.0 ** -8 * np.abs(rv)).all()


@pytest.mark.parametrize("theta", [10.0, 1e4, 5e5, 1e7, 1e8])
def test_qk_norm_rope_far_positions(cas, theta):
    """Angles at positions of up to 31 bits: off by 2^-24 turns at most, which with
    the 2^-21 for sine and cosine stays below 2^-18 of a pair's magnitude."""
    p = np.array([0, 1, 2 ** 20 + 3, 2 ** 24 - 1, 2 ** 29 + 12345, 2 ** 30 + 1, 2 ** 31 - 1, -1, -77777, -2 ** 31], np.int32)
    qkv = torch.randn(len(p), 6 * D, generator=torch.Generator().manual_seed(4))
    q, k, _ = cas.qk_norm_rope(qkv.cuda(), 4, 1, pos=torch.from_numpy(p).cuda(), theta=theta)
    rq, rk, _, qn, kn = serving.qk_norm_rope(qkv.double().numpy(), 4, 1, None, None, 1e-6, p, theta)
    near_rotated(f64(q), rq, qn)
    near_rotated(f64(k), rk, kn)


def test_qk_norm_rope_into_wider_rows(cas):
    """k and v rows land in a larger buffer; what lies between stays."""
    rows, Hq, Hkv = 5, 4, 2
    qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, device="cuda")
    want = cas.qk_norm_rope(qkv, Hq, Hkv, theta=1e4)
    buf = torch.full((rows, 4, Hkv, D), 7.0, dtype=BF, device="cuda")
    cas.qk_norm_rope(qkv, Hq, Hkv, theta=1e4, k=buf[:, 0], v=buf[:, 2])
    assert torch.equal(buf[:, 0].view(torch.int16), want[1]) and torch.equal(buf[:, 2].view(torch.int16), want[2])
    assert (buf[:, 1] == 7).all() and (buf[:, 3] == 7).all()


def test_qk_norm_rope_matches_rope_split_without_norm(cas):
    qkv = torch.randn(6, 48 * D, device="cuda")
    a, b = cas.qk_norm_rope(qkv, 32, 8, pos0=900, theta=5e5), cas.rope_split(qkv, 32, 8, 900, theta=5e5)
    for x, y in zip(a, b):  # both round one fp32 value whose error is far below the rounding
        x, y = f64(x), f64(y)
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(y) + 1e-4).all()


def test_zero_head_stays_zero(cas):
    qkv = torch.zeros(2, 3 * D, device="cuda")
    q, k, v = cas.qk_norm_rope(qkv, 1, 1, torch.ones(D, dtype=BF, device="cuda"), torch.ones(D, dtype=BF, device="cuda"))
    assert (f64(q) == 0).all() and (f64(k) == 0).all()


# ------------------------------------------------------------------ paged cache
def pools(n_pages, page, H, layout, fill=None, seed=0):
    """K and V pools [n_pages][page][H][128] as views of the layout's memory."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def new(*shape):
        t = torch.randn(*shape, generator=g, device="cuda") if fill is None else torch.full(shape, fill, device="cuda")
        return t.to(BF)
    if layout == "tokens":
        return new(n_pages, page, H, D), new(n_pages, page, H, D)
    if layout == "heads":
        return new(n_pages, H, page, D).transpose(1, 2), new(n_pages, H, page, D).transpose(1, 2)
    both = new(n_pages, 2, page, H, D + 8)  # K and V of a page together, rows wider than a head
    return both[:, 0, :, :, :D], both[:, 1, :, :, :D]


def batch(chunks, lens, page, seed=0, spare=2, pad_rows=0, pad_table=1):
    """row_start, kv_len, pages as lists; pages in a random order."""
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width, at, table = max(need) + pad_table, 0, []
    for n in need:
        table.append(perm[at:at + n] + [0] * (width - n))
        at += n
    starts = [0]
    for c in chunks:
        starts.append(starts[-1] + c)
    return starts, list(lens), table, n_pages, starts[-1] + pad_rows


def dev32(*lists):
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in lists)


APPENDS = [  # chunks, lengths with the chunk, Hq, Hkv, page
    ([1], [1], 32, 8, 16),
    ([7, 7], [300, 16], 32, 8, 64),
    ([0, 3, 0, 20, 1, 0], [5, 3, 0, 150, 77, 0], 8, 2, 8),
    ([130], [130], 5, 1, 1024),
    ([2, 4], [1, 2], 4, 4, 16),  # rows before position 0: not written
    ([1] * 45, list(range(1, 46)), 6, 2, 32),
]


@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_paged_append(cas, case, layout, dtype):
    chunks, lens, Hq, Hkv, page = APPENDS[case]
    starts, lens, table, n_pages, rows = batch(chunks, lens, page, seed=case, pad_rows=3)
    g = torch.Generator().manual_seed(case)
    qkv = (2 * torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g)).to(dtype)
    gq, gk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF) for _ in range(2))
    k, v = pools(n_pages, page, Hkv, layout, fill=9.0)
    q = torch.full((rows, Hq, D), 5.0, dtype=BF, device="cuda")
    cas.paged_append(qkv.cuda(), Hq, k, v, *dev32(starts, lens, table), gq.cuda(), gk.cuda(), 1e-6, 1e6, q=q)
    p = np.zeros(rows)
    for r, b, x in serving.rows_of(starts, lens):
        p[r] = x
    rq, rk, rv, qn, kn = serving.qk_norm_rope(qkv.double().numpy(), Hq, Hkv, gq.double().numpy(), gk.double().numpy(),
                                              1e-6, p, 1e6)
    n = starts[-1]
    near_rotated(f64(q)[:n], rq[:n], qn[:n])
    assert (q[n:] == 5).all()  # padding rows stay
    k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
    written = np.zeros((n_pages, page), bool)
    for r, b, x in serving.rows_of(starts, lens):
        if x >= 0:
            at = table[b][x // page], x % page
            written[at] = True
            near_rotated(k[at], rk[r], kn[r])
            assert (np.abs(v[at] - rv[r]) <= 2.0 ** -8 * np.abs(rv[r])).all()
    assert (k[~written] == 9).all() and (v[~written] == 9).all()


def test_paged_append_skips_what_is_out_of_range(cas):
    """A position beyond the table, a page id outside the pool and rows beyond
    the tensor write nothing; the rest of the call is done."""
    Hq, Hkv, page = 4, 2, 16
    k, v = pools(4, page, Hkv, "tokens", fill=9.0)
    qkv = torch.randn(6, (Hq + 2 * Hkv) * D, device="cuda")
    # sequence 0: positions 31, 32 (beyond its two pages), 1: page ids 7 and -3, 2: claims rows past the tensor
    args = dev32([0, 2, 4, 99], [33, 17, 4], [[0, 1], [7, -3], [2, 0]])
    q = cas.paged_append(qkv, Hq, k, v, *args, theta=1e4)
    assert torch.isfinite(q.view(BF)).all()
    touched = (k != 9).any(-1).any(-1).cpu()
    want = torch.zeros(4, page, dtype=torch.bool)
    want[1, 15] = want[2, 2] = want[2, 3] = True
    assert torch.equal(touched, want)


def check_attn(cas, chunks, lens, Hq, Hkv, page, layout="tokens", seed=0, table_edit=None, pad_rows=0, spoil=None,
               scale=1.5):
    starts, lens, table, n_pages, rows = batch(chunks, lens, page, seed=seed, pad_rows=pad_rows)
    k, v = pools(n_pages, page, Hkv, layout, seed=seed)
    if table_edit:
        table_edit(table, n_pages)
    kr, vr = k.clone(), v.clone()
    if spoil is not None:  # slots that hold no visible token
        used = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for x in range(max(n, 0)):
                if x // page < len(table[b]) and 0 <= table[b][x // page] < n_pages:
                    used[table[b][x // page], x % page] = True
        k[~used] = spoil
        v[~used] = spoil
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (scale * torch.randn(rows, Hq, D, generator=g, device="cuda")).to(BF)
    out = torch.full((rows, Hq, D), 5.0, dtype=BF, device="cuda")
    cas.paged_attn(q, k, v, *dev32(starts, lens, table), out=out)
    ref, mass = serving.paged_attn(q, kr, vr, starts, lens, table)
    n = starts[-1]
    err = (out[:n].double() - ref[:n]).abs()
    tol = (2.0 ** -8 + 2.0 ** -12) * mass[:n] + 2.0 ** -8 * ref[:n].abs() + 1e-6
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} at {(err / tol).argmax().item()}"
    assert (out[n:] == 5).all()  # padding rows stay
    return q, k, v, starts, lens, table, out


ATTN = [  # chunks, lengths with the chunk, Hq, Hkv, page
    ([1], [1], 32, 8, 16),
    ([1], [0], 32, 8, 16),                       # a row that sees no key
    ([3], [2], 4, 2, 16),                        # the first row has no position
    ([1], [129], 8, 8, 64),
    ([1, 1], [128, 127], 4, 1, 128),
    ([5], [1500], 32, 8, 64),
    ([7, 7], [1000, 777], 32, 8, 16),
    ([0, 5, 0, 130, 17, 1], [9, 5, 0, 300, 257, 640], 6, 2, 32),
    ([300], [300], 5, 1, 8),
    ([129], [1024], 7, 1, 1024),
    ([64], [64], 16, 1, 256),
    ([1] * 70, list(range(1, 1400, 20)), 8, 2, 16),
    ([33], [4100], 3, 3, 128),
    ([260, 255, 1], [260, 511, 1300], 8, 4, 64),
    ([2], [6000], 64, 1, 64),                    # 128 query rows of one token pair
    ([3], [700], 200, 1, 64),                    # more heads in a group than rows in a tile
    ([1, 2, 0] * 100, [(37 * i) % 400 + 2 for i in range(300)], 4, 1, 16),  # several sequences a lane of the scheduler
    ([300, 1, 0, 290, 400], [400, 30, 20, 290, 1000], 6, 2, 32),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_paged_attn(cas, case):
    check_attn(cas, *ATTN[case], seed=case, pad_rows=case % 3)


@pytest.mark.parametrize("layout", ["heads", "both"])
@pytest.mark.parametrize("case", [5, 7, 11, 13])
def test_paged_attn_layouts(cas, case, layout):
    check_attn(cas, *ATTN[case], layout=layout, seed=case)


@pytest.mark.parametrize("spoil", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("case", [0, 3, 6, 7, 8, 12])
def test_paged_attn_unused_slots_may_hold_anything(cas, case, spoil):
    check_attn(cas, *ATTN[case], seed=case, spoil=spoil)


@pytest.mark.parametrize("spoil", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("chunks,lens,Hq,page", [([5], [300], 8, 16), ([70], [70], 8, 32), ([200, 3], [500, 64], 12, 64),
                                                 ([129, 1, 140], [257, 40, 140], 8, 128)])
def test_paged_attn_values_that_a_row_does_not_see(cas, chunks, lens, Hq, page, spoil):
    """Keys and values of later tokens of the chunk that are not finite: rows
    before them are as without, rows from them on are not finite where the
    values are not. Twice, so that nothing of the first call remains."""
    Hkv = 2
    starts, lens, table, n_pages, rows = batch(chunks, lens, page, seed=5)
    k, v = pools(n_pages, page, Hkv, "tokens", seed=5)
    q = torch.randn(rows, Hq, D, device="cuda").to(BF)
    args = dev32(starts, lens, table)
    clean = cas.paged_attn(q, k, v, *args).view(BF)
    hit = {}
    for b, (c, n) in enumerate(zip(chunks, lens)):
        for back, d in ((1, 3), (c // 2 + 1, 100), (c // 2 + 1, 127)):
            p = n - back
            if p > n - c:  # not the chunk's first token: some row does not see it
                v[table[b][p // page], p % page, 1, d] = spoil
                hit[b, d] = min(hit.get((b, d), n), p)
    bad = cas.paged_attn(q, k, v, *args).view(BF)
    sees = torch.zeros(rows, Hq, D, dtype=torch.bool, device="cuda")
    for r, b, p in serving.rows_of(starts, lens):
        for (s, d), first in hit.items():
            if s == b and p >= first:
                sees[r, Hq // Hkv:, d] = True
    assert not torch.isfinite(bad[sees]).any()
    assert torch.equal(bad[~sees], clean[~sees])
    for (b, d), first in hit.items():  # and keys: a score that is not finite is seen only by later rows
        v[table[b][first // page], first % page, 1, d] = 0.5
    v2 = v.clone()
    v2[~torch.isfinite(v2)] = 0.5
    base = cas.paged_attn(q, k, v2, *args).view(BF)
    p = lens[0] - 1
    k[table[0][p // page], p % page, 0, 0] = spoil
    got = cas.paged_attn(q, k, v2, *args).view(BF)
    last = starts[1] - 1
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[last] = False
    assert torch.equal(got[keep], base[keep])


@pytest.mark.parametrize("chunks,deep", [([64] * 100, 0), ([48, 64] * 100, 500), ([1, 64, 33, 7, 64] * 40, 200)])
def test_paged_attn_many_units_a_cta(cas, chunks, deep):
    """Many short prompts: every CTA takes several units in a row, most of 129 to
    256 rows and of a few key tiles. Then with values that only a sequence's last
    row sees not finite, in every third sequence, several times."""
    Hq, Hkv, page = 32, 8, 16
    lens = [c + ((37 * i) % deep if deep else 0) for i, c in enumerate(chunks)]
    q, k, v, starts, lens, table, out = check_attn(cas, chunks, lens, Hq, Hkv, page, seed=11)
    args = dev32(starts, lens, table)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for b in range(0, len(chunks), 3):
        n, h, d = lens[b], b % Hkv, (7 * b) % D
        v[table[b][(n - 1) // page], (n - 1) % page, h, d] = float("nan")
        hit[starts[b + 1] - 1, 4 * h:4 * h + 4, d] = True
    for _ in range(5):
        got = cas.paged_attn(q, k, v, *args).view(BF)
        assert got[hit].isnan().all()
        assert torch.equal(got[~hit], out[~hit])
    assert cas.cas_device_status() == 0


@pytest.mark.parametrize("T,n", [(1, 1), (1, 300), (3, 9000), (90, 700)])
def test_paged_attn_infinite_scores(cas, T, n):
    """Keys of which one (all: n = 1) holds an infinity or NaN: a score of +inf or
    NaN spoils the row, one of -inf weighs nothing, nothing but -inf gives zeros."""
    page, Hq, Hkv = 32, 8, 2
    starts, lens, table, n_pages, rows = batch([T], [n], page, seed=8)
    k, v = pools(n_pages, page, Hkv, "tokens", seed=8)
    q = torch.randn(rows, Hq, D, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").to(BF)
    q[:, ::2, 5], q[:, 1::2, 5] = 1.0, -1.0
    at = (n - T) // 2  # every row sees it
    where = table[0][at // page], at % page, slice(None), 5
    for x in (float("inf"), float("-inf"), float("nan")):
        k[where] = x
        out = cas.paged_attn(q, k, v, *dev32(starts, lens, table)).view(BF)
        low = torch.zeros(Hq, dtype=torch.bool, device="cuda")  # heads whose score there is -inf
        if x == x:
            low[(slice(1, None, 2) if x > 0 else slice(0, None, 2))] = True
        assert not torch.isfinite(out[:, ~low]).any()
        if n == 1:
            assert (out[:, low] == 0).all()
        elif x == x:
            ref, mass = serving.paged_attn(q, k, v, starts, lens, table)
            err = (out[:, low].double() - ref[:, low]).abs()
            assert (err <= (2.0 ** -8 + 2.0 ** -12) * mass[:, low] + 2.0 ** -8 * ref[:, low].abs() + 1e-6).all()


def test_paged_attn_rows_far_before_the_first_token(cas):
    """A length below the chunk's: the rows before position 0 see no key and are
    zero, also those more than 2^16 before values that are not finite."""
    rows, n = 70000, 3
    k, v = pools(1, 16, 1, "tokens", seed=6)
    q = torch.randn(rows, 1, D, device="cuda").to(BF)
    v[0, 0, 0, 5] = float("nan")
    out = cas.paged_attn(q, k, v, *dev32([0, rows], [n], [[0]])).view(BF)
    assert (out[:rows - n] == 0).all()
    assert out[rows - n:, 0, 5].isnan().all()
    rest = out[rows - n:, 0].clone()
    rest[:, 5] = 0
    assert torch.isfinite(rest).all()


def test_paged_attn_bad_pages_read_as_zeros(cas):
    def edit(table, n_pages):
        table[0][1], table[0][2], table[1][0] = n_pages, -1, 2 ** 31 - 1
    check_attn(cas, [3, 140], [200, 400], 8, 2, 32, table_edit=edit)


def test_paged_attn_length_beyond_the_table(cas):
    """Positions past the block table are not seen."""
    def edit(table, n_pages):
        for row in table:
            del row[2:]
    check_attn(cas, [3, 70], [200, 90], 8, 2, 32, table_edit=edit)


def test_paged_attn_long_context_large_scores(cas):
    """Scores of size 60 and a maximum that moves through 20000 keys."""
    check_attn(cas, [2, 40], [20000, 9001], 8, 2, 64, scale=8.0)


@pytest.mark.parametrize("chunks,lens,Hq,Hkv", [
    ([1], [1], 8, 8), ([1, 1, 1], [700, 129, 5000], 32, 8), ([16], [2000], 32, 8), ([4, 7, 0, 32, 1], [900, 7, 0, 300, 64], 8, 2),
    ([2], [6000], 64, 1),
])
def test_paged_attn_few_rows_keep_their_probabilities(cas, chunks, lens, Hq, Hkv):
    """At most 128 rows of a kv head a sequence: probabilities in two bf16 terms,
    as in the compressed cache's attention. Tolerance: the output's one rounding,
    and 2^-12 of sum p |v| for the scores' fp32 error and all that is smaller (the
    two terms 2^-17, the exponentials 2^-21)."""
    starts, lens, table, n_pages, rows = batch(chunks, lens, 32, seed=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = pools(n_pages, 32, Hkv, "tokens", seed=1)
    q = torch.randn(rows, Hq, D, generator=g, device="cuda").to(BF)
    out = cas.paged_attn(q, k, v, *dev32(starts, lens, table)).view(BF)
    ref, mass = serving.paged_attn(q, k, v, starts, lens, table)
    err = (out.double() - ref).abs()
    assert (err <= 2.0 ** -12 * mass + 2.0 ** -8 * ref.abs() + 1e-6).all()


def test_paged_attn_long_units(cas):
    """Units of 32768 key tiles, two a CTA (every page of the table is the same
    one): no wait gives up, however long a unit takes.

    The page's tokens at positions up to p count (p - s) // 1024 + 1 times each.
    Tolerance: rounding of P and of the output as elsewhere, and fp32 sums of n
    terms in turn, at most n 2^-23 of their absolute sum where each addition may
    be cut instead of rounded: 8 products of 16 keys a tile for the output
    (2^18 additions), one a tile for the sum (2^15)."""
    page, n, T, G = 1024, 1 << 22, 19456, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(1, page, 1, D, generator=g, device="cuda").to(BF)
    v = (1 + torch.randn(1, page, 1, D, generator=g, device="cuda")).to(BF)
    q = torch.randn(T, G, D, generator=g, device="cuda").to(BF)
    out = torch.full((T, G, D), 5.0, dtype=BF, device="cuda")
    cas.paged_attn(q, k, v, *dev32([0, T], [n], [[0] * (n // page)]), out=out)
    assert cas.cas_device_status() == 0
    pick = torch.tensor([0, 1, 63, 64, 5000, 9727, 9728, 15000, T - 2, T - 1], device="cuda")
    pos = n - T + pick
    count = (pos[:, None] - torch.arange(page, device="cuda")) // page + 1
    s = q[pick].double() @ k[0, :, 0].double().T / D ** 0.5
    w = torch.softmax(s + count[:, None, :].double().log(), -1)
    ref, mass = w @ v[0, :, 0].double(), w @ v[0, :, 0].double().abs()
    err = (out[pick].double() - ref).abs()
    tol = (2.0 ** -8 + 2.0 ** -12 + 2.0 ** 18 * 2.0 ** -23) * mass + (2.0 ** -8 + 2.0 ** 15 * 2.0 ** -23) * ref.abs()
    print("worst", (err / mass).max().item())
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g}"


@pytest.mark.parametrize("B,T,G,n", [(1, 9728, 4, 1 << 17), (1, 9728, 4, 1 << 20), (1, 9728, 4, 1 << 22),
                                     (200, 1, 1, 1 << 20), (170, 7, 4, 1 << 19), (40, 200, 1, 1 << 20),
                                     (1, 9728, 4, 40960), (1, 9728, 4, 71680), (300, 1, 1, 66560), (200, 7, 4, 133120)])
def test_paged_attn_sums_do_not_shrink_with_the_context(cas, B, T, G, n):
    """Units of up to 32768 key tiles, one page throughout: the tensor cores' sums
    must not lose what grows with the number of tiles.

    A slot's O takes at most 256 tiles of 8 products (few rows: 16, of two terms of
    P) in a row, 2^12 additions, each of which cuts at most 2^-23 of the sum; the
    rest is rounded to nearest. So the outputs' mean is off by 2^-11 of sum p |v|
    at most, and by the mean of 3840 or more roundings (of 2^-9 each in the root
    mean square: 2^-15 together, taken four times). Each output as elsewhere."""
    page = 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(1, page, 1, D, generator=g, device="cuda").to(BF)
    v = (1 + torch.randn(1, page, 1, D, generator=g, device="cuda")).to(BF)
    q = torch.randn(B * T, G, D, generator=g, device="cuda").to(BF)
    out = cas.paged_attn(q, k, v, *dev32([T * b for b in range(B + 1)], [n] * B), torch.zeros(B, n // page, dtype=torch.int32,
                                                                                        device="cuda")).view(BF)
    assert cas.cas_device_status() == 0
    pick = torch.unique(torch.tensor([0, 1, T // 2, T - 2, T - 1, (B // 2) * T, B * T - 1, (B - 3) * T + T // 3,
                                      *range(0, B * T, max(1, B * T // 30))], device="cuda").clamp(0, B * T - 1))
    count = (n - T + pick % T)[:, None] - torch.arange(page, device="cuda")
    s = q[pick].double() @ k[0, :, 0].double().T / D ** 0.5
    w = torch.softmax(s + (count // page + 1)[:, None, :].double().log(), -1)
    ref, mass = w @ v[0, :, 0].double(), w @ v[0, :, 0].double().abs()
    err = out[pick].double() - ref
    print("mean", (err.sum() / mass.sum()).item())
    assert (err.abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * mass + 2.0 ** -8 * ref.abs()).all()
    assert err.sum().abs() <= (2.0 ** -11 + 2.0 ** -13) * mass.sum()


@pytest.mark.parametrize("B,T,G", [(1, 9728, 4), (200, 7, 4)])
def test_paged_attn_long_units_and_values_that_a_row_does_not_see(cas, B, T, G):
    """Units of 560 tiles whose last token's value is not finite."""
    page, n = 1024, 71680
    k, v = pools(2, page, 1, "tokens", seed=5)
    q = torch.randn(B * T, G, D, device="cuda").to(BF)
    args = dev32([T * b for b in range(B + 1)], [n] * B, [[0] * (n // page - 1) + [1]] * B)
    clean = cas.paged_attn(q, k, v, *args).view(BF)
    v[1, page - 1, 0, 77] = float("nan")
    got = cas.paged_attn(q, k, v, *args).view(BF)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[T - 1::T, :, 77] = True
    assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])


def test_paged_attn_offsets_beyond_32_bits(cas):
    """Pages whose element offsets pass 2^32 in a pool that is mostly unused."""
    H, page = 8, 64
    n_pages = 2 ** 32 // (page * H * D) + 40
    pool = torch.empty(n_pages, page, 2, H, D, dtype=BF, device="cuda")
    k, v = pool[:, :, 0], pool[:, :, 1]
    table = [[n_pages - 1 - 3 * i for i in range(12)], [2 * i for i in range(12)]]
    for row in table:
        for i in row:
            pool[i] = torch.randn(page, 2, H, D, device="cuda").to(BF)
    q = torch.randn(4, 16, D, device="cuda").to(BF)
    out = cas.paged_attn(q, k, v, *dev32([0, 1, 4], [700, 768], table)).view(BF)
    ref, mass = serving.paged_attn(q, k, v, [0, 1, 4], [700, 768], table)
    assert ((out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * ref.abs() + 1e-6).all()
    qkv = torch.randn(4, 32 * D, device="cuda")
    cas.paged_append(qkv, 16, k, v, *dev32([0, 1, 4], [700, 768], table), theta=1e4)
    last = pool[table[0][699 // page], 699 % page, 1]
    assert torch.equal(last, qkv[0].view(32, D)[24:].to(BF))


def test_paged_attn_repeats_bit_for_bit(cas):
    a = check_attn(cas, [1, 9, 300], [5000, 3000, 2000], 32, 8, 64)
    out = [cas.paged_attn(a[0], a[1], a[2], *dev32(*a[3:6])) for _ in range(3)]
    assert all(torch.equal(t.view(BF), a[6]) for t in out)


def test_paged_graph_follows_the_batch_on_the_device(cas):
    """Append and attention captured together; the replay reads the lengths
    that the device holds then."""
    Hq, Hkv, page = 8, 2, 16
    k, v = pools(40, page, Hkv, "tokens")
    starts, lens, table = dev32([0, 1, 2], [100, 37], [list(range(10)), list(range(10, 20))])
    qkv = torch.randn(2, 12 * D, device="cuda")
    q, o = (torch.empty(2, Hq, D, dtype=torch.int16, device="cuda") for _ in range(2))
    ws = torch.empty(cas.cas_paged_attn_workspace_bytes(2, Hq, Hkv), dtype=torch.uint8, device="cuda")

    def step():
        cas.paged_append(qkv, Hq, k, v, starts, lens, table, theta=1e4, q=q)
        cas.paged_attn(q, k, v, starts, lens, table, out=o, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([101, 38], [160, 1], [5, 90]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        qkv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        ref, mass = serving.paged_attn(q.view(BF), k, v, [0, 1, 2], new, table.tolist())
        tol = (2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * ref.abs() + 1e-6
        assert ((o.view(BF).double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("chunks,lens,Hq,Hkv", [([1], [9000], 32, 8), ([300, 1, 70, 600], [3000, 77, 70, 5000], 12, 4),
                                                ([40, 64, 90] * 30, [700, 64, 90] * 30, 12, 2)])
def test_paged_attn_in_place(cas, chunks, lens, Hq, Hkv):
    """The output in q's own memory."""
    starts, lens, table, n_pages, rows = batch(chunks, lens, 32, seed=4, pad_rows=2)
    k, v = pools(n_pages, 32, Hkv, "tokens", seed=4)
    args = dev32(starts, lens, table)
    q = torch.randn(rows, Hq, D, device="cuda").to(BF)
    want = cas.paged_attn(q, k, v, *args).view(BF)
    for _ in range(5):
        o = q.clone()
        assert cas.paged_attn(o, k, v, *args, out=o) is o
        assert torch.equal(o[:-2], want[:-2]) and torch.equal(o[-2:], q[-2:])


def test_paged_attn_shared_and_repeated_pages(cas):
    """Two sequences share their first pages, and one holds a page twice."""
    k, v = pools(20, 32, 2, "tokens", seed=3)
    starts, lens, table = [0, 2, 40, 41], [70, 100, 128], [[4, 7, 9, 0], [4, 7, 11, 2], [5, 5, 6, 5]]
    q = torch.randn(41, 8, D, device="cuda").to(BF)
    out = cas.paged_attn(q, k, v, *dev32(starts, lens, table)).view(BF)
    ref, mass = serving.paged_attn(q, k, v, starts, lens, table)
    assert ((out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * ref.abs() + 1e-6).all()


def test_two_streams_at_once(cas):
    """Calls on two streams, each with its own buffers and workspace (made by
    the call), give what they give one after the other."""
    k, v = pools(300, 64, 8, "tokens", seed=9)
    jobs = []
    for i, (chunks, lens) in enumerate((([1, 1, 1], [6000, 3000, 5000]), ([500], [4000]))):
        starts, lens, table, _, rows = batch(chunks, lens, 64, seed=i)
        q = torch.randn(rows, 32, D, device="cuda").to(BF)
        jobs.append((q, k, v) + dev32(starts, lens, table))
    t, d, x, u = (a.cuda() for a in spec_case(3, 4, 50000, 2, 1.0))
    want = [cas.paged_attn(*j) for j in jobs] + [cas.spec_verify(t, d, x, u)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cas.paged_attn(*jobs[i]) if i < 2 else cas.spec_verify(t, d, x, u))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in got[i])
    assert all(torch.equal(a, b) for o in got[2] for a, b in zip(o, want[2]))
    # and a stream given by name
    out = cas.paged_attn(*jobs[0], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0])


def test_named_stream_orders_copies_and_buffers(cas, monkeypatch):
    """With a stream given, what the call copies and allocates belongs to it:
    the current stream is busy meanwhile, and its memory is not taken."""
    k, v = pools(20, 32, 2, "tokens", seed=7)
    args = dev32([0, 2, 40], [70, 500], [list(range(3)) + [0] * 13, list(range(3, 19))])
    wide = torch.randn(40, 16, D, device="cuda").to(BF)[:, ::2]  # gathered by the call
    qkv = torch.randn(40, 12 * D, device="cuda")
    t, d, x, u = (a.cuda() for a in spec_case(2, 3, 3000, 6, 0.8))
    side = torch.cuda.Stream()

    def run(**kw):
        a = cas.qk_norm_rope(qkv, 8, 2, **kw)
        return (cas.paged_attn(wide, k, v, *args, **kw), *a, cas.paged_append(qkv, 8, k.clone(), v.clone(), *args, **kw),
                *cas.spec_verify(t, d, x, u, **kw))
    want = run()
    torch.cuda.synchronize()
    seen, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (seen.append(torch.cuda.current_stream()), empty(*a, **kw))[1])
    kc, vc = k.clone(), v.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    got = (cas.paged_attn(wide, k, v, *args, stream=side), *cas.qk_norm_rope(qkv, 8, 2, stream=side),
           cas.paged_append(qkv, 8, kc, vc, *args, stream=side), *cas.spec_verify(t, d, x, u, stream=side))
    side.synchronize()
    monkeypatch.undo()
    assert len(seen) >= 10 and all(s == side for s in seen)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_launch_overlap_keeps_the_results(cas):
    """A chain of the operators with launches that may overlap, captured."""
    Hq, Hkv, page = 16, 4, 32
    k, v = pools(64, page, Hkv, "tokens", seed=4)
    args = dev32([0, 3, 300], [300, 700], [list(range(30)), list(range(30, 60))])
    qkv = torch.randn(300, 24 * D, device="cuda")
    t, d, x, u = (a.cuda() for a in spec_case(2, 3, 30000, 6, 0.8))

    def chain():
        q = cas.paged_append(qkv, Hq, k, v, *args, theta=1e6)
        o = cas.paged_attn(q, k, v, *args)
        a = cas.qk_norm_rope(qkv, Hq, Hkv, pos0=5)
        return (q, o, *a, *cas.spec_verify(t, d, x, u), *cas.spec_verify(t, None, x, None, temperature=0.0))
    want = chain()
    torch.cuda.synchronize()
    cas.set_launch_overlap(True)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            chain()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
    finally:
        cas.set_launch_overlap(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cas.cas_device_status() == 0


def test_paged_attn_wait_that_runs_out_is_reported(cas):
    """Waits for work that nobody hands out give up: a status, no output, and
    the next call with the normal limit is right."""
    k, v = pools(40, 32, 2, "tokens", seed=3)
    starts, lens, table = [0, 2, 140], [70, 600], [list(range(19)), list(range(20, 39))]
    args = dev32(starts, lens, table)
    q = torch.randn(140, 8, D, device="cuda").to(BF)
    want = cas.paged_attn(q, k, v, *args)
    assert cas.cas_device_status() == 0
    out = torch.full((140, 8, D), 5.0, dtype=BF, device="cuda")
    try:
        assert cas.lib().cas_test_first_wait_spins(0) == 0
        cas.paged_attn(q, k, v, *args, out=out)
        assert cas.cas_device_status() == -8
        assert cas.cas_device_status() == 0  # read once, then clear
    finally:
        assert cas.lib().cas_test_first_wait_spins(0xFFFFFFFF) == 0
    assert (out == 5).all()
    assert torch.equal(cas.paged_attn(q, k, v, *args), want)
    assert cas.cas_device_status() == 0


def test_paged_attn_pieces_of_a_cta_that_gave_up_are_not_joined(cas):
    """Every second CTA gives up: rows are right or as they were, whatever an
    earlier call has left in the workspace."""
    chunks, lens = [1, 40] + [1] * 200 + [3, 90], [9000, 3000] + [50 + i for i in range(200)] + [12000, 2500]
    starts, lens, table, n_pages, rows = batch(chunks, lens, 32, seed=2)
    k, v = pools(n_pages, 32, 2, "tokens", seed=2)
    args = dev32(starts, lens, table)
    q = torch.randn(rows, 8, D, device="cuda").to(BF)
    ws = torch.empty(cas.cas_paged_attn_workspace_bytes(rows, 8, 2), dtype=torch.uint8, device="cuda")
    want = cas.paged_attn(q, k, v, *args).view(BF)
    cas.paged_attn(-q, k, v, *args, workspace=ws)
    out = torch.full((rows, 8, D), 5.0, dtype=BF, device="cuda")
    try:
        assert cas.lib().cas_test_first_wait_spins(1) == 0
        cas.paged_attn(q, k, v, *args, out=out, workspace=ws)
        assert cas.cas_device_status() == -8
    finally:
        assert cas.lib().cas_test_first_wait_spins(0xFFFFFFFF) == 0
    right, old = (out == want).all(-1), (out == 5).all(-1)
    assert (right | old).all() and right.any() and old.any()
    assert old[0].all() and old[-90:].all()  # cut into pieces of several CTAs
    cas.paged_attn(q, k, v, *args, out=out, workspace=ws)
    assert torch.equal(out, want)
    assert cas.cas_device_status() == 0


def test_misplaced_tensors_are_refused(cas):
    k, v = pools(4, 16, 2, "tokens")
    args = dev32([0, 2], [5], [[0, 1]])
    q = torch.zeros(2, 4, D, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="one device"):
        cas.paged_attn(q, k.cpu(), v.cpu(), *args)
    with pytest.raises(ValueError, match="contiguous"):
        cas.paged_append(torch.zeros(2, 2048, device="cuda")[:, ::2], 4, k, v, *args)
    with pytest.raises(cas.CasError):
        cas.paged_attn(q, k, v, *args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(2, 8, D, dtype=BF, device="cuda")[:, ::2]  # gathered by the call
    assert torch.equal(cas.paged_attn(wide, k, v, *args), cas.paged_attn(q, k, v, *args))


# ------------------------------------------------------------------ acceptance
def spec_case(B, G, V, seed, temp, masked=False, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    t = spread * torch.randn(B, G + 1, V, generator=g)
    d = t[:, :G] + 0.7 * torch.randn(B, G, V, generator=g)
    if masked:
        off = torch.rand(B, 1, V, generator=g) < 0.3
        off[..., V // 2] = False
        t, d = t.masked_fill(off, -torch.inf), d.masked_fill(off[:, :1], -torch.inf)
    race = torch.rand(B, G, V, generator=g).clamp(1e-6, 1 - 1e-6)
    x = (d / max(temp, 1e-3) - torch.log(-torch.log(race))).argmax(-1).int()
    return t, d, x, torch.rand(B, G + 1, generator=g)


def check_spec(cas, t, d, x, u, nd, temp):
    dev = lambda a: None if a is None else a.cuda()  # noqa: E731
    ndt = None if nd is None else torch.tensor(nd, dtype=torch.int32).cuda()
    n, tok, ratio = cas.spec_verify(dev(t), dev(d), dev(x), dev(u), ndt, temp)
    num = lambda a: None if a is None else a.double().numpy()  # noqa: E731
    rn, rt, rr = serving.spec_verify(num(t), num(d), x.numpy(), num(u), nd or [x.shape[1]] * x.shape[0], temp)
    assert list(n.cpu()) == list(rn)
    assert np.array_equal(tok.cpu().numpy(), rt)
    # exponents up to 80 in fp32: each probability is off by less than 2^-22 * (80 + 32) relative
    assert (np.abs(ratio.double().cpu().numpy() - rr) <= 2.0 ** -21 * 112 * rr + 1e-30).all()
    return rn


@pytest.mark.parametrize("B,G,V,temp,masked", [
    (1, 4, 128256, 1.0, False), (2, 6, 151936, 0.7, True), (5, 1, 1, 1.0, False), (3, 2, 2, 1.0, False),
    (7, 3, 33, 0.5, True), (2, 15, 50257, 1.3, False), (40, 2, 1023, 1.0, False), (1, 64, 4096, 0.9, False),
    (3, 0, 1000, 1.0, False), (2, 3, 16385, 0.05, False), (4, 4, 5000, 0.0, True), (1, 4, 128256, 0.0, False),
])
def test_spec_verify(cas, B, G, V, temp, masked):
    t, d, x, u = spec_case(B, G, V, B + G + V, temp, masked)
    check_spec(cas, t, d, x, u, None, temp)


def test_spec_verify_uneven_drafts(cas):
    t, d, x, u = spec_case(6, 5, 3001, 3, 1.0)
    rn = check_spec(cas, t, d, x, u, [0, 5, 3, 9, -2, 1], 1.0)
    assert rn[0] == 0 and rn[4] == 0


def test_spec_verify_many_draws(cas):
    """Hundreds of borders in one call: flat, peaked and equal distributions."""
    for seed, spread in ((0, 0.01), (1, 1.0), (2, 6.0)):
        t, d, x, u = spec_case(300, 2, 4001, seed, 1.0, spread=spread)
        d[::5] = t[::5, :2]  # the draft is the target: all accepted
        rn = check_spec(cas, t, d, x, u, None, 1.0)
        assert (rn[::5] == 2).all()


def test_spec_verify_edges(cas):
    inf, nan = float("inf"), float("nan")
    V = 700
    t, d, x, u = spec_case(10, 2, V, 11, 1.0)
    t[0, 0] = -inf                                   # the target has no mass: nothing accepted, no token
    d[1, 0] = nan                                    # the draft has no mass: ratio 1
    x[2, 0], x[3, 0] = -1, V                         # no such token
    t[4, 0, 5] = t[4, 0, 600] = inf                  # infinite maxima share the mass
    x[5, 0] = 9
    d[5, 0, 9] = -inf                                # the draft says it cannot be: accepted where the target has mass
    u[6, 0] = nan                                    # accepts nothing
    u[7, 2], u[8, 2], u[9, 2] = 1.5, -1.0, nan       # beyond [0, 1)
    u[7:, :2] = 0.0
    t[8, 2, :4] = -inf                               # the first token with mass is the fifth
    check_spec(cas, t, d, x, u, None, 1.0)


def test_spec_verify_greedy_needs_no_draft(cas):
    t, d, x, _ = spec_case(4, 3, 2000, 5, 0.0)
    t[1, 2, 7] = t[1, 2, 1500] = 90.0                # a tie: the lower index
    x[1] = t[1, :3].argmax(-1).int()
    x[1, 2] = 7
    rn = check_spec(cas, t, None, x, None, None, 0.0)
    assert rn[1] == 3


def test_spec_verify_strided_rows(cas):
    """Rows inside a padded vocabulary, at any alignment."""
    B, G, V, W = 3, 2, 1001, 1027
    t, d, x, u = spec_case(B, G, V, 8, 1.0)
    want = cas.spec_verify(t.cuda(), d.cuda(), x.cuda(), u.cuda())
    bt = torch.full((B * (G + 1), W), 99.0, device="cuda")
    bd = torch.full((B * G, W), 99.0, device="cuda")
    vt, vd = bt.view(B, G + 1, W)[..., 3:3 + V], bd.view(B, G, W)[..., 1:1 + V]
    vt.copy_(t)
    vd.copy_(d)
    got = cas.spec_verify(vt, vd, x.cuda(), u.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want[:2]))
    assert torch.allclose(got[2], want[2], rtol=1e-5)


# ------------------------------------------------------------------ the operators together
def test_prompt_then_draft_step(cas):
    """A prompt read in ragged chunks through the paged cache, its keys and
    values encoded into the compressed cache, and the two caches' attentions
    over the same tokens compared at the verify rows, which a step's
    acceptance ends."""
    Hq, Hkv, page, T0, T = 32, 8, 16, 300, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = pools(40, page, Hkv, "tokens", fill=0.0)
    table = dev32([list(range(3, 3 + 25))])[0]
    gq, gk = ((1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF) for _ in range(2))
    qkv = torch.randn(T0 + T, 48 * D, generator=g, device="cuda")
    q_all, k_all, v_all = cas.qk_norm_rope(qkv, Hq, Hkv, gq, gk, theta=1e6)
    kv = cas.KVCache(Hkv, 512, cas.params(1, 64, 3), k_all[:64].contiguous(), v_all[:64].contiguous())
    at = 0
    for n in (1, 130, 169, T):  # prompt chunks, then the verify rows
        args = dev32([0, n], [at + n]) + (table,)
        q = cas.paged_append(qkv[at:at + n].contiguous(), Hq, k, v, *args, gq, gk, theta=1e6)
        assert torch.equal(q, q_all[at:at + n])
        o = cas.paged_attn(q, k, v, *args)
        kv.append(k_all[at:at + n], v_all[at:at + n])
        at += n
    assert kv.status() == (T0 + T, 0)
    flat = [x.view(40 * page, Hkv, D)[3 * page:3 * page + at].view(torch.int16) for x in (k, v)]
    assert torch.equal(flat[0], k_all) and torch.equal(flat[1], v_all)
    exact = cas.verify_attn([kv], q.view(1, T, Hq, D))[0].double()  # fp32 over the same, losslessly kept bits
    _, mass = serving.paged_attn(q.view(BF), k, v, [0, T], [at], table.tolist())
    tol = (2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * exact.abs() + 2e-3 * mass + 1e-6
    assert ((o.view(BF).double() - exact).abs() <= tol).all()
    # the step ends: 4 drafted tokens judged by the verify rows' logits
    t, d, x, u = spec_case(1, T - 1, 2000, 4, 1.0)
    check_spec(cas, t, d, x, u, None, 1.0)
