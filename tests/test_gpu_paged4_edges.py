"""Attention over the 4-bit cache: rows that one key decides (over the bf16 cache,
too), and what is left of a call whose waits ran out.

Scores: Q and K are exact in the products (Q but for 2^-38 of its row's
largest), each of a score's 128 products and sums is off by at most 2^-23 of the
sum of magnitudes, which makes 2^-16, and the scaling by less than 2^-22. Two scores
further apart than twice that and 40 leave the smaller one e^-40 of the larger
one's weight: the output is then the larger one's value, off by the
probability's rounding (2^-11; of long chunks and over the bf16 cache 2^-8) and its own (2^-8), and by what the n others add, each
less than 2^-57 (e^-40 is 2^-57.7) of the largest magnitude that they hold (a value of
zero shows that)."""
import pytest
import torch

from oracle import serving
from test_gpu_paged4 import BF, D, FEW, LONG, cache_of, cas  # noqa: F401
from test_gpu_serving import batch, dev32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["4-bit", "bf16"])
@pytest.mark.parametrize("case", [FEW[0], FEW[5], FEW[6], FEW[7], FEW[9], FEW[11], FEW[16], LONG[0], LONG[7], LONG[10]])
@pytest.mark.parametrize("scale", [1e4, 1e8, 1e30])
def test_the_largest_score_decides(cas, case, scale, kind):  # noqa: F811
    chunks, lens, Hq, Hkv, page = case
    starts, lens, table, n_pages, rows = batch(chunks, lens, page, seed=1)
    cache = cache_of(n_pages, page, Hkv, "heads", seed=1)
    q = scale * torch.randn(rows, Hq, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    q[1::2, :, ::3] *= 1e-9
    q = q.to(BF)
    k, v = serving.q4_values(cache)  # (exact in bf16)
    if kind == "bf16":
        out = cas.paged_attn(q, k.to(BF).contiguous(), v.to(BF).contiguous(), *dev32(starts, lens, table)).view(BF)
    else:
        out = cas.paged4_attn(q, cache, *dev32(starts, lens, table)).view(BF)
    tol_p = 2.0 ** -11 if kind == "4-bit" and rows * Hq // Hkv <= 32 * len(lens) else 2.0 ** -8
    sure = 0
    for r, b, x in serving.rows_of(starts, lens):
        if x < 1:
            continue
        at = torch.arange(x + 1, device="cuda")
        pages = torch.tensor(table[b], device="cuda")[at // page]
        kk, vv = (t[pages, at % page].repeat_interleave(Hq // Hkv, 1) for t in (k, v))  # [x + 1][Hq][128]
        prod = q[r].double() * kk / D ** 0.5
        s, size = prod.sum(-1), prod.abs().sum(-1).amax(0)
        two, which = s.topk(2, dim=0)
        clear = two[0] - two[1] > 2 * (2.0 ** -16 + 2.0 ** -22) * size + 40
        want = vv[which[0], torch.arange(Hq, device="cuda")]
        err = (out[r].double() - want).abs()
        rest = 2.0 ** -57 * (x + 1) * vv.abs().amax(0)
        assert (err <= (2.0 ** -8 + tol_p + 2.0 ** -15) * want.abs() + rest)[clear].all()
        sure += int(clear.sum())
    assert sure >= 0.8 * Hq * sum(x > 0 for _, _, x in serving.rows_of(starts, lens))


@pytest.mark.parametrize("case", [FEW[0], FEW[6], FEW[9], FEW[10], FEW[15], LONG[0], LONG[7], LONG[12]])
def test_what_is_left_when_every_second_block_gave_up(cas, case):  # noqa: F811
    """A row's head is right or as it was, never half of either."""
    chunks, lens, Hq, Hkv, page = case
    starts, lens, table, n_pages, rows = batch(chunks, lens, page)
    cache = cache_of(n_pages, page, Hkv, "heads")
    q = torch.randn(rows, Hq, D, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(BF)
    out = torch.full((rows, Hq, D), 5.0, dtype=BF, device="cuda")
    ref, mass = serving.paged4_attn(q, cache, starts, lens, table)
    args = dev32(starts, lens, table)
    L = cas.lib()
    assert L.cas_test_first_wait_spins(1) == 0
    try:
        cas.paged4_attn(q, cache, *args, out=out)
        assert cas.cas_device_status() == -8
    finally:
        assert L.cas_test_first_wait_spins(0xFFFFFFFF) == 0
    fp16 = rows * Hq // Hkv <= 32 * len(lens)
    tol = (2.0 ** -12 + (2.0 ** -11 if fp16 else 2.0 ** -8)) * mass + 2.0 ** -8 * ref.abs() + 1e-6
    right = ((out.double() - ref).abs() <= tol).all(-1)
    kept = (out == 5).all(-1)
    assert (right | kept).all()
    assert kept.any()
