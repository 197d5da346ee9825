"""Pins of the serving oracle (oracle/serving.py) by closed forms: an equal
draft is always accepted, a hand-worked two-token rejection, long-run
frequencies follow the target, one visible key returns its value, and equal
scores return the mean."""
import numpy as np
import torch

from oracle import serving


def test_equal_draft_is_accepted_and_bonus_is_drawn():
    rng = np.random.default_rng(0)
    t = rng.standard_normal((1, 4, 50))
    x = np.array([[3, 7, 9]])
    n, tok, ratio = serving.spec_verify(t, t[:, :3], x, np.array([[0.9, 0.5, 0.99, 0.0]]), [3], 1.0)
    assert n[0] == 3 and list(tok[0]) == [3, 7, 9, 0] and (ratio == 1).all()


def test_hand_worked_rejection():
    # p = (1/4, 3/4), q = (3/4, 1/4): x = 0 has ratio 1/3; the remainder is all on token 1
    p, q = np.log([0.25, 0.75]), np.log([0.75, 0.25])
    for u, n_want, tok in ((0.33, 1, [0, 1]), (0.34, 0, [1, -1])):
        n, t, r = serving.spec_verify(np.stack([p, p])[None], q[None, None], np.array([[0]]), np.array([[u, 0.5]]),
                                      [1], 1.0)
        assert n[0] == n_want and list(t[0]) == tok and abs(r[0, 0] - 1 / 3) < 1e-12


def test_frequencies_follow_the_target():
    rng = np.random.default_rng(1)
    t, d = rng.standard_normal((2, 5)), rng.standard_normal((1, 5))
    p, q = serving.distribution(t[0], 0.8), serving.distribution(d[0], 0.8)
    count, N = np.zeros(5), 20000
    for _ in range(N):
        x = rng.choice(5, p=q)
        count[serving.spec_verify(t[None], d[None], np.array([[x]]), rng.random((1, 2)), [1], 0.8)[1][0, 0]] += 1
    assert np.abs(count / N - p).max() < 5 * 0.5 / np.sqrt(N)  # five standard deviations of a frequency


def test_distribution_edges():
    inf = np.inf
    assert list(serving.distribution([1.0, inf, np.nan, inf], 1.0)) == [0, 0.5, 0, 0.5]
    assert list(serving.distribution([-inf, np.nan], 1.0)) == [0, 0]
    assert list(serving.distribution([2.0, 5.0, 5.0], 0)) == [0, 1, 0]


def test_attention_closed_forms():
    k = torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16)
    v = torch.arange(2 * 8, dtype=torch.bfloat16).view(2, 8, 1, 1).expand(2, 8, 1, 128).contiguous()
    q = torch.ones(3, 2, 128, dtype=torch.bfloat16)
    # pages in reverse order: tokens 0..7 hold 8..15, tokens 8..9 hold 0..1
    o, a = serving.paged_attn(q, k, v, [0, 3], [10], [[1, 0]])
    assert torch.allclose(o[0, 0, 0], torch.tensor(sum(range(8, 16)) / 8, dtype=torch.float64))
    assert torch.allclose(o[2, 1, 5], torch.tensor((sum(range(8, 16)) + 1) / 10, dtype=torch.float64))
    o, _ = serving.paged_attn(q, k, v, [0, 3], [1], [[1, 0]])  # only the last row has a position
    assert (o[:2] == 0).all() and (o[2] == 8).all()
    assert [p for _, _, p in serving.rows_of([0, 3], [1])] == [-2, -1, 0]


def test_norm_rope_closed_forms():
    x = np.full((1, 3 * 128), 2.0)
    q, k, v, _, _ = serving.qk_norm_rope(x, 1, 1, np.full(128, 3.0), None, 0.0, [0], 1e4)
    assert np.allclose(q, 3.0) and np.allclose(k, 2.0) and np.allclose(v, 2.0)
    q, _, _, qn, _ = serving.qk_norm_rope(np.arange(3 * 128.0)[None], 1, 1, np.ones(128), None, 0.0, [12345], 1e4)
    assert np.allclose(q[..., :64] ** 2 + q[..., 64:] ** 2, qn[..., :64] ** 2 + qn[..., 64:] ** 2)
