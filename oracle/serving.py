"""Float64 statements of the serving operators around the split: q/k head
norms with rotary embedding, the paged cache, attention of a ragged batch over
it and the acceptance of drafted tokens.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain definitions, row
by row, with no blocking or fusion.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import glue


def qk_norm_rope(qkv, n_q: int, n_kv: int, gamma_q, gamma_k, eps: float, pos, theta: float):
    """float64 (q, k, v) of a fused QKV product [rows][(n_q + 2 n_kv) * 128];
    gammas: float64 [128] or None."""
    h = np.asarray(qkv, dtype=np.float64).reshape(-1, n_q + 2 * n_kv, 128)
    out = []
    for x, g in ((h[:, :n_q], gamma_q), (h[:, n_q:n_q + n_kv], gamma_k)):
        if g is not None:
            x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(g, dtype=np.float64)
        out.append((glue.rope(x, pos, theta), x))
    (q, qn), (k, kn) = out
    return q, k, h[:, n_q + n_kv:], qn, kn


def rows_of(row_start, kv_len):
    """(row, sequence, position) of every row that belongs to a sequence."""
    for b in range(len(kv_len)):
        for r in range(row_start[b], row_start[b + 1]):
            yield r, b, kv_len[b] - (row_start[b + 1] - r)


def gather(pool: torch.Tensor, pages, n: int) -> torch.Tensor:
    """Tokens 0..n-1 of a sequence, float64 [n][H][128]; a page id outside the
    pool reads as zeros. pool: bfloat16 [n_pages][S][H][128]."""
    S = pool.shape[1]
    out = torch.zeros(n, pool.shape[2], 128, dtype=torch.float64, device=pool.device)
    for i in range(-(-n // S)):
        if 0 <= pages[i] < pool.shape[0]:
            m = min(S, n - i * S)
            out[i * S:i * S + m] = pool[pages[i], :m].double()
    return out


def paged_attn(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, row_start, kv_len, pages):
    """float64 (o, sum p |v|) of every row that belongs to a sequence, zeros
    elsewhere; q: bfloat16 [rows][Hq][128]; the other arguments as lists."""
    rows, Hq, _ = q.shape
    S, H = k_pool.shape[1], k_pool.shape[2]
    o = torch.zeros(rows, Hq, 128, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    for b in range(len(kv_len)):
        r0, r1 = row_start[b], row_start[b + 1]
        n = min(max(kv_len[b], 0), len(pages[b]) * S)
        if r1 <= r0 or n == 0:
            continue
        k, v = gather(k_pool, pages[b], n), gather(v_pool, pages[b], n)
        p = torch.arange(max(kv_len[b], 0) - (r1 - r0), max(kv_len[b], 0), device=q.device)
        hidden = torch.arange(n, device=q.device)[None, :] > p[:, None]
        for h in range(Hq):
            w = (q[r0:r1, h].double() @ k[:, h // (Hq // H)].T) / math.sqrt(128)
            w = w.masked_fill(hidden, -math.inf)
            w = torch.where(hidden.all(1, keepdim=True), torch.zeros_like(w), torch.softmax(w, -1))
            vh = v[:, h // (Hq // H)]
            o[r0:r1, h] = w @ vh
            a[r0:r1, h] = w @ vh.abs()
    return o, a


def distribution(logits, temperature: float) -> np.ndarray:
    """softmax(logits / temperature) in float64 with NaN as -inf, infinite
    maxima sharing the mass, zeros for a row of -inf; temperature 0: one at
    the lowest index of the maximum."""
    z = np.asarray(logits, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z)
    if temperature == 0:
        w = np.zeros_like(z)
        w[np.argmax(z)] = 1.0
        return w
    with np.errstate(invalid="ignore"):
        w = np.where(z == m, 1.0, np.exp((z - m) / temperature))
    return w / w.sum()


def spec_verify(target, draft, x, u, n_draft, temperature: float):
    """(n_accepted [B], tokens [B][G + 1], ratio [B][G]) of B sequences; draft
    and u may be None at temperature 0."""
    B, G = x.shape
    V = target.shape[-1]
    n, tokens, ratio = np.zeros(B, np.int32), np.full((B, G + 1), -1, np.int32), np.zeros((B, G))
    for b in range(B):
        nd = min(max(int(n_draft[b]), 0), G)
        left = None
        for j in range(nd):
            p, t = distribution(target[b, j], temperature), int(x[b, j])
            if temperature == 0:
                ratio[b, j] = p[t] if 0 <= t < V else 0.0
                ok = ratio[b, j] > 0
            else:
                q = distribution(draft[b, j], temperature)
                if 0 <= t < V and p[t] > 0:
                    ratio[b, j] = min(1.0, p[t] / q[t]) if q[t] > 0 else 1.0
                ok = float(u[b, j]) < ratio[b, j]
            if left is None and not ok:
                n[b] = j
                left = p if temperature == 0 else np.maximum(p - q, 0.0)
                if left.sum() == 0:
                    left = p
        if left is None:
            n[b], left = nd, distribution(target[b, nd], temperature)
        tokens[b, :n[b]] = x[b, :n[b]]
        if left.sum() > 0:
            c = np.cumsum(left)
            last = np.nonzero(left > 0)[0][-1]
            goal = 0.0 if temperature == 0 or not u[b, G] > 0 else float(u[b, G]) * c[-1]
            tokens[b, n[b]] = min(np.searchsorted(c, goal, side="right"), last)
    return n, tokens, ratio
