"""Cases of the serving operators around the split's draft and verify calls:
per-head norms of q and k with the rotary embedding, the append to a paged
cache, attention of a chunk of new tokens over that cache, and the acceptance
of drafted tokens. Shapes are those of the Llama-3-8B and Qwen3-8B steps of
the benchmark (32 query heads, 8 kv heads of 128; vocabularies of 128256 and
151936; 32K and 16K contexts; 4 and 6 drafted tokens) and generic ones."""
import math
import random

import numpy as np
import torch

own = False
D = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of one sequence (Qwen3-8B heads): latency counts
        dict(name="qk_norm_rope_1", op="qk", rows=1, hq=32, hkv=8, bf16=False, theta=1000000.0),
        # a prompt chunk whose QKV product came from a bf16 matrix product
        dict(name="qk_norm_rope_4096", op="qk", rows=4096, hq=32, hkv=8, bf16=True, theta=1000000.0),
        # the verify rows of two sequences, 6 drafted tokens + 1 each
        dict(name="append_2x7", op="append", batch=2, chunk=7, ctx=16384, ragged=False, hq=32, hkv=8, page=64,
             bf16=False, norm=True, theta=1000000.0),
        # ragged prompt chunks of 13 sequences, fp32 product, no head norms (Llama-3-8B)
        dict(name="append_13_ragged", op="append", batch=13, chunk=701, ctx=4001, ragged=True, hq=32, hkv=8, page=16,
             bf16=False, norm=False, theta=500000.0),
        # one long prompt chunk, bf16 product
        dict(name="append_4096", op="append", batch=1, chunk=4096, ctx=8192, ragged=False, hq=32, hkv=8, page=128,
             bf16=True, norm=True, theta=1000000.0),
        # one token of one sequence over the 32K context of the benchmark's step
        dict(name="attn_1x1_32k", op="attn", batch=1, chunk=1, ctx=32768, ragged=False, hq=32, hkv=8, page=64),
        # the verify rows of two sequences over 16K
        dict(name="attn_2x7_16k", op="attn", batch=2, chunk=7, ctx=16384, ragged=False, hq=32, hkv=8, page=64),
        # single tokens of 61 sequences of uneven lengths: a serving batch
        dict(name="attn_61x1_ragged", op="attn", batch=61, chunk=1, ctx=8191, ragged=True, hq=32, hkv=8, page=16),
        # ragged prompt chunks of 5 sequences, odd sizes
        dict(name="attn_5_ragged", op="attn", batch=5, chunk=777, ctx=5003, ragged=True, hq=32, hkv=8, page=32),
        # a long prompt's chunk late in a 32K context: the largest
        dict(name="attn_2048_32k", op="attn", batch=1, chunk=2048, ctx=32768, ragged=False, hq=32, hkv=8, page=128),
        # the end of a step: 4 drafted tokens of one sequence, Llama-3 vocabulary
        dict(name="spec_1x4", op="spec", batch=1, gamma=4, vocab=128256, temp=1.0, ragged=False, masked=False),
        # a serving batch with uneven numbers of drafted tokens and masked vocabularies
        dict(name="spec_29x6_ragged", op="spec", batch=29, gamma=6, vocab=151936, temp=0.7, ragged=True, masked=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["qk", "append", "attn", "attn", "spec"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8) if g * hkv <= 40])
    theta = rng.choice([10000.0, 500000.0, 1000000.0])
    if op == "qk":
        return dict(op=op, rows=_log(rng, 1, 4096), hq=hq, hkv=hkv, bf16=rng.random() < 0.5, theta=theta)
    if op == "append":
        batch = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(2, 4096 // batch))
        return dict(op=op, batch=batch, chunk=chunk, ctx=chunk + _log(rng, 1, 4096), ragged=rng.random() < 0.5, hq=hq,
                    hkv=hkv, page=rng.choice([16, 32, 64, 128]), bf16=rng.random() < 0.5, norm=rng.random() < 0.5,
                    theta=theta)
    if op == "attn":
        if rng.random() < 0.5:  # single tokens and short drafts of a batch
            batch, chunk = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5, 7, 16])
            ctx = chunk + _log(rng, 1, 131072 // batch)
        else:  # prompt chunks
            batch = _log(rng, 1, 8)
            chunk = _log(rng, 17, 2048 // batch)
            ctx = chunk + _log(rng, 1, 16384 // batch)
        return dict(op=op, batch=batch, chunk=chunk, ctx=ctx, ragged=rng.random() < 0.5, hq=hq, hkv=hkv,
                    page=rng.choice([16, 32, 64, 128]))
    return dict(op=op, batch=_log(rng, 1, 24), gamma=rng.randint(1, 7), vocab=_log(rng, 1000, 151936),
                temp=rng.choice([0.6, 0.7, 1.0, 1.3]), ragged=rng.random() < 0.5, masked=rng.random() < 0.5)


def _lengths(case):
    """(tokens in the chunk, tokens in the cache with the chunk) of every sequence."""
    B, T, L = case["batch"], case["chunk"], case["ctx"]
    if not case["ragged"]:
        return [T] * B, [L] * B
    r = random.Random(B * 1000003 + T * 1009 + L)
    t = [r.randint(1, T) for _ in range(B)]
    return t, [max(x, r.randint(x, L)) for x in t]


def _drafts(case):
    B, g = case["batch"], case["gamma"]
    if not case["ragged"]:
        return [g] * B
    r = random.Random(B * 1000003 + g * 1009 + case["vocab"])
    return [r.randint(0, g) for _ in range(B)]


# ------------------------------------------------------------------ inputs
def _paged(case, g, dev):
    t, n = _lengths(case)
    B, S, H = case["batch"], case["page"], case["hkv"]
    width = max(-(-x // S) for x in n)
    used = [-(-x // S) for x in n]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
    # keys and values with uneven channels, as caches have
    sc = torch.exp(0.5 * torch.randn(2, 1, 1, H, D, generator=g, device=dev))
    pools = [(torch.randn(n_pages, S, H, D, generator=g, device=dev) * sc[i]).to(torch.bfloat16) for i in (0, 1)]
    row_start = torch.tensor([0] + list(np.cumsum(t)), dtype=torch.int32, device=dev)
    kv_len = torch.tensor(n, dtype=torch.int32, device=dev)
    return dict(k=pools[0], v=pools[1], table=table, row_start=row_start, kv_len=kv_len, rows=sum(t), longest=max(t))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("qk", "append"):
        if op == "append":
            s.update(_paged(case, g, dev))
        heads = case["hq"] + 2 * case["hkv"]
        x = torch.randn(s["rows"], heads * D, generator=g, device=dev) * 2.0
        s["qkv"] = x.to(torch.bfloat16) if case["bf16"] else x
        s["gamma_q"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        s["gamma_k"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        if op == "qk":  # positions of a packed batch
            s["pos"] = torch.randint(0, 131072, (s["rows"],), generator=g, device=dev, dtype=torch.int32)
    elif op == "attn":
        s.update(_paged(case, g, dev))
        s["q"] = (1.5 * torch.randn(s["rows"], case["hq"], D, generator=g, device=dev)).to(torch.bfloat16)
    else:
        B, G, V = case["batch"], case["gamma"], case["vocab"]
        # a few likely tokens over a broad tail; the draft is the target with noise
        base = 2.5 * torch.randn(B, G + 1, V, generator=g, device=dev)
        s["target"] = base
        s["draft"] = base[:, :G] + 0.7 * torch.randn(B, G, V, generator=g, device=dev)
        if case["masked"]:  # tokens that a grammar forbids
            off = torch.rand(B, 1, V, generator=g, device=dev) < 0.1
            s["target"] = s["target"].masked_fill(off, float("-inf"))
            s["draft"] = s["draft"].masked_fill(off, float("-inf"))
        race = torch.rand(B, G, V, generator=g, device=dev).clamp_(1e-9, 1 - 1e-7)
        s["x"] = (s["draft"] / case["temp"] - torch.log(-torch.log(race))).argmax(-1).to(torch.int32)
        s["u"] = torch.rand(B, G + 1, generator=g, device=dev)
        s["n_draft"] = torch.tensor(_drafts(case), dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, theta):
    """x [rows][heads][128], pos [rows]: pairs (i, i + 64) turn by pos * theta^(-i/64), the angle in 64 bits."""
    i = torch.arange(64, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * torch.exp(i * (-math.log(theta) / 64))
    c, s = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _head_norm(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.float()


def _split(s, pos, norm):
    hq, hkv = s["hq"], s["hkv"]
    h = s["qkv"].float().view(-1, hq + 2 * hkv, D)
    q, k, v = h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:]
    if norm:
        q, k = _head_norm(q, s["gamma_q"]), _head_norm(k, s["gamma_k"])
    return tuple(t.to(torch.bfloat16) for t in (_rotate(q, pos, s["theta"]), _rotate(k, pos, s["theta"]), v))


def _row_places(s):
    """(sequence, position) of every row."""
    r = torch.arange(s["rows"], device=s["kv_len"].device)
    seq = torch.searchsorted(s["row_start"][1:].long(), r, right=True)
    start, end = s["row_start"].long()[seq], s["row_start"].long()[seq + 1]
    return seq, s["kv_len"].long()[seq] - (end - start) + (r - start)


def _plain_append(s):
    seq, pos = _row_places(s)
    q, k, v = _split(s, pos, s["norm"])
    page = s["table"].long()[seq, pos // s["page"]]
    s["k"][page, pos % s["page"]] = k
    s["v"][page, pos % s["page"]] = v
    return q, s["k"], s["v"]


def _plain_attn(s):
    hq, hkv, B, T = s["hq"], s["hkv"], s["batch"], s["longest"]
    seq, pos = _row_places(s)
    at = torch.arange(s["rows"], device=seq.device) - s["row_start"].long()[seq]
    q = torch.zeros(B, T, hq, D, device=seq.device)
    q[seq, at] = s["q"].float()
    where = torch.full((B, T), -1, device=seq.device)
    where[seq, at] = pos
    n = s["table"].shape[1] * s["page"]
    k = s["k"][s["table"].long()].reshape(B, n, hkv, D).permute(0, 2, 3, 1).float()   # [B][H][128][n]
    v = s["v"][s["table"].long()].reshape(B, n, hkv, D).permute(0, 2, 1, 3).float()   # [B][H][n][128]
    # a kv head's query heads are rows of one product: [B][H][T * group][128]
    q = q.view(B, T, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * (hq // hkv), D)
    p = (q @ k).mul_(1 / math.sqrt(D)).view(B, hkv, T, hq // hkv, n)
    seen = torch.arange(n, device=seq.device) <= where[..., None]                     # [B][T][n]
    p.masked_fill_(~seen[:, None, :, None], float("-inf"))
    p = torch.exp_(p.sub_(p.amax(-1, keepdim=True).clamp_min_(-3e38))).view(B, hkv, T * (hq // hkv), n)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min_(1e-38)
    o = o.view(B, hkv, T, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, hq, D)
    return o[seq, at].to(torch.bfloat16)


def _plain_spec(s):
    B, G, V, temp = s["batch"], s["gamma"], s["vocab"], s["temp"]
    dev = s["u"].device
    x, n_draft = s["x"].long(), s["n_draft"].long()

    def chosen(logits):  # probability of x under each row
        z = (logits - logits.amax(-1, keepdim=True)) / temp
        return torch.exp(z.gather(-1, x[..., None]))[..., 0] / torch.exp(z).sum(-1)

    p, q = chosen(s["target"][:, :G]), chosen(s["draft"])
    j = torch.arange(G, device=dev)
    drafted = j < n_draft[:, None]
    ratio = torch.where(drafted, (p / q).clamp_max(1), torch.zeros_like(p))
    n = (s["u"][:, :G] < ratio).long().cumprod(-1).sum(-1)
    # the next token's border lies between sums over the vocabulary: 64 bits
    b = torch.arange(B, device=dev)

    def row(logits):
        z = torch.exp((logits.double() - logits.double().amax(-1, keepdim=True)) / temp)
        return z / z.sum(-1, keepdim=True)

    pn = row(s["target"][b, n])
    qn = row(s["draft"][b, n.clamp_max(G - 1)]) * (n < n_draft)[:, None]
    c = (pn - qn).clamp_min(0).cumsum(-1)
    nxt = (c <= s["u"][:, G:].double() * c[:, -1:]).sum(-1)
    j = torch.arange(G + 1, device=dev)
    tokens = torch.where(j < n[:, None], torch.cat([x, x[:, :1]], 1), torch.full_like(j, -1))
    tokens = torch.where(j == n[:, None], nxt[:, None], tokens)
    return n.to(torch.int32), tokens.to(torch.int32), ratio


def run(state):
    s = state
    op = s["op"]
    if own:
        import bit_level_weight_gb300 as cas
        bf = torch.bfloat16
        if op == "qk":
            q, k, v = cas.qk_norm_rope(s["qkv"], s["hq"], s["hkv"], s["gamma_q"], s["gamma_k"], 1e-6, pos=s["pos"],
                                       theta=s["theta"])
            return q.view(bf), k.view(bf), v.view(bf)
        if op == "append":
            gq, gk = (s["gamma_q"], s["gamma_k"]) if s["norm"] else (None, None)
            q = cas.paged_append(s["qkv"], s["hq"], s["k"], s["v"], s["row_start"], s["kv_len"], s["table"], gq, gk,
                                 1e-6, s["theta"])
            return q.view(bf), s["k"], s["v"]
        if op == "attn":
            return cas.paged_attn(s["q"], s["k"], s["v"], s["row_start"], s["kv_len"], s["table"]).view(bf)
        return cas.spec_verify(s["target"], s["draft"], s["x"], s["u"], s["n_draft"], s["temp"])
    if op == "qk":
        return _split(s, s["pos"], True)
    if op == "append":
        return _plain_append(s)
    return _plain_attn(s) if op == "attn" else _plain_spec(s)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "spec":
        g = case["gamma"]
        rows = sum(2 * n + 1 for n in _drafts(case))  # every logit that decides something, once
        return {"bytes": 4.0 * rows * case["vocab"] + case["batch"] * (2 * g + 1) * 8, "flops": 4.0 * rows * case["vocab"]}
    heads = case["hq"] + 2 * case["hkv"]
    if op in ("qk", "append"):
        rows = case["rows"] if op == "qk" else sum(_lengths(case)[0])
        return {"bytes": float(rows * heads * D * ((2 if case["bf16"] else 4) + 2)), "flops": 10.0 * rows * heads * D}
    t, n = _lengths(case)
    pairs = sum(x * (m - x) + x * (x + 1) // 2 for x, m in zip(t, n))
    return {"bytes": float(sum(n) * case["hkv"] * D * 4 + sum(t) * case["hq"] * D * 4),
            "flops": 4.0 * D * case["hq"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_heads(case, s, pos, norm):
    heads = case["hq"] + 2 * case["hkv"]
    x = s["qkv"].double().view(-1, heads, D)
    out = []
    z = torch.polar(torch.ones(len(pos), 64, dtype=torch.float64, device=x.device),
                    pos.double()[:, None] * case["theta"] ** (-torch.arange(64, device=x.device).double() / 64))
    for lo, hi, gamma in ((0, case["hq"], s["gamma_q"]), (case["hq"], heads - case["hkv"], s["gamma_k"])):
        h = x[:, lo:hi]
        if norm:
            h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / D + 1e-6) * gamma.double()
        turned = torch.complex(h[..., :64].contiguous(), h[..., 64:].contiguous()) * z[:, None]
        out.append(torch.cat([turned.real, turned.imag], -1))
    return out[0], out[1], x[:, heads - case["hkv"]:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "qk":
        return _exact_heads(case, s, s["pos"], True)
    if op == "spec":
        return _exact_spec(case, s)
    t, n = _lengths(case)
    S, r = case["page"], 0
    if op == "append":
        pos = torch.cat([torch.arange(m - x, m) for x, m in zip(t, n)]).cuda()
        q, k, v = _exact_heads(case, s, pos, case["norm"])
        pools = s["k"].double(), s["v"].double()
        table = s["table"].cpu().tolist()
        for b, (x, m) in enumerate(zip(t, n)):
            flat = torch.tensor([table[b][p // S] * S + p % S for p in range(m - x, m)]).cuda()
            for pool, new in zip(pools, (k, v)):
                pool.view(-1, case["hkv"], D)[flat] = new[r:r + x]
            r += x
        return q, pools[0], pools[1]
    out, group = [], case["hq"] // case["hkv"]
    for b, (x, m) in enumerate(zip(t, n)):
        pages = s["table"][b, :-(-m // S)].long()
        k, v = (s[w][pages].reshape(-1, case["hkv"], D)[:m].double() for w in ("k", "v"))
        late = torch.ones(x, m, dtype=torch.bool, device=k.device).triu(m - x + 1)
        heads = []
        for h in range(case["hq"]):
            w = s["q"][r:r + x, h].double() @ k[:, h // group].T / math.sqrt(D)
            w = torch.softmax(w.masked_fill(late, -math.inf), -1)
            heads.append(w @ v[:, h // group])
        out.append(torch.stack(heads, 1))
        r += x
    return torch.cat(out)


def _exact_spec(case, s):
    B, G = case["batch"], case["gamma"]
    u, x = s["u"].cpu().numpy().astype(np.float64), s["x"].cpu().numpy()
    n, tokens = np.zeros(B, np.int32), np.full((B, G + 1), -1, np.int32)
    ratio = np.zeros((B, G))

    def probabilities(row):
        w = np.exp((row - row.max()) / case["temp"])
        return w / w.sum()

    for b, drafted in enumerate(_drafts(case)):
        target = s["target"][b].cpu().numpy().astype(np.float64)
        draft = s["draft"][b].cpu().numpy().astype(np.float64)
        left = None
        for j in range(drafted):
            p, q = probabilities(target[j]), probabilities(draft[j])
            ratio[b, j] = min(1.0, p[x[b, j]] / q[x[b, j]])
            if left is None and not u[b, j] < ratio[b, j]:
                left, n[b] = np.maximum(p - q, 0), j
        if left is None:
            left, n[b] = probabilities(target[drafted]), drafted
        c = np.cumsum(left)
        tokens[b, :n[b]] = x[b, :n[b]]
        tokens[b, n[b]] = np.searchsorted(c, u[b, G] * c[-1], side="right")
    return torch.from_numpy(n), torch.from_numpy(tokens), torch.from_numpy(ratio)
