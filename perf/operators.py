"""Measured cases of the packed and paged attention operators.

Four kinds of pass, each as a program calls it:

  prompt  fa.forward_varlen: attention over packed sequences of different
          lengths (q, k, v either tensors of their own or slices of one fused
          projection), giving O and the log-sum-exp;
  train   the same followed by fa.backward_varlen: O, LSE, dQ, dK, dV;
  paged   fa.forward_paged: every sequence's new tokens (one token, a chunk,
          or a mixture of both) over a cache kept in pages;
  append  fa.cache_append: the new tokens' K and V written into that cache.

`run` computes them with elementary torch operations in 32 bits where `own`
is false, and with the framework's calls where it is true. `exact` is the
definition in 64 bits, one sequence and one head at a time.

A case's lengths are drawn from its own "lens_seed" (spread over their
logarithm, the longest always present), so that `work` follows from the case;
`prepare` puts them in an order of its seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False


def listed():
    return [
        # a short question to a small model with one head per kv head: nothing but latency
        dict(name="prompt_short", op="prompt", heads=2, kv_heads=2, dim=64, batch=1, min_new=77, max_new=77, page=0,
             min_ctx=0, max_ctx=0, causal=True, window=-1, fused=False, lens_seed=1),
        # prompts of many users packed together, read from the fused projection
        dict(name="prompt_packed", op="prompt", heads=32, kv_heads=8, dim=128, batch=16, min_new=16, max_new=4096,
             page=0, min_ctx=0, max_ctx=0, causal=True, window=-1, fused=True, lens_seed=2),
        # one long document beside a shorter one (the library's long causal grouped-head workload)
        dict(name="prompt_long", op="prompt", heads=32, kv_heads=8, dim=128, batch=2, min_new=5000, max_new=16384,
             page=0, min_ctx=0, max_ctx=0, causal=True, window=-1, fused=False, lens_seed=3),
        # a layer with a sliding window of 1024 keys over documents of odd lengths
        dict(name="prompt_window", op="prompt", heads=16, kv_heads=16, dim=128, batch=5, min_new=700, max_new=8191,
             page=0, min_ctx=0, max_ctx=0, causal=True, window=1023, fused=True, lens_seed=4),
        # a small model's training step on a few short samples
        dict(name="train_small", op="train", heads=8, kv_heads=4, dim=64, batch=6, min_new=33, max_new=500, page=0,
             min_ctx=0, max_ctx=0, causal=True, window=-1, fused=False, lens_seed=5),
        # a training step on documents packed into one row of about 16 thousand tokens
        dict(name="train_packed", op="train", heads=32, kv_heads=8, dim=128, batch=9, min_new=200, max_new=6000,
             page=0, min_ctx=0, max_ctx=0, causal=True, window=-1, fused=True, lens_seed=6),
        # one user, one token at a time, a short context: latency
        dict(name="decode_one", op="paged", heads=32, kv_heads=8, dim=128, batch=1, min_new=1, max_new=1, page=16,
             min_ctx=1000, max_ctx=1000, causal=True, window=-1, fused=False, lens_seed=7),
        # a busy server: one token of each of 64 sequences of very different lengths
        dict(name="decode_batch", op="paged", heads=32, kv_heads=8, dim=128, batch=64, min_new=1, max_new=1, page=64,
             min_ctx=300, max_ctx=32000, causal=True, window=-1, fused=True, lens_seed=8),
        # the next chunk of long prompts whose first part is in the cache
        dict(name="chunk_long", op="paged", heads=32, kv_heads=8, dim=128, batch=3, min_new=512, max_new=512, page=64,
             min_ctx=6000, max_ctx=16384, causal=True, window=-1, fused=True, lens_seed=9),
        # continuous batching: chunks and single tokens in one call, small heads, small pages
        dict(name="mixed_batch", op="paged", heads=16, kv_heads=2, dim=64, batch=24, min_new=1, max_new=400, page=16,
             min_ctx=100, max_ctx=8000, causal=True, window=-1, fused=True, lens_seed=10),
        # one new token of each of 100 sequences goes into the cache
        dict(name="append_tokens", op="append", heads=0, kv_heads=8, dim=128, batch=100, min_new=1, max_new=1, page=16,
             min_ctx=10, max_ctx=2000, causal=True, window=-1, fused=True, lens_seed=11),
        # whole prompts go into the cache
        dict(name="append_prompts", op="append", heads=0, kv_heads=8, dim=128, batch=12, min_new=500, max_new=12000,
             page=64, min_ctx=0, max_ctx=3000, causal=True, window=-1, fused=True, lens_seed=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "paged", "paged", "paged", "append"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dim = rng.choice([64, 128])
    c = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, causal=True, window=-1, fused=rng.random() < 0.5,
             lens_seed=rng.randrange(1 << 20), page=0, min_ctx=0, max_ctx=0)
    if op in ("prompt", "train"):
        c["batch"] = _spread(rng, 1, 24)
        # long sequences only in small batches: no case costs more than the largest listed one
        top = 9000 if c["batch"] <= 2 else 4000 if c["batch"] <= 6 else 1500
        c["max_new"] = _spread(rng, 1, top if op == "prompt" else top // 2)
        c["min_new"] = _spread(rng, 1, c["max_new"])
        c["causal"] = rng.random() < 0.75
        if c["causal"] and rng.random() < 0.3:
            c["window"] = _spread(rng, 1, 2000)
    elif op == "paged":
        c["page"] = rng.choice([16, 32, 48, 64, 128, 256])
        c["batch"] = _spread(rng, 1, 64)
        one = rng.random() < 0.5
        c["max_new"] = 1 if one else _spread(rng, 1, 600 if c["batch"] <= 8 else 150)
        c["min_new"] = 1 if one else _spread(rng, 1, c["max_new"])
        c["max_ctx"] = _spread(rng, 1, 40000 if c["batch"] <= 4 else 12000)
        c["min_ctx"] = _spread(rng, 1, c["max_ctx"])
        if rng.random() < 0.25:
            c["window"] = _spread(rng, 1, 5000)
    else:
        c["page"] = rng.choice([16, 32, 48, 64, 128, 256])
        c["batch"] = _spread(rng, 1, 200)
        c["max_new"] = _spread(rng, 1, 8000 if c["batch"] <= 8 else 300)
        c["min_new"] = _spread(rng, 1, c["max_new"])
        c["max_ctx"] = _spread(rng, 1, 4000)
        c["min_ctx"] = _spread(rng, 1, c["max_ctx"])
        c["heads"] = 0
    return c


def _lens(case):
    """(new tokens, tokens already in the cache) of each sequence."""
    rng = random.Random(case["lens_seed"])
    new = [_spread(rng, case["min_new"], case["max_new"]) for _ in range(case["batch"])]
    new[0] = case["max_new"]
    if case["op"] in ("prompt", "train"):
        return new, [0] * len(new)
    ctx = [_spread(rng, case["min_ctx"] + 1, case["max_ctx"] + 1) - 1 for _ in new]
    ctx[-1] = case["max_ctx"]
    return new, ctx


def prepare(case, seed):
    new, ctx = _lens(case)
    order = list(range(len(new)))
    random.Random(seed).shuffle(order)
    new, ctx = [new[i] for i in order], [ctx[i] for i in order]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hk, d, total = case["heads"], case["kv_heads"], case["dim"], sum(new)
    all_k = [n + c for n, c in zip(new, ctx)]

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)

    def starts(lens):
        out = [0]
        for n in lens:
            out.append(out[-1] + n)
        return torch.tensor(out, dtype=torch.int32, device="cuda")

    if case["fused"]:  # q, k, v of a token side by side, as one projection leaves them
        qkv = normal(total, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = normal(total, hq, d), normal(total, hk, d), normal(total, hk, d)
    s = dict(case=case, new=new, all_k=all_k, q=q, k=k, v=v, cu=starts(new), scale=d ** -0.5,
             window=None if case["window"] < 0 else (case["window"], 0))
    if case["op"] == "train":
        s["dout"] = normal(total, hq, d)
    if case["page"]:
        page = case["page"]
        need = [-(-n // page) for n in all_k]
        pages = sum(need) + 7  # some pages belong to nobody
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((len(new), max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        # rows past a sequence's end hold what earlier sequences left there
        s.update(k_pages=normal(pages, page, hk, d), v_pages=normal(pages, page, hk, d), table=table,
                 lens=torch.tensor(all_k, dtype=torch.int32, device="cuda"))
    return s


def _visible(case, rows, lq, lk, keys):
    """[B, rows, keys]: which keys each row of a padded batch sees."""
    i = rows[None, :, None] + (lk - lq)[:, None, None]
    j = keys[None, None, :]
    see = (j < lk[:, None, None]) & (rows[None, :, None] < lq[:, None, None])
    if case["causal"]:
        see = see & (j <= i)
    if case["window"] >= 0:
        see = see & (j >= i - case["window"])
    return see


def _attention(case, q, k, v, lq, lk, scale, dout=None):
    """Attention of a padded batch in 32 bits, some query rows at a time.
    q [B, Lq, Hq, d], k, v [B, Lk, Hk, d] (padding finite); returns O, LSE
    [B, Hq, Lq] and, where dout is given, dQ, dK, dV."""
    B, Lq, hq, d = q.shape
    Lk, hk = k.shape[1], k.shape[2]
    G = hq // hk
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)  # [B, Hk, Lk, d]
    o = torch.zeros((B, hk, G, Lq, d), device=q.device)
    lse = torch.zeros((B, hk, G, Lq), device=q.device)
    q5 = q.view(B, Lq, hk, G, d).permute(0, 2, 3, 1, 4)
    if dout is not None:
        do5 = dout.view(B, Lq, hk, G, d).permute(0, 2, 3, 1, 4)
        dq, dk, dv = torch.zeros_like(o), torch.zeros_like(k), torch.zeros_like(v)
    keys = torch.arange(Lk, device=q.device)
    step = max(1, min(Lq, (1 << 29) // (B * hq * Lk)))
    for r in range(0, Lq, step):
        rows = torch.arange(r, min(Lq, r + step), device=q.device)
        n = rows.numel()
        see = _visible(case, rows, lq, lk, keys)[:, None, None]
        qr = q5[:, :, :, r:r + n].reshape(B, hk, G * n, d)
        s = ((qr * scale) @ k.transpose(2, 3)).view(B, hk, G, n, Lk)
        s = torch.where(see, s, -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l > 0, l, 1.0)
        o_r = (p.view(B, hk, G * n, Lk) @ v).view(B, hk, G, n, d)
        o[:, :, :, r:r + n] = o_r
        lse[:, :, :, r:r + n] = (m + torch.log(l))[..., 0]
        if dout is not None:
            do_r = do5[:, :, :, r:r + n]
            dp = (do_r.reshape(B, hk, G * n, d) @ v.transpose(2, 3)).view(B, hk, G, n, Lk)
            ds = p * (dp - (do_r * o_r).sum(-1, keepdim=True))
            ds = ds.view(B, hk, G * n, Lk)
            dq[:, :, :, r:r + n] = scale * (ds @ k).view(B, hk, G, n, d)
            dk += scale * (ds.transpose(2, 3) @ qr)
            dv += p.view(B, hk, G * n, Lk).transpose(2, 3) @ do_r.reshape(B, hk, G * n, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, hq, d)
    lse = lse.view(B, hq, Lq)
    if dout is None:
        return o, lse
    return o, lse, dq.permute(0, 3, 1, 2, 4).reshape(B, Lq, hq, d), dk.permute(0, 2, 1, 3), dv.permute(0, 2, 1, 3)


def _tokens(cu, total):
    """Of each packed token: its sequence, and its place in it."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu, t.to(cu.dtype), right=True) - 1
    return b, t - cu[b]


def _plain(s):
    case, cu, q = s["case"], s["cu"], s["q"]
    total = s["k"].shape[0]
    b, i = _tokens(cu, total)
    lq = cu[1:] - cu[:-1]
    if case["op"] == "append":
        t = s["lens"][b] - lq[b] + i
        at = s["table"][b, t // case["page"]].long() * case["page"] + t % case["page"]
        s["k_pages"].view(-1, *s["k"].shape[1:])[at] = s["k"]
        s["v_pages"].view(-1, *s["v"].shape[1:])[at] = s["v"]
        return s["k_pages"], s["v_pages"]

    lens = torch.tensor(s["all_k"], device=cu.device)
    out = [torch.empty_like(q), torch.empty(q.shape[1::-1], device=cu.device)]
    if case["op"] == "train":
        out += [torch.empty_like(x) for x in (q, s["k"], s["v"])]
    for group in _alike(s["all_k"]):
        if len(group) == len(lens):  # all of them: as they are
            g = mine = slice(None)
            bg, ig = b, i
        else:
            g = torch.tensor(group, device=cu.device)
            slot = torch.full(lens.shape, -1, dtype=torch.long, device=cu.device)
            slot[g] = torch.arange(len(group), device=cu.device)
            mine = (slot[b] >= 0).nonzero()[:, 0]
            bg, ig = slot[b[mine]], i[mine]
        most = max(s["new"][j] for j in group)

        def padded(x):
            y = torch.zeros((len(group), most) + x.shape[1:], device=x.device)
            y[bg, ig] = x[mine].float()
            return y

        if case["op"] == "paged":
            pages = s["table"][g, : -(-max(s["all_k"][j] for j in group) // case["page"])].long()
            k, v = (x[pages].flatten(1, 2).float() for x in (s["k_pages"], s["v_pages"]))
        else:
            k, v = padded(s["k"]), padded(s["v"])
        r = _attention(case, padded(q), k, v, lq[g], lens[g], s["scale"], padded(s["dout"]) if case["op"] == "train" else None)
        out[1][:, mine] = r[1].permute(1, 0, 2)[:, bg, ig]
        for y, x in zip(out[:1] + out[2:], r[:1] + r[2:]):
            y[mine] = x[bg, ig].to(y.dtype)
    return tuple(out)


def _alike(lens):
    """Groups of sequences that are padded together: none is below half of its group's longest."""
    order = sorted(range(len(lens)), key=lambda j: -lens[j])
    groups = [[order[0]]]
    for j in order[1:]:
        if 2 * lens[j] >= lens[groups[-1][0]]:
            groups[-1].append(j)
        else:
            groups.append([j])
    return groups


def _own(s):
    import exact_attention_99_gb300 as fa
    case = s["case"]
    kw = dict(causal=case["causal"], scale=s["scale"], window=s["window"])
    if case["op"] == "append":
        fa.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["cu"], s["lens"], s["table"])
        return s["k_pages"], s["v_pages"]
    if case["op"] == "paged":
        return fa.forward_paged(s["q"], s["k_pages"], s["v_pages"], s["cu"], s["lens"], s["table"], **kw)
    o, lse = fa.forward_varlen(s["q"], s["k"], s["v"], s["cu"], s["cu"], **kw)
    if case["op"] == "prompt":
        return o, lse
    return (o, lse) + tuple(fa.backward_varlen(s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu"], s["cu"], **kw))


def run(state):
    return _own(state) if own else _plain(state)


def _pairs(case, n, c):
    """Visible (row, key) pairs of a sequence of n new tokens behind c old ones."""
    if not case["causal"]:
        return n * (n + c)
    w = case["window"] + 1 if case["window"] >= 0 else n + c
    # row i sees min(c + i + 1, w) keys
    short = min(max(w - c, 0), n)  # rows that see all there is
    return short * c + short * (short + 1) // 2 + (n - short) * w


def work(case):
    new, ctx = _lens(case)
    hq, hk, d, total = case["heads"], case["kv_heads"], case["dim"], sum(new)
    if case["op"] == "append":
        return {"bytes": 4 * 2 * total * hk * d, "flops": 0}
    keys = 0
    for n, c in zip(new, ctx):  # keys that some row sees
        keys += n + c if not case["causal"] or case["window"] < 0 else min(n + c, n + case["window"])
    pairs = sum(_pairs(case, n, c) for n, c in zip(new, ctx))
    b = 2 * 2 * total * hq * d + 2 * 2 * keys * hk * d + 4 * total * hq
    f = 4 * d * hq * pairs
    if case["op"] == "train":  # dO and dQ; dK and dV; five products more
        b += 2 * 2 * total * hq * d + 2 * 2 * total * hk * d
        f += 10 * d * hq * pairs
    return {"bytes": b, "flops": f}


def exact(case, seed):
    if case["op"] == "append":  # copies: there is nothing to compute
        return None
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    train = case["op"] == "train"
    total = s["q"].shape[0]
    out = {"o": torch.zeros((total, hq, d), dtype=torch.float64, device="cuda"),
           "lse": torch.zeros((hq, total), dtype=torch.float64, device="cuda")}
    if train:
        out["dq"] = torch.zeros_like(out["o"])
        out["dk"] = torch.zeros((total, hk, d), dtype=torch.float64, device="cuda")
        out["dv"] = torch.zeros_like(out["dk"])
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["all_k"])):
        here = slice(at, at + n)
        at += n
        # distance of each key from its row's own place: visible from -window to 0
        far = torch.arange(m, device="cuda")[None, :] - (torch.arange(n, device="cuda")[:, None] + (m - n))
        hidden = torch.zeros((n, m), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= far > 0
        if case["window"] >= 0:
            hidden |= far < -case["window"]
        for h in range(hk):
            if case["op"] == "paged":
                pages = s["table"][b, : -(-m // case["page"])].long()
                k, v = (x[pages, :, h].reshape(-1, d)[:m].double() for x in (s["k_pages"], s["v_pages"]))
            else:
                k, v = s["k"][here, h].double(), s["v"][here, h].double()
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                q = s["q"][here, g].double()
                a = torch.einsum("id,jd->ij", q, k).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                out["lse"][g, here] = torch.logsumexp(a, 1)
                a = torch.softmax(a, 1)
                out["o"][here, g] = a @ v
                if train:
                    do = s["dout"][here, g].double()
                    out["dv"][here, h] += a.T @ do
                    # the gradient of a softmax: its rows' changes, less their mean
                    c = do @ v.T
                    c -= (a * c).sum(1, keepdim=True)
                    a *= c
                    out["dq"][here, g] = s["scale"] * (a @ k)
                    out["dk"][here, h] += s["scale"] * (a.T @ q)
    return tuple(out[x] for x in ("o", "lse", "dq", "dk", "dv") if x in out)
