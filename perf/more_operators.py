"""Measured cases of rotary positions and of a cache held in 8 bits.

Four kinds of pass, each as a program calls it:

  rotary        fa.rotary: q and k of packed tokens (tensors of their own or
                slices of one fused projection) turned by their places, which
                follow from the sequences' lengths;
  rotary_train  the same followed by fa.rotary_backward of the gradients that
                the attention's backward pass hands back;
  append        fa.cache_append_fp8: the new tokens' K and V rounded to e4m3,
                with a power of two as the scale of each block of 16 tokens
                and head, and written into the pages;
  attend        fa.forward_paged_fp8: every sequence's new tokens (one token, a
                chunk, or a mixture of both) over such a cache.

`run` computes them with elementary torch operations in 32 bits (angles in 64)
where `own` is false, and with the framework's calls where it is true. `exact`
is the definition in 64 bits, one sequence and one head at a time.

A case's lengths are drawn from its own "lens_seed" (spread over their
logarithm, the longest always present), so that `work` follows from the case;
`prepare` puts them in an order of its seed.

The scale of a block is 2^e with the smallest whole e, -64 at least, for which
every finite value of its rows is at most 448 * 2^e. Rows that come into a
block which holds some already leave its scale or raise it; raised, the rows
held are rounded again in the new scale.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16  # tokens of a block that has a scale


def listed():
    rope = dict(interleaved=False, rot=128, factor=1.0)
    cache = dict(interleaved=False, rot=0, factor=1.0)
    return [
        # one user's next token: nothing but latency
        dict(name="rotary_one", op="rotary", heads=32, kv_heads=8, dim=128, batch=1, min_new=1, max_new=1, page=0,
             min_ctx=1000, max_ctx=1000, window=-1, fused=True, lens_seed=21, **rope),
        # chunks of prompts far into long contexts (frequencies scaled by 8), read from the fused projection
        dict(name="rotary_prompts", op="rotary", heads=32, kv_heads=8, dim=128, batch=16, min_new=16, max_new=4096,
             page=0, min_ctx=0, max_ctx=200000, window=-1, fused=True, lens_seed=22, interleaved=False, rot=128, factor=8.0),
        # a small model's training step on short samples, a quarter of the head turned
        dict(name="rotary_train_small", op="rotary_train", heads=8, kv_heads=4, dim=64, batch=6, min_new=33, max_new=500,
             page=0, min_ctx=0, max_ctx=0, window=-1, fused=False, lens_seed=23, interleaved=False, rot=16, factor=1.0),
        # a training step on packed documents, neighbours paired, half of the head turned
        dict(name="rotary_train", op="rotary_train", heads=32, kv_heads=8, dim=128, batch=9, min_new=200, max_new=6000,
             page=0, min_ctx=0, max_ctx=0, window=-1, fused=True, lens_seed=24, interleaved=True, rot=64, factor=1.0),
        # one new token of each of 100 sequences goes into the cache
        dict(name="append_tokens", op="append", heads=0, kv_heads=8, dim=128, batch=100, min_new=1, max_new=1, page=16,
             min_ctx=10, max_ctx=2000, window=-1, fused=True, lens_seed=25, **cache),
        # whole prompts go into the cache
        dict(name="append_prompts", op="append", heads=0, kv_heads=8, dim=128, batch=12, min_new=500, max_new=12000,
             page=64, min_ctx=0, max_ctx=3000, window=-1, fused=True, lens_seed=26, **cache),
        # one user, one token at a time, a short context: latency
        dict(name="attend_one", op="attend", heads=32, kv_heads=8, dim=128, batch=1, min_new=1, max_new=1, page=16,
             min_ctx=1000, max_ctx=1000, window=-1, fused=False, lens_seed=27, **cache),
        # a busy server: one token of each of 64 sequences of very different lengths
        dict(name="attend_batch", op="attend", heads=32, kv_heads=8, dim=128, batch=64, min_new=1, max_new=1, page=64,
             min_ctx=300, max_ctx=32000, window=-1, fused=True, lens_seed=28, **cache),
        # two users with very long documents, eight query heads to a kv head
        dict(name="attend_long", op="attend", heads=64, kv_heads=8, dim=128, batch=2, min_new=1, max_new=1, page=256,
             min_ctx=60000, max_ctx=131000, window=-1, fused=False, lens_seed=29, **cache),
        # the next chunk of long prompts whose first part is in the cache
        dict(name="attend_chunk", op="attend", heads=32, kv_heads=8, dim=128, batch=3, min_new=512, max_new=512, page=64,
             min_ctx=6000, max_ctx=16384, window=-1, fused=True, lens_seed=30, **cache),
        # continuous batching: chunks and single tokens in one call, small heads, small pages
        dict(name="attend_mixed", op="attend", heads=16, kv_heads=2, dim=64, batch=24, min_new=1, max_new=400, page=16,
             min_ctx=100, max_ctx=8000, window=-1, fused=True, lens_seed=31, **cache),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_train", "append", "append", "attend", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dim = rng.choice([64, 128])
    c = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, window=-1, fused=rng.random() < 0.5,
             lens_seed=rng.randrange(1 << 20), page=0, min_ctx=0, max_ctx=0, interleaved=False, rot=0, factor=1.0)
    if op in ("rotary", "rotary_train"):
        c["batch"] = _spread(rng, 1, 64)
        c["max_new"] = _spread(rng, 1, 6000 if c["batch"] <= 6 else 500)
        c["min_new"] = _spread(rng, 1, c["max_new"])
        if op == "rotary":
            c["max_ctx"] = _spread(rng, 1, 1000000)
            c["min_ctx"] = _spread(rng, 1, c["max_ctx"])
        c["interleaved"] = rng.random() < 0.5
        c["rot"] = 16 * rng.randint(1, dim // 16)
        c["factor"] = rng.choice([1.0, 4.0, 32.0])
        return c
    c["page"] = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "attend":
        c["batch"] = _spread(rng, 1, 64)
        one = rng.random() < 0.5
        c["max_new"] = 1 if one else _spread(rng, 1, 600 if c["batch"] <= 8 else 150)
        c["min_new"] = 1 if one else _spread(rng, 1, c["max_new"])
        c["max_ctx"] = _spread(rng, 1, 40000 if c["batch"] <= 4 else 12000)
        c["min_ctx"] = _spread(rng, 1, c["max_ctx"])
        if rng.random() < 0.25:
            c["window"] = _spread(rng, 1, 5000)
    else:
        c["heads"] = 0
        c["batch"] = _spread(rng, 1, 200)
        c["max_new"] = _spread(rng, 1, 8000 if c["batch"] <= 8 else 300)
        c["min_new"] = _spread(rng, 1, c["max_new"])
        c["max_ctx"] = _spread(rng, 1, 4000)
        c["min_ctx"] = _spread(rng, 1, c["max_ctx"])
    return c


def _lens(case):
    """(new tokens, tokens before them) of each sequence."""
    rng = random.Random(case["lens_seed"])
    new = [_spread(rng, case["min_new"], case["max_new"]) for _ in range(case["batch"])]
    new[0] = case["max_new"]
    if case["op"] == "rotary_train":
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
             lens=torch.tensor(all_k, dtype=torch.int32, device="cuda"),
             window=None if case["window"] < 0 else (case["window"], 0))
    if case["rot"]:
        # inverse frequencies of base 10000; for longer contexts than the
        # model's first ones, all of them divided by the factor
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / case["rot"]) / case["factor"]).float().cuda()
        s["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
    if case["op"] == "rotary_train":
        s["dq"], s["dk"] = normal(total, hq, d), normal(total, hk, d)
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

        def held():  # rows past a sequence's end hold what earlier sequences left there
            codes = torch.empty((pages, page, hk, d), dtype=torch.float8_e4m3fn, device="cuda")
            for p in range(0, pages, 4096):
                n = min(pages, p + 4096) - p
                codes[p:p + n] = (torch.randn((n, page, hk, d), generator=g, device="cuda") * 90.0).clamp(-448, 448).to(codes.dtype)
            e = torch.randint(-8, -5, (pages, page // BLOCK, hk), generator=g, device="cuda")
            return codes, torch.exp2(e.float())

        (s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]) = held(), held()
        s["table"] = table
    return s


def _tokens(cu, total):
    """Of each packed token: its sequence, and its place in it."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu, t.to(cu.dtype), right=True) - 1
    return b, t - cu[b]


# --- rotary positions ------------------------------------------------------------

def _turn(case, x, cos, sin):
    """x [tokens, heads, d] in 32 bits, turned: pair (a, b) becomes (a cos - b sin, b cos + a sin)."""
    r = case["rot"]
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        t = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        t = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((t, y[..., r:]), -1).to(x.dtype)


def _rotary(s, place):
    a = place.double()[:, None] * s["inv_freq"].double()  # angles: 32 bits lose those of far places
    cos, sin = (s["mscale"] * f(a).float()[:, None] for f in (torch.cos, torch.sin))
    case = s["case"]
    out = [_turn(case, s["q"], cos, sin), _turn(case, s["k"], cos, sin)]
    if case["op"] == "rotary_train":  # the transposed turn: back by the same angle
        out += [_turn(case, s["dq"], cos, -sin), _turn(case, s["dk"], cos, -sin)]
    return tuple(out)


# --- the cache -------------------------------------------------------------------

def _exponent(amax):
    """The smallest e >= -64 with amax <= 448 * 2^e (448 = 1.75 * 2^8)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, -64).clamp(min=-64)


def _append(s, b, i):
    case = s["case"]
    lq = s["cu"][1:] - s["cu"][:-1]
    t = s["lens"][b] - lq[b] + i  # place in the sequence
    page = s["table"][b, t // case["page"]].long()
    row = page * case["page"] + t % case["page"]
    block = row // BLOCK
    # rows of its block before the first new one hold what the sequence has already
    first = (s["lens"] - lq)[b]
    old = torch.where(t // BLOCK == first // BLOCK, first % BLOCK, 0)
    for x, pages, scales in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        hk, d = x.shape[1:]
        codes = pages.view(-1, BLOCK, hk, d)
        sc = scales.view(-1, hk)
        amax = torch.zeros_like(sc)
        amax.index_reduce_(0, block, x.float().abs().amax(-1), "amax")
        new = torch.exp2(_exponent(amax[block]).float())
        before = sc[block]
        after = torch.where(old[:, None] > 0, torch.maximum(before, new), new)
        # the rows held, in the new scale (one token speaks for its block)
        mine = ((t % BLOCK == old) & (old > 0)).nonzero()[:, 0]
        blk = block[mine]
        kept = codes[blk].float() * (before[mine] / after[mine])[:, None, :, None]
        held = torch.arange(BLOCK, device=x.device)[None, :] < old[mine][:, None]
        where, which = held.nonzero(as_tuple=True)
        codes[blk[where], which] = kept[where, which].to(codes.dtype)
        pages.view(-1, hk, d)[row] = (x.float() / after[:, :, None]).to(codes.dtype)
        sc[block] = after
    return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _visible(case, rows, lq, lk, keys):
    """[B, rows, keys]: which keys each row of a padded batch sees."""
    i = rows[None, :, None] + (lk - lq)[:, None, None]
    j = keys[None, None, :]
    see = (j < lk[:, None, None]) & (rows[None, :, None] < lq[:, None, None]) & (j <= i)
    if case["window"] >= 0:
        see = see & (j >= i - case["window"])
    return see


def _attention(case, q, k, v, lq, lk, scale):
    """Attention of a padded batch in 32 bits, some query rows at a time.
    q [B, Lq, Hq, d], k, v [B, Lk, Hk, d]; returns O and LSE [B, Hq, Lq]."""
    B, Lq, hq, d = q.shape
    Lk, hk = k.shape[1], k.shape[2]
    G = hq // hk
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)  # [B, Hk, Lk, d]
    o = torch.zeros((B, hk, G, Lq, d), device=q.device)
    lse = torch.zeros((B, hk, G, Lq), device=q.device)
    q5 = q.view(B, Lq, hk, G, d).permute(0, 2, 3, 1, 4)
    keys = torch.arange(Lk, device=q.device)
    step = max(1, min(Lq, (1 << 29) // (B * hq * Lk)))
    for r in range(0, Lq, step):
        rows = torch.arange(r, min(Lq, r + step), device=q.device)
        n = rows.numel()
        see = _visible(case, rows, lq, lk, keys)[:, None, None]
        qr = q5[:, :, :, r:r + n].reshape(B, hk, G * n, d)
        a = ((qr * scale) @ k.transpose(2, 3)).view(B, hk, G, n, Lk)
        a = torch.where(see, a, -math.inf)
        m = a.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(a - m)
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l > 0, l, 1.0)
        o[:, :, :, r:r + n] = (p.view(B, hk, G * n, Lk) @ v).view(B, hk, G, n, d)
        lse[:, :, :, r:r + n] = (m + torch.log(l))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, hq, d), lse.view(B, hq, Lq)


def _attend(s, b, i):
    case, cu, q = s["case"], s["cu"], s["q"]
    lq = cu[1:] - cu[:-1]
    lens = s["lens"].long()
    o, lse = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(q.shape[1::-1], device=cu.device)
    for group in _alike(s["all_k"]):
        g = torch.tensor(group, device=cu.device)
        slot = torch.full(lens.shape, -1, dtype=torch.long, device=cu.device)
        slot[g] = torch.arange(len(group), device=cu.device)
        mine = (slot[b] >= 0).nonzero()[:, 0]
        bg, ig = slot[b[mine]], i[mine]
        pages = s["table"][g, : -(-max(s["all_k"][j] for j in group) // case["page"])].long()
        k, v = ((x[pages].float().unflatten(2, (-1, BLOCK)) * c[pages][:, :, :, None, :, None]).flatten(1, 3)
                for x, c in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
        padded = torch.zeros((len(group), max(s["new"][j] for j in group)) + q.shape[1:], device=q.device)
        padded[bg, ig] = q[mine].float()
        x, y = _attention(case, padded, k, v, lq[g], lens[g], s["scale"])
        o[mine] = x[bg, ig].to(o.dtype)
        lse[:, mine] = y.permute(1, 0, 2)[:, bg, ig]
    return o, lse


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


def _plain(s):
    op = s["case"]["op"]
    b, i = _tokens(s["cu"], s["k"].shape[0])
    if op == "append":
        return _append(s, b, i)
    if op == "attend":
        return _attend(s, b, i)
    lq = s["cu"][1:] - s["cu"][:-1]
    return _rotary(s, i if op == "rotary_train" else (s["lens"] - lq)[b] + i)


def _own(s):
    import exact_attention_99_gb300 as fa
    case = s["case"]
    if case["op"] == "append":
        fa.cache_append_fp8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["cu"], s["lens"],
                            s["table"])
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if case["op"] == "attend":
        return fa.forward_paged_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["cu"], s["lens"],
                                    s["table"], causal=True, scale=s["scale"], window=s["window"])
    kw = dict(interleaved=case["interleaved"], mscale=s["mscale"])
    if case["op"] == "rotary":
        return fa.rotary(s["q"], s["k"], s["inv_freq"], s["cu"], s["lens"], **kw)
    q, k = fa.rotary(s["q"], s["k"], s["inv_freq"], s["cu"], **kw)
    return (q, k) + tuple(fa.rotary_backward(s["dq"], s["dk"], s["inv_freq"], s["cu"], **kw))


def run(state):
    return _own(state) if own else _plain(state)


def _pairs(case, n, c):
    """Visible (row, key) pairs of a sequence of n new tokens behind c old ones."""
    w = case["window"] + 1 if case["window"] >= 0 else n + c
    # row i sees min(c + i + 1, w) keys
    short = min(max(w - c, 0), n)  # rows that see all there is
    return short * c + short * (short + 1) // 2 + (n - short) * w


def work(case):
    new, ctx = _lens(case)
    hq, hk, d, total = case["heads"], case["kv_heads"], case["dim"], sum(new)
    if case["op"] in ("rotary", "rotary_train"):
        both = 2 if case["op"] == "rotary_train" else 1
        return {"bytes": both * 2 * 2 * total * (hq + hk) * d, "flops": both * 3 * total * (hq + hk) * case["rot"]}
    if case["op"] == "append":  # 2 bytes of each value read, one written, 4 for a block's scale
        blocks = sum((n + c - 1) // BLOCK - c // BLOCK + 1 for n, c in zip(new, ctx))
        return {"bytes": 2 * 3 * total * hk * d + 2 * 4 * blocks * hk, "flops": 2 * 2 * total * hk * d}
    keys = 0
    for n, c in zip(new, ctx):  # keys that some row sees
        keys += n + c if case["window"] < 0 else min(n + c, n + case["window"])
    pairs = sum(_pairs(case, n, c) for n, c in zip(new, ctx))
    return {"bytes": 2 * 2 * total * hq * d + 2 * keys * hk * d + 2 * 4 * keys * hk // BLOCK + 4 * total * hq,
            "flops": 4 * d * hq * pairs}


# --- the definitions in 64 bits ----------------------------------------------------

def _exact_rotary(s):
    case = s["case"]
    train, r = case["op"] == "rotary_train", case["rot"]
    out = []
    for x, back in [(s["q"], 1), (s["k"], 1)] + ([(s["dq"], -1), (s["dk"], -1)] if train else []):
        y = x.double().clone()
        at = 0
        for n, m in zip(s["new"], s["all_k"]):
            p = torch.arange(m - n, m, device="cuda", dtype=torch.float64)
            turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device="cuda"),
                               back * torch.outer(p, s["inv_freq"].double()))[:, None]
            z = y[at:at + n]
            a, b = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            w = torch.complex(z[..., a], z[..., b]) * turn
            z[..., a], z[..., b] = w.real, w.imag
            at += n
        out.append(y)
    return tuple(out)


def _exact_append(s):
    """Codes before their rounding, and the scales."""
    case = s["case"]
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    out = []
    for x, pages, scales in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        rows = pages.double().view(-1, hk, d)
        blocks = scales.double().reshape(-1, hk)
        at = 0
        for b, (n, m) in enumerate(zip(s["new"], s["all_k"])):
            # the sequence from the start of the first block that gets a row
            c = m - n
            lo = c - c % BLOCK
            j = torch.arange(lo, m, device="cuda")
            row = s["table"][b, j // page].long() * page + j % page
            ids = row // BLOCK
            vals = rows[row]
            vals[:c - lo] *= blocks[ids[:c - lo]][:, :, None]
            vals[c - lo:] = x[at:at + n].double()
            at += n
            big = vals.abs().amax(-1)
            big[:c - lo] = 0  # of the new rows
            nb = -(-(m - lo) // BLOCK)
            pad = torch.zeros((nb * BLOCK, hk), dtype=torch.float64, device="cuda")
            pad[:m - lo] = big
            most = pad.view(nb, BLOCK, hk).amax(1)
            e = torch.ceil(torch.log2(most.clamp(min=1e-300) / 448.0)).clamp(min=-64.0)
            e += (448.0 * torch.exp2(e) < most).double()  # where log2 is off by its last bit
            e -= ((448.0 * torch.exp2(e - 1) >= most) & (e > -64)).double()
            sc = torch.exp2(e)
            heads = ids[::BLOCK]
            if c > lo:
                sc[0] = torch.maximum(sc[0], blocks[heads[0]])
            blocks[heads] = sc
            rows[row] = vals / sc.repeat_interleave(BLOCK, 0)[:m - lo, :, None]
        out.append((rows.view(pages.shape), blocks.view(scales.shape)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_attend(s):
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    total = s["q"].shape[0]
    o = torch.zeros((total, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((hq, total), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["all_k"])):
        here = slice(at, at + n)
        at += n
        # distance of each key from its row's own place: visible from -window to 0
        far = torch.arange(m, device="cuda")[None, :] - (torch.arange(n, device="cuda")[:, None] + (m - n))
        hidden = far > 0
        if case["window"] >= 0:
            hidden |= far < -case["window"]
        pages = s["table"][b, : -(-m // case["page"])].long()
        for h in range(hk):
            k, v = ((x[pages, :, h].double().view(-1, BLOCK, d) * c[pages, :, h].double().view(-1, 1, 1)).view(-1, d)[:m]
                    for x, c in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                a = (s["q"][here, g].double() @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                lse[g, here] = torch.logsumexp(a, 1)
                o[here, g] = torch.softmax(a, 1) @ v
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s) if case["op"] == "attend" else _exact_rotary(s)
