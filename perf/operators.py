"""Measured cases of the operators that surround the CompKV decode step.

  rope_step     norms of the query and key heads and the position rotation for one token a sequence: the inputs of a
                decode step, from the fused projection's output
  rope_prefill  the same for many tokens, with the keys and values packed into the cache and their block summaries formed
  fork          a sequence's tokens and summaries copied to other sequences of the cache, over several layers
  compact       the listed blocks of a sequence moved to the front of another one, or of itself
  shared        exact attention of a batch whose sequences share a long prefix that the cache holds once

Where `own` is false, `run` uses elementary torch operations; where it is true, it calls the framework.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 16
EPS = 1e-6
BASE = 1000000.0  # base of the rotation's frequencies


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's chat on the smallest layer: latency is all that counts
        dict(name="step_small", op="rope_step", batch=1, hkv=2, g=4, d=64, r=4, rot=64, paired=False, norm=True, context=1025),
        # a full decode batch of ragged contexts on the headline layer
        dict(name="step_batch", op="rope_step", batch=64, hkv=8, g=4, d=128, r=4, rot=128, paired=False, norm=True, context=131072),
        # a chunk of prefill for a batch in mid-flight: odd starts and counts, a partial rotation of adjacent pairs, no norms
        dict(name="prefill_ragged", op="rope_prefill", batch=16, hkv=8, g=8, d=128, r=128, rot=64, paired=True, norm=False,
             tokens=301, start=77, ragged=True, qtype="float32"),
        # one long prompt
        dict(name="prefill_long", op="rope_prefill", batch=1, hkv=8, g=4, d=128, r=4, rot=128, paired=False, norm=True,
             tokens=32768, start=0, ragged=False, qtype="bfloat16"),
        # three more answers to a short prompt
        dict(name="fork_small", op="fork", layers=1, hkv=2, d=64, r=4, copies=3, tokens=1025),
        # a prompt sampled sixteen times, four layers at once
        dict(name="fork_fan", op="fork", layers=4, hkv=8, d=128, r=4, copies=15, tokens=8201),
        # one sequence cut down to the blocks that a selection kept, into a slot of its own
        dict(name="compact_small", op="compact", layers=1, batch=1, hkv=8, d=128, r=4, tokens=4099, kept=64, inplace=False),
        # a batch of branches forked whole and then cut down in place to 4096 tokens
        dict(name="compact_batch", op="compact", layers=2, batch=8, hkv=8, d=128, r=4, tokens=32764, kept=256, inplace=True),
        # a handful of short answers behind a short instruction, the smallest layer
        dict(name="shared_small", op="shared", batch=4, hkv=2, g=4, d=64, prefix=1000, tail=41, dtype="float32"),
        # a medium batch behind a 32K document, in the types of the decode step
        dict(name="shared_document", op="shared", batch=16, hkv=8, g=4, d=128, prefix=32768, tail=500, dtype="float32"),
        # a full batch behind a 128K context
        dict(name="shared_long", op="shared", batch=64, hkv=8, g=4, d=128, prefix=131072, tail=1024, dtype="bfloat16"),
        # a full batch of wide groups, tails as long as a conversation
        dict(name="shared_wide", op="shared", batch=64, hkv=8, g=8, d=128, prefix=16381, tail=2048, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_step", "rope_prefill", "fork", "compact", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op in ("rope_step", "rope_prefill"):
        c = dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, g=rng.choice([1, 2, 4, 8]), d=d, r=rng.choice([1, 4, 16, 64]),
                 rot=rng.choice([d // 2, d]), paired=rng.random() < 0.4, norm=rng.random() < 0.6)
        if op == "rope_step":
            return dict(c, context=_log(rng, 17, 131072))
        most = max(1, min(32768 // c["batch"], 32768 * 4 // (c["g"] * c["batch"])))
        return dict(c, tokens=_log(rng, 1, most), start=rng.choice([0, rng.randrange(1, 2000)]), ragged=rng.random() < 0.5,
                    qtype=rng.choice(["float32", "bfloat16"]))
    if op == "fork":
        copies = _log(rng, 1, 15)
        return dict(op=op, layers=rng.randrange(1, 5), hkv=hkv, d=d, r=rng.choice([1, 4, 16, 64]), copies=copies,
                    tokens=_log(rng, 1, min(65536, 8201 * 15 // copies)))
    if op == "compact":
        batch = _log(rng, 1, 8)
        tokens = _log(rng, 40, 32764)
        blocks = (tokens + BLOCK - 1) // BLOCK
        return dict(op=op, layers=rng.randrange(1, 3), batch=batch, hkv=hkv, d=d, r=rng.choice([1, 4, 16, 64]), tokens=tokens,
                    kept=_log(rng, 1, blocks), inplace=rng.random() < 0.5)
    return dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, g=rng.choice([1, 2, 4, 8]), d=d, prefix=_log(rng, 1, 65536),
                tail=_log(rng, 1, 1024), dtype=rng.choice(["float32", "bfloat16"]))


# ------------------------------------------------------------------ sizes
def _up(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEVICE, generator=g)


def _counts(c):
    """Tokens that each sequence brings to a prefill, and the tokens that it holds before."""
    n, B = c["tokens"], c["batch"]
    if not c["ragged"]:
        return [n] * B, [c["start"]] * B
    return [n if s == 0 else (n * (s * 37 % 64)) // 64 for s in range(B)], [(c["start"] * (s % 5 + 1)) // 5 for s in range(B)]


def _tails(c):
    """Own tokens of each sequence of a shared batch: the first is the longest, some have none."""
    return [c["tail"] if s == 0 else (c["tail"] * (s * 29 % 64)) // 63 for s in range(c["batch"])]


class _Tensors:
    """The cache's buffers where the framework is not in use."""

    def __init__(self, layers, caps, hkv, d, r):
        rows = layers * hkv * sum(caps) // BLOCK
        self.k = torch.zeros((rows, BLOCK, d), dtype=torch.bfloat16, device=DEVICE)
        self.v = torch.zeros((rows, BLOCK, d), dtype=torch.bfloat16, device=DEVICE)
        self.kbar = torch.zeros((rows, d), device=DEVICE)
        self.vbar = torch.zeros((rows, d), device=DEVICE)
        self.dbar = torch.zeros((rows, r), device=DEVICE)
        self.seq_len = torch.zeros((layers, len(caps)), dtype=torch.int32, device=DEVICE)


def _cache(layers, caps, hkv, g, d, r):
    """The cache that a program keeps: a handle with its buffers, or the buffers alone."""
    if own:
        from block_sparse_kv_summary_gb300 import CompKVCache
        return CompKVCache(num_layers=layers, batch=len(caps), num_kv_heads=hkv, group_size=g, head_dim=d, r=r,
                           budget_tokens=128, capacity_tokens=caps, device=DEVICE)
    return _Tensors(layers, caps, hkv, d, r)


def _whole(t):
    return dict(k=t.k, v=t.v, kbar=t.kbar, vbar=t.vbar, dbar=t.dbar, seq_len=t.seq_len)


def _table(positions, rot):
    """cos and sin of every position's angles, 32 bits, formed in 64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEVICE)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * BASE ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _summaries(k, v, valid, r):
    """Mean key, mean value and grouped variance of blocks [..., 16, d], of the tokens that `valid` [..., 16] names."""
    m = valid[..., None].to(k.dtype)
    n = m.sum(-2).clamp(min=1)
    kbar = (k * m).sum(-2) / n
    vbar = (v * m).sum(-2) / n
    var = ((k - kbar[..., None, :]).square() * m).sum(-2) / n
    return kbar, vbar, var.unflatten(-1, (r, -1)).mean(-1)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    return {"rope_step": _prepare_rope, "rope_prefill": _prepare_rope, "fork": _prepare_pages, "compact": _prepare_pages,
            "shared": _prepare_shared}[case["op"]](case, seed)


def _prepare_rope(c, seed):
    g = _gen(seed)
    B, H, G, d = c["batch"], c["hkv"], c["g"], c["d"]
    Hq = H * G
    if c["op"] == "rope_step":
        counts, starts = [1] * B, [c["context"] - 1 if s == 0 else (c["context"] * (s * 41 % 64)) // 64 for s in range(B)]
        caps = [2048] * B  # the keys of earlier tokens take no part here; longer contexts stand in front of the cache
        positions = c["context"]
    else:
        counts, starts = _counts(c)
        caps = [max(2048, _up(max(a + n for a, n in zip(starts, counts))))] * B
        positions = caps[0]
    T = sum(counts)
    cache = _cache(1, caps, H, G, d, c["r"])
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(counts)).to(DEVICE)
    slot = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).to(DEVICE)
    # projections: keys of one block lie around a centre of their own, as in the decode step's inputs
    centre = _randn(g, B, (slot.max().item() // BLOCK) + 1, H, d)
    q = _randn(g, T, Hq, d)
    k = centre[seq, slot // BLOCK] + 0.3 * _randn(g, T, H, d)
    v = _randn(g, T, H, d)
    pad = 64  # the projection's rows stand further apart than they are long
    qkv = torch.zeros((T, (Hq + 2 * H) * d + pad), device=DEVICE, dtype=torch.bfloat16)[:, :(Hq + 2 * H) * d]
    qkv.copy_(torch.cat([q, k, v], 1).flatten(1))
    if c["op"] == "rope_prefill":
        # what the sequences hold already
        old = torch.arange(caps[0], device=DEVICE)[None] < torch.tensor(starts, device=DEVICE)[:, None]
        for t in (cache.k, cache.v):
            x = _randn(g, B, H, caps[0], d) * old[:, None, :, None]
            t.copy_(x.view(t.shape))
    lens = torch.tensor(starts, dtype=torch.int32)
    ahead = c["op"] == "rope_step" and c["context"] > caps[0]
    cache.seq_len.copy_((lens % 1000 if ahead else lens)[None])
    wq, wk = (1 + 0.1 * _randn(g, d) if c["norm"] else None for _ in range(2))
    return dict(case=c, cache=cache, qkv=qkv, table=_table(positions, c["rot"]), counts=counts, starts=starts, seq=seq, slot=slot,
                cap=caps[0], positions=lens.to(DEVICE) if ahead else None, wq=wq, wk=wk)


def _prepare_pages(c, seed):
    g = _gen(seed)
    L, H, d, r = c["layers"], c["hkv"], c["d"], c["r"]
    src = 1 if c["op"] == "fork" else c["batch"]
    dst = c["copies"] if c["op"] == "fork" else c["batch"]
    held = c["tokens"] + 5 if c["op"] == "fork" else c["tokens"]  # a fork leaves off a few tokens that were only tried
    cap = _up(held)
    cache = _cache(L, [cap] * (src + dst), H, 4, d, r)
    shape = (L, src + dst, H, cap // BLOCK, BLOCK)
    k, v = cache.k.view(*shape, d), cache.v.view(*shape, d)
    tok = torch.arange(cap, device=DEVICE).view(cap // BLOCK, BLOCK) < held
    for s in range(src):
        for l in range(L):
            centre = _randn(g, H, cap // BLOCK, 1, d)
            k[l, s] = (centre + 0.3 * _randn(g, H, cap // BLOCK, BLOCK, d)) * tok[..., None]
            v[l, s] = _randn(g, H, cap // BLOCK, BLOCK, d) * tok[..., None]
            for t, x in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(k[l, s].float(), v[l, s].float(), tok, r)):
                t.view(*shape[:4], -1)[l, s] = x
    cache.seq_len[:, :src] = held
    state = dict(case=c, cache=cache, shape=shape, src=list(range(src)), dst=list(range(src, src + dst)))
    if c["op"] == "compact":
        # the sink, the last block and others at random, ascending, another choice for each layer, sequence and head
        n, kept = cap // BLOCK, c["kept"]
        w = torch.rand(L, src, H, n, device=DEVICE, generator=g)
        w[..., 0] = 2.0
        w[..., -1] = 3.0
        state["keep"] = w.topk(kept, -1).indices.sort(-1).values.int().contiguous()
    return state


def _prepare_shared(c, seed):
    g = _gen(seed)
    B, H, G, d, P = c["batch"], c["hkv"], c["g"], c["d"], c["prefix"]
    tails = _tails(c)
    own_cap = _up(max(c["tail"], BLOCK))
    caps = [max(2048, _up(P + own_cap))] + [own_cap] * (B - 1)
    cache = _cache(1, caps, H, G, d, 4)
    for t in (cache.k, cache.v):
        for h in range(0, t.shape[0], 65536):
            n = min(65536, t.shape[0] - h)
            t[h:h + n].copy_(_randn(g, n, BLOCK, d))
    cache.seq_len.copy_(torch.tensor([[P + tails[0]] + tails[1:]], dtype=torch.int32))
    q = 1.5 * _randn(g, B, H * G, d)  # logits of a standard deviation of 1.5: some keys weigh a hundred times others
    return dict(case=c, cache=cache, q=q.to(getattr(torch, c["dtype"])), caps=caps, own_cap=own_cap, tails=tails)


# ------------------------------------------------------------------ one pass
def run(state):
    return {"rope_step": _run_step, "rope_prefill": _run_prefill, "fork": _run_fork, "compact": _run_compact,
            "shared": _run_shared}[state["case"]["op"]](state)


def _rotate(x, cos, sin, rot, paired):
    """Rotation of the first `rot` coordinates: pairs (2i, 2i+1), or (i, i + rot/2)."""
    y, rest = x[..., :rot], x[..., rot:]
    if paired:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(x.dtype)


def _plain_rope(state, pos, qtype):
    c = state["case"]
    H, d, rot = c["hkv"], c["d"], c["rot"]
    Hq = H * c["g"]
    x = state["qkv"].unflatten(-1, (Hq + 2 * H, d))
    cs = state["table"][pos][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _rotate(_norm(x[:, :Hq].float(), state["wq"]), cos, sin, rot, c["paired"]).to(qtype)
    # keys in 64 bits: which way a value next to a border rounds decides the block's variance
    k = _rotate(_norm(x[:, Hq:Hq + H].double(), state["wk"]), cos.double(), sin.double(), rot, c["paired"]).to(torch.bfloat16)
    return q, k, x[:, Hq + H:].clone()


def _run_step(state):
    c, cache = state["case"], state["cache"]
    if own:
        q, k, v = cache.rope(0, state["qkv"], state["table"], q_weight=state["wq"], k_weight=state["wk"], eps=EPS,
                             interleaved=c["paired"], positions=state["positions"])
    else:
        q, k, v = _plain_rope(state, (cache.seq_len[0] if state["positions"] is None else state["positions"]).long(), torch.float32)
    return dict(q=q, k=k, v=v)


def _run_prefill(state):
    c, cache = state["case"], state["cache"]
    qtype = getattr(torch, c["qtype"])
    if own:
        q = cache.prefill_qkv(0, state["qkv"], state["counts"], state["table"], starts=state["starts"], q_weight=state["wq"],
                              k_weight=state["wk"], eps=EPS, interleaved=c["paired"], q_dtype=qtype)
    else:
        B, H, d, r, nb = c["batch"], c["hkv"], c["d"], c["r"], state["cap"] // BLOCK
        q, k, v = _plain_rope(state, state["slot"], qtype)
        kc, vc = cache.k.view(B, H, -1, d), cache.v.view(B, H, -1, d)
        kc[state["seq"], :, state["slot"]] = k
        vc[state["seq"], :, state["slot"]] = v
        # the blocks that got a token, as (sequence, block)
        at, blk = torch.unique(torch.stack([state["seq"], state["slot"] // BLOCK]), dim=1)
        new = torch.zeros((B,), dtype=torch.long, device=DEVICE)  # tokens that each sequence holds now
        new = new.scatter_reduce(0, state["seq"], state["slot"] + 1, "amax")
        valid = (blk[:, None] * BLOCK + torch.arange(BLOCK, device=DEVICE) < new[at][:, None])[:, None].expand(-1, H, -1)
        kb = kc.view(B, H, nb, BLOCK, d)[at, :, blk].float()
        vb = vc.view(B, H, nb, BLOCK, d)[at, :, blk].float()
        for t, x in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(kb, vb, valid, r)):
            t.view(B, H, nb, -1)[at, :, blk] = x
        cache.seq_len[0] = torch.where(new > 0, new.int(), cache.seq_len[0])
    return dict(q=q, **_whole(cache))


def _run_fork(state):
    c, cache = state["case"], state["cache"]
    n, dst = c["tokens"], state["dst"]
    if own:
        cache.fork([0] * len(dst), dst, [n] * len(dst))
        return _whole(cache)
    L, S, H, nb, _ = state["shape"]
    for t in (cache.k, cache.v):
        x = t.view(L, S, H, nb * BLOCK, -1)
        x[:, 1:, :, :n] = x[:, :1, :, :n]
    full, part = n // BLOCK, n % BLOCK
    for t in (cache.kbar, cache.vbar, cache.dbar):
        x = t.view(L, S, H, nb, -1)
        x[:, 1:, :, :full] = x[:, :1, :, :full]
    if part:
        blocks = [t.view(L, S, H, nb, BLOCK, -1)[:, 0, :, full].float() for t in (cache.k, cache.v)]
        valid = (torch.arange(BLOCK, device=DEVICE) < part).expand(L, H, BLOCK)
        for t, x in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(*blocks, valid, c["r"])):
            t.view(L, S, H, nb, -1)[:, 1:, :, full] = x[:, None]
    cache.seq_len[:, 1:] = n
    return _whole(cache)


def _run_compact(state):
    c, cache = state["case"], state["cache"]
    B, keep, kept = c["batch"], state["keep"], c["kept"]
    if own:
        if c["inplace"]:
            cache.fork(state["src"], state["dst"])
            cache.compact(keep, state["dst"])
        else:
            cache.compact(keep, state["src"], state["dst"])
        return _whole(cache)
    L, S, H, nb, _ = state["shape"]
    last = c["tokens"] - (nb - 1) * BLOCK
    i = torch.arange(L, device=DEVICE)[:, None, None, None], torch.arange(B, device=DEVICE)[:, None, None], torch.arange(H, device=DEVICE)[:, None]
    for t in (cache.k, cache.v, cache.kbar, cache.vbar, cache.dbar):
        x = t.view(L, S, H, nb, *t.shape[1:])
        tokens = t.dim() == 3
        if c["inplace"]:
            if tokens:
                y = t.view(L, S, H, nb * BLOCK, -1)
                y[:, B:, :, :c["tokens"]] = y[:, :B, :, :c["tokens"]]
            else:
                x[:, B:] = x[:, :B]
        moved = x[:, :B][i[0], i[1], i[2], keep.long()]
        if tokens:  # what stands behind the last token stays as it was
            y = t.view(L, S, H, nb * BLOCK, -1)
            m = (kept - 1) * BLOCK + last
            y[:, B:, :, :m] = moved.flatten(3, 4)[:, :, :, :m]
        else:
            x[:, B:, :, :kept] = moved
    cache.seq_len[:, B:] = (kept - 1) * BLOCK + last
    return _whole(cache)


def _split(state, t):
    """The prefix [H, P, d] and every sequence's own tokens [B, H, own_cap, d] of one of the cache's buffers."""
    c, caps, n = state["case"], state["caps"], state["own_cap"]
    H, P, d = c["hkv"], c["prefix"], c["d"]
    rows = H * caps[0] // BLOCK
    first = t[:rows].view(H, caps[0], d)
    rest = t[rows:].view(-1, H, n, d)
    return first[:, :P], torch.cat([first[None, :, P:P + n], rest], 0)


def _run_shared(state):
    c, cache = state["case"], state["cache"]
    B, H, G, d, P = c["batch"], c["hkv"], c["g"], c["d"], c["prefix"]
    if own:
        return cache.attend_shared(0, state["q"], [0] * B, [P] + [0] * (B - 1))
    kp, ko = _split(state, cache.k)
    vp, vo = _split(state, cache.v)
    lens = cache.seq_len[0].long().clone()
    lens[0] -= P
    q = state["q"].float().view(B, H, G, d) / math.sqrt(d)
    zp = q.transpose(0, 1).reshape(H, B * G, d) @ kp.float().transpose(1, 2)
    zo = q @ ko.float().transpose(2, 3)
    dead = torch.arange(state["own_cap"], device=DEVICE)[None] >= lens[:, None]
    zo = zo.masked_fill(dead[:, None, None], -math.inf)
    mp = zp.amax(-1).view(H, B, G).transpose(0, 1)
    m = torch.maximum(mp, zo.amax(-1))
    zp = torch.exp(zp - m.transpose(0, 1).reshape(H, B * G, 1))
    zo = torch.exp(zo - m[..., None])
    total = zp.sum(-1).view(H, B, G).transpose(0, 1) + zo.sum(-1)
    o = (zp @ vp.float()).view(H, B, G, d).transpose(0, 1) + zo @ vo.float()
    return (o / total[..., None]).reshape(B, H * G, d).to(state["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    H, d = c["hkv"], c["d"]
    if c["op"] in ("rope_step", "rope_prefill"):
        Hq = H * c["g"]
        T = c["batch"] if c["op"] == "rope_step" else sum(_counts(c)[0])
        qb = 4 if c["op"] == "rope_step" or c["qtype"] == "float32" else 2
        b = T * ((Hq + 2 * H) * d * 2 + Hq * d * qb + 2 * H * d * 2 + c["rot"] * 4)
        if c["op"] == "rope_prefill":
            blocks = sum((a + n - 1) // BLOCK - a // BLOCK + 1 for n, a in zip(*_counts(c)) if n)
            b += blocks * H * (2 * d + c["r"]) * 4
        return {"bytes": b, "flops": T * (Hq + H) * d * 8}
    if c["op"] == "fork":
        n = (c["tokens"] + BLOCK - 1) // BLOCK
        one = c["layers"] * H * (c["tokens"] * d * 4 + n * (2 * d + c["r"]) * 4)
        return {"bytes": one * (1 + c["copies"]), "flops": 0}
    if c["op"] == "compact":
        def size(tokens, blocks):
            return c["layers"] * c["batch"] * H * (tokens * d * 4 + blocks * (2 * d + c["r"]) * 4)
        nb = (c["tokens"] + BLOCK - 1) // BLOCK
        b = 2 * size((c["kept"] - 1) * BLOCK + c["tokens"] - (nb - 1) * BLOCK, c["kept"])
        return {"bytes": b + (2 * size(c["tokens"], nb) if c["inplace"] else 0), "flops": 0}
    tails, G, B, P = _tails(c), c["g"], c["batch"], c["prefix"]
    keys = H * (P + sum(tails))
    return {"bytes": keys * d * 4 + 2 * B * H * G * d * (4 if c["dtype"] == "float32" else 2),
            "flops": 4 * d * G * H * (B * P + sum(tails))}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "shared":
        return _exact_shared(state)
    if op in ("rope_step", "rope_prefill"):
        return _exact_rope(state)
    # pages hold copies: what they hold comes from the rows that prepare() filled
    return None if op == "compact" else _exact_fork(state)


def _exact_rope(state):
    c, cache = state["case"], state["cache"]
    H, d, rot, r = c["hkv"], c["d"], c["rot"], c["r"]
    Hq = H * c["g"]
    x = state["qkv"].double().reshape(-1, Hq + 2 * H, d)
    pos = state["slot"]
    half = rot // 2
    z = torch.complex(state["table"][pos, :half].double(), state["table"][pos, half:].double())[:, None]

    def turn(y, w):
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        first = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) if c["paired"] else torch.complex(y[..., :half], y[..., half:rot])
        first = first * z
        parts = torch.view_as_real(first).reshape(*y.shape[:-1], rot) if c["paired"] else torch.cat([first.real, first.imag], -1)
        return torch.cat([parts, y[..., rot:]], -1)

    q, k, v = turn(x[:, :Hq], state["wq"]), turn(x[:, Hq:Hq + H], state["wk"]), x[:, Hq + H:]
    if c["op"] == "rope_step":
        return dict(q=q, k=k, v=v)
    B, cap = c["batch"], state["cap"]
    kc, vc = cache.k.view(B, H, cap, d).double(), cache.v.view(B, H, cap, d).double()
    kbar, vbar = torch.zeros(B, H, cap // BLOCK, d, dtype=torch.float64, device=DEVICE), torch.zeros(B, H, cap // BLOCK, d, dtype=torch.float64, device=DEVICE)
    dbar = torch.zeros(B, H, cap // BLOCK, r, dtype=torch.float64, device=DEVICE)
    at = 0
    for s, (n, a) in enumerate(zip(state["counts"], state["starts"])):
        if not n:
            continue
        kc[s, :, a:a + n] = k[at:at + n].transpose(0, 1)
        vc[s, :, a:a + n] = v[at:at + n].transpose(0, 1)
        at += n
        b0, b1, e = a // BLOCK, (a + n - 1) // BLOCK + 1, a + n
        stored = [t[s, :, b0 * BLOCK:e].to(torch.bfloat16).double() for t in (kc, vc)]  # the summaries are those of the stored tokens
        full = (e - b0 * BLOCK) // BLOCK
        for lo, hi in ((0, full), (full, b1 - b0)):
            if hi > lo:
                kk, vv = (t[:, lo * BLOCK:hi * BLOCK].unflatten(1, (hi - lo, -1)) for t in stored)
                kbar[s, :, b0 + lo:b0 + hi] = kk.mean(2)
                vbar[s, :, b0 + lo:b0 + hi] = vv.mean(2)
                dbar[s, :, b0 + lo:b0 + hi] = kk.var(2, unbiased=False).unflatten(-1, (r, d // r)).mean(-1)
    return dict(q=q, k=kc.view(cache.k.shape), v=vc.view(cache.v.shape), kbar=kbar.view(cache.kbar.shape),
                vbar=vbar.view(cache.vbar.shape), dbar=dbar.view(cache.dbar.shape), seq_len=None)


def _exact_fork(state):
    """The means and variances of the copies, from the tokens in 64 bits; the tokens are copies."""
    c, cache = state["case"], state["cache"]
    n, r, d = c["tokens"], c["r"], c["d"]
    L, S, H, nb, _ = state["shape"]
    out = {}
    full = n // BLOCK
    for name in ("kbar", "vbar", "dbar"):
        x = getattr(cache, name).double().view(L, S, H, nb, -1)
        t = (cache.v if name == "vbar" else cache.k).view(L, S, H, nb * BLOCK, d)[:, 0, :, :n].double()
        for lo, hi in ((0, full), (full, (n + BLOCK - 1) // BLOCK)):
            if hi > lo:
                y = t[:, :, lo * BLOCK:hi * BLOCK].unflatten(2, (hi - lo, -1))
                y = y.var(3, unbiased=False).unflatten(-1, (r, d // r)).mean(-1) if name == "dbar" else y.mean(3)
                x[:, 1:, :, lo:hi] = y[:, None]
        out[name] = x.view(getattr(cache, name).shape)
    return dict(k=None, v=None, seq_len=None, **out)


def _exact_shared(state):
    c, cache = state["case"], state["cache"]
    B, H, G, d = c["batch"], c["hkv"], c["g"], c["d"]
    if 4 * d * G * H * B * c["prefix"] > 3e11:
        return None
    kp, ko = _split(state, cache.k)
    vp, vo = _split(state, cache.v)
    q = state["q"].double().view(B, H, G, d)
    out = torch.empty(B, H, G, d, dtype=torch.float64, device=DEVICE)
    for h in range(H):
        z = torch.einsum("bgd,pd->bgp", q[:, h], kp[h].double()) / d ** 0.5
        for s, n in enumerate(state["tails"]):
            w = torch.softmax(torch.cat([z[s], q[s, h] @ ko[s, h, :n].double().T / d ** 0.5], -1), -1)
            out[s, h] = w[:, :c["prefix"]] @ vp[h].double() + w[:, c["prefix"]:] @ vo[s, h, :n].double()
    return out.view(B, H * G, d)
