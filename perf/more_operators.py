"""Measured cases of the operators on a cache that holds K and V in 8 bits, with one scale per 16-token block and KV head.

  store   projected heads normed, rotated and written: every block that gets a token is quantised, its summary formed,
          and the blocks are read back as the attention of the same chunk takes them in
  read    the tokens of sequences read back
  all     exact attention of one query token per sequence over everything that the sequence holds
  sparse  the attention of a decode step: exact over the selected blocks, Mean compensation for the others

A block's K (or V) of one head is held as codes c and one fp32 scale; its values are c * scale.  With m the largest
magnitude among the block's tokens and M the type's largest value (int8: 127, e4m3: 448),

    scale = m / M,   c = nearest(x * (M / m))        (to even; all zero where m < 2^-100)

in fp32, each operation rounded once.  Where `own` is false, `run` uses elementary torch operations; where it is true,
it calls the framework.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 16
EPS = 1e-6
BASE = 1000000.0  # base of the rotation's frequencies
LEAST = 2.0 ** -100
MOST = {"int8": 127.0, "float8_e4m3fn": 448.0}


# ------------------------------------------------------------------ cases
def listed():
    i8, e4 = "int8", "float8_e4m3fn"
    return [
        # the token of a decode step for a batch in mid-flight: the single-token form, most tokens inside a block
        dict(name="store_token", op="store", batch=64, hkv=8, g=4, d=128, r=4, rot=128, paired=False, norm=True, kv=i8,
             tokens=1, start=1000, ragged=True, qtype="float32"),
        # a chunk of prefill for a ragged batch: odd starts and counts, a partial rotation of adjacent pairs, no norms
        dict(name="store_ragged", op="store", batch=16, hkv=8, g=8, d=128, r=128, rot=64, paired=True, norm=False, kv=e4,
             tokens=301, start=77, ragged=True, qtype="float32"),
        # one long prompt
        dict(name="store_long", op="store", batch=1, hkv=8, g=4, d=128, r=4, rot=128, paired=False, norm=True, kv=i8,
             tokens=32768, start=0, ragged=False, qtype="bfloat16"),
        # a short conversation of the smallest layer taken out of the cache
        dict(name="read_small", op="read", batch=2, hkv=2, d=64, kv=e4, tokens=1025, start=3, dtype="float32"),
        # a batch of contexts handed to an attention that reads bf16
        dict(name="read_batch", op="read", batch=16, hkv=8, d=128, kv=i8, tokens=16381, start=0, dtype="bfloat16"),
        # one user's chat on the smallest layer: latency is all that counts
        dict(name="all_small", op="all", batch=1, hkv=2, g=4, d=64, kv=i8, tokens=1025, dtype="float32"),
        # one 128K context of the headline layer
        dict(name="all_long", op="all", batch=1, hkv=8, g=4, d=128, kv=i8, tokens=131072, dtype="float32"),
        # a ragged batch of wide groups
        dict(name="all_wide", op="all", batch=16, hkv=8, g=8, d=128, kv=e4, tokens=65521, dtype="bfloat16"),
        # a full decode batch, contexts up to 64K
        dict(name="all_batch", op="all", batch=64, hkv=8, g=4, d=128, kv=i8, tokens=65536, dtype="bfloat16"),
        # the decode step's attention on the smallest layer
        dict(name="sparse_small", op="sparse", batch=1, hkv=2, g=4, d=64, r=4, kv=i8, tokens=1025, blocks=8),
        # the headline layer: 2048 of 131072 tokens selected
        dict(name="sparse_long", op="sparse", batch=1, hkv=8, g=4, d=128, r=4, kv=i8, tokens=131072, blocks=128),
        # a ragged batch
        dict(name="sparse_batch", op="sparse", batch=16, hkv=8, g=4, d=128, r=4, kv=e4, tokens=65535, blocks=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "store", "read", "all", "all", "sparse"])
    c = dict(op=op, hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128]), kv=rng.choice(sorted(MOST)))
    if op == "store":
        c.update(batch=_log(rng, 1, 64), g=rng.choice([1, 2, 4, 8]), r=rng.choice([1, 4, 16, 64]))
        c.update(rot=rng.choice([c["d"] // 2, c["d"]]), paired=rng.random() < 0.4, norm=rng.random() < 0.6)
        most = max(1, min(32768 // c["batch"], 32768 * 4 // (c["g"] * c["batch"])))
        return dict(c, tokens=_log(rng, 1, most), start=rng.choice([0, rng.randrange(1, 2000)]), ragged=rng.random() < 0.5,
                    qtype=rng.choice(["float32", "bfloat16"]))
    if op == "read":
        c.update(batch=_log(rng, 1, 64), start=rng.choice([0, rng.randrange(1, 100)]))
        return dict(c, tokens=_log(rng, 1, 16 * 16381 // max(16, c["batch"])), dtype=rng.choice(["float32", "bfloat16"]))
    if op == "all":
        c.update(batch=_log(rng, 1, 64), g=rng.choice([1, 2, 4, 8]), dtype=rng.choice(["float32", "bfloat16"]))
        return dict(c, tokens=_log(rng, 1, 131072 if c["batch"] <= 32 else 65536))
    c.update(batch=_log(rng, 1, 16), g=rng.choice([1, 2, 4, 8]), r=4)
    return dict(c, tokens=_log(rng, 1, 131072 if c["batch"] <= 4 else 65536), blocks=_log(rng, 3, 128))


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
    """Tokens that each sequence brings to a store, and the tokens that it holds before."""
    n, B = c["tokens"], c["batch"]
    if not c["ragged"]:
        return [n] * B, [c["start"]] * B
    starts = [c["start"] * (s * 13 % 64 + 1) // 64 for s in range(B)]
    return [n if s == 0 or n == 1 else (n * (s * 37 % 64)) // 64 for s in range(B)], starts


def _lens(c):
    """Tokens of each sequence: the first is the longest, one of a larger batch holds none."""
    return [c["tokens"] if s == 0 else 0 if s == 5 else (c["tokens"] * (s * 29 % 64 + 1)) // 65 for s in range(c["batch"])]


def _codes(kv):
    return getattr(torch, kv)


class _Tensors:
    """The cache's buffers where the framework is not in use."""

    def __init__(self, caps, hkv, d, r, kv):
        rows = hkv * sum(caps) // BLOCK
        self.k = torch.zeros((rows, BLOCK, d), dtype=_codes(kv), device=DEVICE)
        self.v = torch.zeros((rows, BLOCK, d), dtype=_codes(kv), device=DEVICE)
        self.kscale = torch.zeros((rows,), device=DEVICE)
        self.vscale = torch.zeros((rows,), device=DEVICE)
        self.kbar = torch.zeros((rows, d), device=DEVICE)
        self.vbar = torch.zeros((rows, d), device=DEVICE)
        self.dbar = torch.zeros((rows, r), device=DEVICE)
        self.seq_len = torch.zeros((1, len(caps)), dtype=torch.int32, device=DEVICE)


def _cache(c, caps):
    """The cache that a program keeps: a handle with its buffers, or the buffers alone."""
    if own:
        from block_sparse_kv_summary_gb300 import CompKVCache
        return CompKVCache(num_layers=1, batch=len(caps), num_kv_heads=c["hkv"], group_size=c.get("g", 1), head_dim=c["d"],
                           r=c.get("r", 4), budget_tokens=BLOCK * max(3, c.get("blocks", 8)), capacity_tokens=caps, device=DEVICE,
                           kv_dtype=_codes(c["kv"]))
    return _Tensors(caps, c["hkv"], c["d"], c.get("r", 4), c["kv"])


def _quantise(x, kv):
    """Codes and scales of blocks x [..., 16, d] (slots without a token are zero)."""
    m = x.abs().amax((-1, -2))
    most = torch.full_like(m, MOST[kv])
    held = m >= LEAST
    scale = torch.where(held, m / most, 0.0)
    y = x * torch.where(held, most / m, 0.0)[..., None, None]
    return (y.round() if kv == "int8" else y).to(_codes(kv)), scale


def _take(t, *at):
    """t[at] for codes of any type."""
    return t.view(torch.int8)[at].view(t.dtype)


def _values(codes, scale):
    return codes.float() * scale[..., None, None]


def _summaries(k, v, valid, r):
    """Mean key, mean value and grouped variance of blocks [..., 16, d], of the tokens that `valid` [..., 16] names."""
    m = valid[..., None].to(k.dtype)
    n = m.sum(-2).clamp(min=1)
    kbar = (k * m).sum(-2) / n
    vbar = (v * m).sum(-2) / n
    var = ((k - kbar[..., None, :]).square() * m).sum(-2) / n
    return kbar, vbar, var.unflatten(-1, (r, -1)).mean(-1)


def _table(positions, rot):
    """cos and sin of every position's angles, 32 bits, formed in 64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEVICE)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * BASE ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    return (_prepare_store if case["op"] == "store" else _prepare_held)(case, seed)


def _blocks(g, n, d):
    """K and V of n blocks: keys lie around a centre of their own, two of their channels are wide."""
    k = _randn(g, n, 1, d) + 0.3 * _randn(g, n, BLOCK, d)
    k[..., 5] *= 5
    k[..., d - 3] *= 5
    return k.bfloat16().float(), _randn(g, n, BLOCK, d).bfloat16().float()


def _fill(c, g, cache, summaries):
    """Every block of the cache, used or not."""
    for lo in range(0, cache.k.shape[0], 32768):
        hi = min(cache.k.shape[0], lo + 32768)
        k, v = _blocks(g, hi - lo, c["d"])
        for t, s, x in ((cache.k, cache.kscale, k), (cache.v, cache.vscale, v)):
            codes, s[lo:hi] = _quantise(x, c["kv"])
            t[lo:hi].copy_(codes)
        if summaries:
            valid = torch.ones(hi - lo, BLOCK, dtype=torch.bool, device=DEVICE)
            for t, x in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(k, v, valid, c["r"])):
                t[lo:hi] = x


def _prepare_store(c, seed):
    g = _gen(seed)
    B, H, G, d = c["batch"], c["hkv"], c["g"], c["d"]
    Hq = H * G
    counts, starts = _counts(c)
    cap = max(2048, _up(max(a + n for a, n in zip(starts, counts))))
    nb = cap // BLOCK
    cache = _cache(c, [cap] * B)
    _fill(c, g, cache, True)  # what the sequences hold already
    cache.seq_len.copy_(torch.tensor([starts], dtype=torch.int32))
    T = sum(counts)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(counts)).to(DEVICE)
    slot = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).to(DEVICE)
    centre = _randn(g, B, nb, H, d)
    k = centre[seq, slot // BLOCK] + 0.3 * _randn(g, T, H, d)
    pad = 64  # the projection's rows stand further apart than they are long
    qkv = torch.zeros((T, (Hq + 2 * H) * d + pad), device=DEVICE, dtype=torch.bfloat16)[:, :(Hq + 2 * H) * d]
    qkv.copy_(torch.cat([_randn(g, T, Hq, d), k, _randn(g, T, H, d)], 1).flatten(1))
    wq, wk = (1 + 0.1 * _randn(g, d) if c["norm"] else None for _ in range(2))
    # blocks that get a token: (sequence, block), the block of each token, and the tokens that stand in front of them
    at, blk, first, read0, reads = [], [], [], [], []
    for s in range(B):
        first.append(len(at))
        b0 = starts[s] // BLOCK
        b1 = (starts[s] + counts[s] - 1) // BLOCK + 1 if counts[s] else b0
        at += [s] * (b1 - b0)
        blk += list(range(b0, b1))
        read0.append(b0 * BLOCK)
        reads.append(starts[s] + counts[s] - b0 * BLOCK if counts[s] else 0)
    at, blk, first = (torch.tensor(x, device=DEVICE) for x in (at, blk, first))
    lo = torch.tensor(starts, device=DEVICE)
    end = lo + torch.tensor(counts, device=DEVICE)
    pos = blk[:, None] * BLOCK + torch.arange(BLOCK, device=DEVICE)
    old = pos < lo[at][:, None]
    held = [_values(_take(t.view(B, H, nb, BLOCK, d), at, slice(None), blk), s.view(B, H, nb)[at, :, blk]).bfloat16() * old[:, None, :, None]
            for t, s in ((cache.k, cache.kscale), (cache.v, cache.vscale))]
    return dict(case=c, cache=cache, qkv=qkv, table=_table(cap, c["rot"]), counts=counts, starts=starts, seq=seq, slot=slot,
                cap=cap, wq=wq, wk=wk, at=at, blk=blk, entry=first[seq] + slot // BLOCK - (lo // BLOCK)[seq],
                valid=pos < end[at][:, None], held=held, read0=read0, reads=reads,
                lens=torch.where(end > lo, end, lo).int())


def _prepare_held(c, seed):
    g = _gen(seed)
    H, d = c["hkv"], c["d"]
    lens = _lens(c) if c["op"] != "read" else [c["tokens"] + c["start"]] * c["batch"]
    caps = [max(BLOCK, _up(n)) for n in lens]
    cache = _cache(c, caps)
    _fill(c, g, cache, c["op"] == "sparse")
    cache.seq_len.copy_(torch.tensor([lens], dtype=torch.int32))
    state = dict(case=c, cache=cache, lens=lens, caps=caps)
    if c["op"] == "read":
        state.update(starts=[c["start"]] * c["batch"], counts=[c["tokens"] * (s * 29 % 64 + 1) // 64 if s else c["tokens"]
                                                               for s in range(c["batch"])])
        return state
    # logits of a standard deviation of 1.5: some keys weigh a hundred times others
    q = 1.2 * _randn(g, c["batch"], H * c["g"], d)
    state["q"] = q.to(getattr(torch, c.get("dtype", "float32")))
    if c["op"] == "sparse":
        K = max(3, c["blocks"])
        sel = torch.full((c["batch"], H, K), -1, dtype=torch.int32, device=DEVICE)
        for s, n in enumerate(lens):
            N = (n + BLOCK - 1) // BLOCK
            w = torch.rand(H, N, device=DEVICE, generator=g)
            if N:
                w[:, 0] = 2.0  # the sink and the two most recent blocks are always there
                w[:, -2:] = 3.0
            m = min(K, N)
            sel[s, :, :m] = w.topk(m, -1).indices.sort(-1).values.int()
            # the mean key, mean value and variance of a last block that is not full
            if n % BLOCK:
                valid = (torch.arange(BLOCK, device=DEVICE) < n % BLOCK).expand(H, BLOCK)
                rows = _rows(state, s)[:, N - 1]
                k, v = (_values(_take(t, rows), x[rows]) for t, x in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
                for t, x in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(k, v, valid, c["r"])):
                    t[rows] = x
        state["sel"] = sel
    return state


def _rows(state, s):
    """Rows of sequence s in the cache's buffers: [H, blocks of its capacity]."""
    H, caps = state["case"]["hkv"], state["caps"]
    n = caps[s] // BLOCK
    return H * sum(caps[:s]) // BLOCK + torch.arange(H * n, device=DEVICE).view(H, n)


def _tokens(state, s, t, scale, dtype=torch.float32):
    """Values of everything that sequence s has room for: [H, capacity, d]."""
    r = _rows(state, s)
    lo, hi = int(r[0, 0]), int(r[-1, -1]) + 1
    return (t[lo:hi].to(dtype) * scale[lo:hi, None, None].to(dtype)).view(r.shape[0], -1, t.shape[-1])


# ------------------------------------------------------------------ one pass
def run(state):
    return {"store": _run_store, "read": _run_read, "all": _run_all, "sparse": _run_sparse}[state["case"]["op"]](state)


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


def _run_store(state):
    c, cache = state["case"], state["cache"]
    qtype = getattr(torch, c["qtype"])
    if own:
        q = cache.prefill_qkv(0, state["qkv"], state["counts"], state["table"], starts=state["starts"], q_weight=state["wq"],
                              k_weight=state["wk"], eps=EPS, interleaved=c["paired"], q_dtype=qtype)
        k, v = cache.read(0, state["read0"], state["reads"])
    else:
        B, H, d, rot, nb = c["batch"], c["hkv"], c["d"], c["rot"], state["cap"] // BLOCK
        Hq = H * c["g"]
        x = state["qkv"].unflatten(-1, (Hq + 2 * H, d))
        cs = state["table"][state["slot"]][:, None]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        q = _rotate(_norm(x[:, :Hq].float(), state["wq"]), cos, sin, rot, c["paired"]).to(qtype)
        # keys in 64 bits: which way a value next to a border rounds decides the block's variance
        k = _rotate(_norm(x[:, Hq:Hq + H].double(), state["wk"]), cos.double(), sin.double(), rot, c["paired"]).to(torch.bfloat16)
        at, blk = state["at"], state["blk"]
        blocks, back = [], []
        for new, held, t, s in ((k, state["held"][0], cache.k, cache.kscale), (x[:, Hq + H:], state["held"][1], cache.v, cache.vscale)):
            y = held.clone()
            y[state["entry"], :, state["slot"] % BLOCK] = new
            blocks.append(y.float())
            codes, scale = _quantise(blocks[-1], c["kv"])
            t.view(torch.int8).view(B, H, nb, BLOCK, d)[at, :, blk] = codes.view(torch.int8)
            s.view(B, H, nb)[at, :, blk] = scale
            back.append(_values(codes, scale).to(torch.bfloat16).transpose(1, 2)[state["valid"]])
        k, v = back
        valid = state["valid"][:, None].expand(-1, H, -1)
        for t, y in zip((cache.kbar, cache.vbar, cache.dbar), _summaries(*blocks, valid, c["r"])):
            t.view(B, H, nb, -1)[at, :, blk] = y
        cache.seq_len[0] = state["lens"]
    return dict(q=q, k=k, v=v, kscale=cache.kscale, vscale=cache.vscale, kbar=cache.kbar, vbar=cache.vbar, dbar=cache.dbar,
                seq_len=cache.seq_len)


def _run_read(state):
    c, cache = state["case"], state["cache"]
    dtype = getattr(torch, c["dtype"])
    if own:
        k, v = cache.read(0, state["starts"], state["counts"], dtype=dtype)
    else:
        k, v = (torch.cat([_tokens(state, s, t, x)[:, a:a + n].transpose(0, 1)
                           for s, (a, n) in enumerate(zip(state["starts"], state["counts"]))]).to(dtype)
                for t, x in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
    return dict(k=k, v=v)


def _run_all(state):
    c, cache = state["case"], state["cache"]
    H, G, d = c["hkv"], c["g"], c["d"]
    if own:
        return cache.attend_all(0, state["q"])
    out = torch.zeros_like(state["q"])
    q = state["q"].float().view(-1, H, G, d) / math.sqrt(d)
    for s, n in enumerate(state["lens"]):
        if not n:
            continue
        z = q[s] @ _tokens(state, s, cache.k, cache.kscale)[:, :n].transpose(1, 2)
        w = torch.exp(z - z.amax(-1, keepdim=True))
        o = w @ _tokens(state, s, cache.v, cache.vscale)[:, :n] / w.sum(-1, keepdim=True)
        out[s] = o.view(H * G, d).to(out.dtype)
    return out


def _run_sparse(state):
    c, cache = state["case"], state["cache"]
    H, G, d = c["hkv"], c["g"], c["d"]
    if own:
        return cache.attend(0, state["q"], state["sel"])
    out = torch.zeros_like(state["q"])
    q = state["q"].view(-1, H, G, d) / math.sqrt(d)
    j = torch.arange(BLOCK, device=DEVICE)
    for s, n in enumerate(state["lens"]):
        if not n:
            continue
        N = (n + BLOCK - 1) // BLOCK
        sel = state["sel"][s, :, :min(N, state["sel"].shape[2])].long()
        rows = _rows(state, s)
        picked = rows.gather(1, sel)
        k = _values(_take(cache.k, picked), cache.kscale[picked]).flatten(1, 2)
        v = _values(_take(cache.v, picked), cache.vscale[picked]).flatten(1, 2)
        z = q[s] @ k.transpose(1, 2)
        z = z.masked_fill((sel[..., None] * BLOCK + j >= n).flatten(1)[:, None], -math.inf)
        # every other block stands for its tokens with its mean key and mean value
        zb = q[s] @ cache.kbar[rows[:, :N]].transpose(1, 2)
        count = torch.full((N,), float(BLOCK), device=DEVICE)
        count[-1] = n - (N - 1) * BLOCK
        taken = torch.zeros(H, N, dtype=torch.bool, device=DEVICE).scatter(1, sel, True)
        zb = zb.masked_fill(taken[:, None], -math.inf)
        m = torch.maximum(z.amax(-1, keepdim=True), zb.amax(-1, keepdim=True))
        w, wb = torch.exp(z - m), torch.exp(zb - m) * count
        o = (w @ v + wb @ cache.vbar[rows[:, :N]]) / (w.sum(-1, keepdim=True) + wb.sum(-1, keepdim=True))
        out[s] = o.view(H * G, d)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    H, d = c["hkv"], c["d"]
    if c["op"] == "store":
        counts, starts = _counts(c)
        Hq, T = H * c["g"], sum(counts)
        b = T * ((Hq + 2 * H) * d * 2 + Hq * d * (4 if c["qtype"] == "float32" else 2) + c["rot"] * 4)
        for n, a in zip(counts, starts):
            if n:
                blocks = (a + n - 1) // BLOCK - a // BLOCK + 1
                # codes and the values read back; summaries and scales; the tokens that stood in the first block
                b += (a % BLOCK + n) * 2 * H * d * 3 + blocks * H * (2 * d + c["r"] + 2) * 4 + (a % BLOCK) * 2 * H * d
        return {"bytes": b, "flops": T * (Hq + H) * d * 8}
    if c["op"] == "read":
        T = sum(c["tokens"] * (s * 29 % 64 + 1) // 64 if s else c["tokens"] for s in range(c["batch"]))
        return {"bytes": T * 2 * H * d * (1 + (4 if c["dtype"] == "float32" else 2)) + T // BLOCK * H * 8, "flops": T * 2 * H * d}
    G, B = c["g"], c["batch"]
    lens = _lens(c)
    blocks = [(n + BLOCK - 1) // BLOCK for n in lens]
    if c["op"] == "all":
        qb = 4 if c["dtype"] == "float32" else 2
        return {"bytes": H * (sum(lens) * d * 2 + sum(blocks) * 8 + 2 * B * G * d * qb), "flops": 4 * d * G * H * sum(lens)}
    took = [min(n, c["blocks"]) for n in blocks]
    rest = [n if n > t else 0 for n, t in zip(blocks, took)]  # the means of all blocks, unless every block is selected
    return {"bytes": H * (sum(took) * (BLOCK * d * 2 + 12) + sum(rest) * d * 8 + 2 * B * G * d * 4),
            "flops": 4 * d * G * H * (sum(took) * BLOCK + sum(rest))}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "all": _exact_attend, "sparse": _exact_attend}[case["op"]](state)


def _nearest(x, kv):
    """Codes of x in 64 bits, halfway cases to even."""
    if kv == "int8":
        return x.round()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)  # e4m3: 3 bits behind the leading one
    return (x / step).round() * step


def _exact_store(state):
    c, cache = state["case"], state["cache"]
    B, H, d, rot, r, nb = c["batch"], c["hkv"], c["d"], c["rot"], c["r"], state["cap"] // BLOCK
    Hq, half = H * c["g"], c["rot"] // 2
    x = state["qkv"].double().reshape(-1, Hq + 2 * H, d)
    row = state["table"][state["slot"]].double()
    z = torch.complex(row[:, :half], row[:, half:])[:, None]

    def turn(y, w):
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        first = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) if c["paired"] else torch.complex(y[..., :half], y[..., half:rot])
        first = first * z
        parts = torch.view_as_real(first).reshape(*y.shape[:-1], rot) if c["paired"] else torch.cat([first.real, first.imag], -1)
        return torch.cat([parts, y[..., rot:]], -1)

    out = dict(q=turn(x[:, :Hq], state["wq"]))
    new = dict(k=turn(x[:, Hq:Hq + H], state["wk"]), v=x[:, Hq + H:])
    for name in ("k", "v"):
        bar, scale, var = (getattr(cache, n).double().view(B, H, nb, -1) for n in (name + "bar", name + "scale", "dbar"))
        back, at = [], 0
        for s, (n, a) in enumerate(zip(state["counts"], state["starts"])):
            if not n:
                continue
            b0, b1 = a // BLOCK, (a + n - 1) // BLOCK + 1
            # the tokens as they come to be stored: bf16, those that stood there before at their 8-bit values
            y = torch.zeros(H, (b1 - b0) * BLOCK, d, dtype=torch.float64, device=DEVICE)
            lo = a - b0 * BLOCK
            if lo:
                codes = _take(getattr(cache, name).view(B, H, nb, BLOCK, d), s, slice(None), b0, slice(0, lo)).double()
                y[:, :lo] = (codes * scale[s, :, b0, :, None]).bfloat16().double()
            y[:, lo:lo + n] = new[name][at:at + n].transpose(0, 1).to(torch.bfloat16).double()
            at += n
            y = y.view(H, b1 - b0, BLOCK, d)
            m = y.abs().flatten(2).amax(-1)
            held = m >= LEAST
            scale[s, :, b0:b1, 0] = torch.where(held, m / MOST[c["kv"]], 0.0)
            codes = _nearest(y * torch.where(held, MOST[c["kv"]] / m, 0.0)[..., None, None], c["kv"])
            back.append((codes * scale[s, :, b0:b1, :, None]).flatten(1, 2)[:, :lo + n].transpose(0, 1))
            for b in range(b1 - b0 - 1, b1 - b0) if b1 - b0 == 1 else (slice(0, b1 - b0 - 1), b1 - b0 - 1):
                last = not isinstance(b, slice)
                t = y[:, b:b + 1, :lo + n - b * BLOCK] if last else y[:, b]
                where = slice(b0 + b, b0 + b + 1) if last else slice(b0, b1 - 1)
                bar[s, :, where] = t.mean(2)
                if name == "k":
                    var[s, :, where] = t.var(2, unbiased=False).unflatten(-1, (r, d // r)).mean(-1)
        out[name] = torch.cat(back) if back else torch.zeros(0, H, d, dtype=torch.float64, device=DEVICE)
        out[name + "scale"], out[name + "bar"] = scale.flatten(), bar.view(-1, d)
        if name == "k":
            out["dbar"] = var.view(-1, r)
    order = ("q", "k", "v", "kscale", "vscale", "kbar", "vbar", "dbar")
    return dict({n: out[n] for n in order}, seq_len=None)


def _exact_read(state):
    cache, out = state["cache"], []
    for t, x in ((cache.k, cache.kscale), (cache.v, cache.vscale)):
        parts = []
        for s, (a, n) in enumerate(zip(state["starts"], state["counts"])):
            slots = torch.arange(a, a + n, device=DEVICE)
            rows = _rows(state, s)[:, slots // BLOCK]
            parts.append((_take(t, rows, slots % BLOCK).double() * x[rows].double()[..., None]).transpose(0, 1))
        out.append(torch.cat(parts))
    return dict(k=out[0], v=out[1])


def _exact_attend(state):
    """Attention over tokens; in the sparse form the tokens of a block that is not selected have its mean key and value."""
    c, cache = state["case"], state["cache"]
    H, G, d = c["hkv"], c["g"], c["d"]
    if d * G * H * sum(state["lens"]) > 2e10:
        return None
    q = state["q"].double().view(-1, H, G, d)
    out = torch.zeros(c["batch"], H, G, d, dtype=torch.float64, device=DEVICE)
    for s, n in enumerate(state["lens"]):
        if not n:
            continue
        N = (n + BLOCK - 1) // BLOCK
        rows = _rows(state, s)
        for h in range(H):
            r = rows[h, :N]
            k, v = (_take(t, r).double() * x[r].double()[:, None, None] for t, x in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
            if c["op"] == "sparse":
                sel = state["sel"][s, h].long()
                rest = torch.ones(N, dtype=torch.bool, device=DEVICE)
                rest[sel[sel >= 0]] = False
                k[rest], v[rest] = cache.kbar[r[rest]].double()[:, None], cache.vbar[r[rest]].double()[:, None]
            w = torch.softmax(q[s, h] @ k.reshape(-1, d)[:n].T / d ** 0.5, -1)
            out[s, h] = w @ v.reshape(-1, d)[:n]
    return out.view(-1, H * G, d)
