"""The calls around the decode step against plain 64-bit restatements.

Norms with rotation (one token per sequence, and many into the cache), copies
and cuts of sequences, compaction to listed blocks, attention over a shared
prefix; alone at the sizes where they can go wrong, refused where they must
be, on streams and in graphs, and together as a server would use them.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 16
F32 = 2.0 ** -24   # largest relative error of one fp32 rounding
BF16 = 2.0 ** -8   # and of one bf16 rounding


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_sparse_kv_summary_gb300 as P
    P.build()
    P.lib()


def make_cache(caps, *, layers=1, hkv=2, g=4, d=64, r=4, budget=128, fill=None, kv_memory="device"):
    from block_sparse_kv_summary_gb300 import CompKVCache
    c = CompKVCache(num_layers=layers, batch=len(caps), num_kv_heads=hkv, group_size=g, head_dim=d, r=r,
                    budget_tokens=budget, capacity_tokens=list(caps), kv_memory=kv_memory)
    if fill is not None:
        for t in (c.k, c.v, c.kbar, c.vbar, c.dbar):
            t.fill_(fill)
    return c


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def table(positions, rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


# ------------------------------------------------------------------ norms and rotation
def rope64(x, w, tab, pos, rot, interleaved, eps):
    """(result, sum of the magnitudes that each coordinate adds up) in 64 bits; x [T, H, d]."""
    x = x.double()
    if w is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    cs = tab[pos].double()[:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, mag = x.clone(), x.abs()
    for dst, u, v, s in ((0, a, b, -1.0), (1, b, a, 1.0)):
        sl = (..., slice(dst, rot, 2)) if interleaved else (..., slice(dst * rot // 2, (dst + 1) * rot // 2))
        y[sl] = u * cos + s * v * sin
        mag[sl] = (u * cos).abs() + (v * sin).abs()
    return y, mag


def check_q(got, want, mag):
    # fp32: mean of squares (<= 13 roundings, halved by the root), the root (2 ulp), three products, the sum, and bf16 where asked
    tol = 16 * F32 * mag + (BF16 * want.abs() if got.dtype == torch.bfloat16 else 0)
    bad = (got.double() - want).abs() - tol
    assert bad.max().item() <= 0, bad.max().item()


def check_k(got, want):
    # rounded once from some 40 bits: no further from the value than the nearest bf16 is, up to 2^-36 of it
    near = want.float().bfloat16().double()
    assert ((got.double() - want).abs() <= (near - want).abs() + 2.0 ** -36 * want.abs()).all()


def split_heads(qkv, hkv, g, d):
    x = qkv.unflatten(-1, ((g + 2) * hkv, d))
    return x[:, :g * hkv], x[:, g * hkv:(g + 1) * hkv], x[:, (g + 1) * hkv:]


ROPES = [
    # hkv, g, d, rot, interleaved, norm, dtype, q type
    (2, 4, 64, 64, False, True, torch.bfloat16, torch.float32),
    (8, 4, 128, 128, False, True, torch.bfloat16, torch.bfloat16),
    (1, 1, 64, 16, True, False, torch.float32, torch.float32),
    (3, 8, 128, 48, False, True, torch.float32, torch.bfloat16),
    (4, 2, 128, 128, True, True, torch.bfloat16, torch.float32),
    (8, 8, 128, 64, False, False, torch.bfloat16, torch.float32),
]


@pytest.mark.parametrize("case", ROPES)
@pytest.mark.parametrize("batch", [1, 5, 64])
def test_rope_one_token(case, batch):
    hkv, g, d, rot, inter, norm, dt, qt = case
    c = make_cache([2048] * batch, hkv=hkv, g=g, d=d)
    width = (g + 2) * hkv * d
    qkv = randn(batch, batch, width + 24).to(dt)[:, :width]
    wq, wk = (1 + 0.2 * randn(2, d), 1 + 0.2 * randn(3, d)) if norm else (None, None)
    tab = table(2048, rot)
    lens = torch.randint(0, 2048, (batch,), generator=torch.Generator().manual_seed(7)).int().cuda()
    c.seq_len[0] = lens
    for positions in (None, torch.flip(lens, [0]).contiguous()):
        q, k, v = c.rope(0, qkv, tab, q_weight=wq, k_weight=wk, eps=1e-5, positions=positions, interleaved=inter, q_dtype=qt)
        pos = (lens if positions is None else positions).long()
        xq, xk, xv = split_heads(qkv, hkv, g, d)
        check_q(q, *rope64(xq, wq, tab, pos, rot, inter, 1e-5))
        check_k(k, rope64(xk, wk, tab, pos, rot, inter, 1e-5)[0])
        assert torch.equal(v, xv.bfloat16())
    assert c.device_status() == 0 and torch.equal(c.seq_len[0], lens)


def test_rope_small_and_zero_heads():
    # zeros stay zeros under a norm, and tiny heads are scaled by 1 / sqrt(eps)
    c = make_cache([64], hkv=1, g=1)
    qkv = torch.zeros(1, 3 * 64, device="cuda")
    q, k, v = c.rope(0, qkv, table(4, 64), q_weight=torch.ones(64, device="cuda"), k_weight=torch.ones(64, device="cuda"))
    assert not q.any() and not k.any() and not v.any()
    qkv = 1e-6 * randn(0, 1, 3 * 64)
    w = torch.ones(64, device="cuda")
    q, k, v = c.rope(0, qkv, table(4, 64), q_weight=w, k_weight=w)
    xq, xk, xv = split_heads(qkv, 1, 1, 64)
    pos = torch.zeros(1, dtype=torch.long, device="cuda")
    check_q(q, *rope64(xq, w, table(4, 64), pos, 64, False, 1e-6))
    check_k(k, rope64(xk, w, table(4, 64), pos, 64, False, 1e-6)[0])


def summaries64(k, v, r):
    """Of the tokens [n, d] of one block."""
    k, v = k.double(), v.double()
    return k.mean(0), v.mean(0), k.var(0, unbiased=False).view(r, -1).mean(-1)


def check_summaries(c, layer, s, h, blocks, length):
    kv, vv = c.token_view(layer, s, h)
    kb, db, vb = c.summary_view(layer, s, h)
    for b in blocks:
        k, v = (t[b * BLOCK:min(length, (b + 1) * BLOCK)].cuda() for t in (kv, vv))
        ek, ev, ed = summaries64(k, v, c.r)
        # at most 17 roundings of sums and one quotient
        assert ((kb[b].double() - ek).abs() <= 18 * F32 * k.double().abs().mean(0)).all()
        assert ((vb[b].double() - ev).abs() <= 18 * F32 * v.double().abs().mean(0)).all()
        # deviations are off by the mean's error, 18 F32 mean|k|; squares, 17 + 7 sums and quotients on top
        m = k.double().abs().mean(0)
        dev = (k.double() - ek).abs()
        tol = (2 * dev * (18 * F32 * m + F32 * dev) + (18 * F32 * m) ** 2).mean(0) + 28 * F32 * dev.square().mean(0)
        assert ((db[b].double() - ed).abs() <= tol.view(c.r, -1).mean(-1) + 1e-30).all()


@pytest.mark.parametrize("case", ROPES)
@pytest.mark.parametrize("plan", [
    ([1], [0]), ([16], [0]), ([15], [16]), ([17], [5]), ([1], [31]),
    ([0, 37, 0, 5, 200, 0], [0, 3, 9, 16, 47, 1]),
])
@pytest.mark.parametrize("r", [1, 16, 64])
def test_prefill_many_tokens(case, plan, r):
    hkv, g, d, rot, inter, norm, dt, qt = case
    counts, starts = plan
    B, T = len(counts), sum(counts)
    c = make_cache([256 + 16 * s for s in range(B)], hkv=hkv, g=g, d=d, r=r)
    for t, seed in ((c.k, 1), (c.v, 2)):
        t.copy_(randn(seed, *t.shape))
    before = [t.clone() for t in (c.k, c.v, c.kbar, c.vbar, c.dbar)]
    c.seq_len[0] = torch.tensor([77] * B)
    width = (g + 2) * hkv * d
    qkv = randn(B, T, width).to(dt)
    wq, wk = (1 + 0.2 * randn(2, d), 1 + 0.2 * randn(3, d)) if norm else (None, None)
    tab = table(512, rot)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).cuda()
    positions = (511 - pos).int() if r == 16 else None
    q = c.prefill_qkv(0, qkv, counts, tab, starts=starts, q_weight=wq, k_weight=wk, eps=1e-5, positions=positions,
                      interleaved=inter, q_dtype=qt)
    assert c.device_status() == 0
    if positions is not None:
        pos = positions.long()
    xq, xk, xv = split_heads(qkv, hkv, g, d)
    check_q(q, *rope64(xq, wq, tab, pos, rot, inter, 1e-5))
    ek = rope64(xk, wk, tab, pos, rot, inter, 1e-5)[0]
    at = 0
    touched = [torch.zeros(t.shape[0] * (BLOCK if t.dim() == 3 else 1), dtype=torch.bool, device="cuda") for t in before]
    for s, (n, a) in enumerate(zip(counts, starts)):
        assert c.seq_len[0, s].item() == (a + n if n else 77)
        for h in range(hkv if n else 0):
            kv, vv = c.token_view(0, s, h)
            check_k(kv[a:a + n], ek[at:at + n, h])
            assert torch.equal(vv[a:a + n], xv[at:at + n, h].bfloat16())
            check_summaries(c, 0, s, h, {a // BLOCK, (a + n - 1) // BLOCK, (a + n // 2) // BLOCK}, a + n)
            r0, _ = c.rows(0, s, h)
            for t in touched[:2]:
                t[r0 * BLOCK + a:r0 * BLOCK + a + n] = True
            for t in touched[2:]:
                t[r0 + a // BLOCK:r0 + (a + n - 1) // BLOCK + 1] = True
        at += n
    for old, new, m in zip(before, (c.k, c.v, c.kbar, c.vbar, c.dbar), touched):  # nothing else changed
        o, x = (t.reshape(m.numel(), -1) for t in (old, new))
        assert torch.equal(o[~m], x[~m])


def test_prefill_into_host_memory():
    # K and V in page-locked memory: the same rows and summaries as in device memory
    a, b = (make_cache([64, 96], hkv=2, g=2, kv_memory=m) for m in ("device", "host"))
    tab, w = table(128, 64), 1 + 0.1 * randn(9, 64)
    for x in (a, b):
        for counts, starts, seed in (([9, 50], None, 1), ([30, 0], [9, 0], 2), ([0, 30], [0, 50], 3)):
            x.prefill_qkv(0, randn(seed, sum(counts), 6 * 64 + 128), counts, tab, starts=starts, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    for x, y in zip(state(a), state(b)):
        assert torch.equal(x, y.to(x.device))
    assert a.seq_len.tolist() == [[39, 80]]


def test_prefill_empty_and_positions_outside_the_table():
    c = make_cache([64, 64], hkv=1, g=1)
    q = c.prefill_qkv(0, torch.empty(0, 192, device="cuda"), [0, 0], table(64, 64))
    assert q.shape == (0, 1, 64) and c.device_status() == 0
    qkv = randn(0, 3, 192)
    tab = table(8, 64)
    q = c.prefill_qkv(0, qkv, [0, 3], tab, starts=[0, 6])
    assert c.device_status() == 1 and c.device_status() == 0
    want, mag = rope64(qkv[:, None, :64], None, tab, torch.tensor([6, 7, 7], device="cuda"), 64, False, 0)
    check_q(q, want, mag)
    pos = torch.tensor([-5, 100], dtype=torch.int32, device="cuda")
    q, _, _ = c.rope(0, qkv[:2], tab, positions=pos)
    assert c.device_status() == 1
    check_q(q, *rope64(qkv[:2, None, :64], None, tab, torch.tensor([0, 7], device="cuda"), 64, False, 0))


# ------------------------------------------------------------------ pages
def filled(caps, lens, layers=2, hkv=2, d=64, r=4, seed=0, **kw):
    c = make_cache(caps, layers=layers, hkv=hkv, d=d, r=r, **kw)
    c.k.copy_(randn(seed + 1, *c.k.shape))
    c.v.copy_(randn(seed + 2, *c.v.shape))
    for l in range(layers):
        c.prefill(l, lens)
    torch.cuda.synchronize()
    return c


def state(c):
    return [t.clone() for t in (c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len)]


def heads_of(c, t, l, s):
    """[Hkv, capacity in blocks, ...] view of a buffer's rows of one (layer, sequence)."""
    r0, cap = c.rows(l, s, 0)
    return t[r0:r0 + c.Hkv * cap].view(c.Hkv, cap, *t.shape[1:])


@pytest.mark.parametrize("d,r,hkv", [(64, 1, 1), (128, 4, 8), (128, 128, 3), (64, 64, 2)])
@pytest.mark.parametrize("kv_memory", ["device", "host"])
def test_fork(d, r, hkv, kv_memory):
    caps = [640, 1024, 640, 656, 48, 640, 640]
    held = [631, 1000, 20, 7, 48, 64, 0]
    src = [0, 1, 0, 0, 4, 6]
    dst = [2, 3, 5, 4, 4, 6]
    src[3], dst[3] = 1, 1     # a cut in place
    src[1], dst[1] = 0, 3
    lens = [-1, 333, 320, 17, 31, 0]
    c = filled(caps, held, hkv=hkv, d=d, r=r, kv_memory=kv_memory)
    old = state(c)
    c.fork(src, dst, lens, layers=(1, 2))
    torch.cuda.synchronize()
    assert c.device_status() == 0
    want = [t.clone() for t in old]
    for s, t, n in zip(src, dst, lens):
        n = held[s] if n < 0 else n
        want[5][1, t] = n
        for x, o in zip(want[:2], old[:2]):
            a, b = heads_of(c, o, 1, s), heads_of(c, x, 1, t)
            b.flatten(1, 2)[:, :n] = a.flatten(1, 2)[:, :n]
        whole = n // BLOCK + (n % BLOCK > 0 and n == held[s])
        for x, o in zip(want[2:5], old[2:5]):
            heads_of(c, x, 1, t)[:, :whole] = heads_of(c, o, 1, s)[:, :whole]
        if n % BLOCK and n < held[s]:  # the cut block's summary is new
            for h in range(hkv):
                check_summaries(c, 1, t, h, [n // BLOCK], n)
                for x, got in zip(want[2:5], (c.kbar, c.vbar, c.dbar)):
                    heads_of(c, x, 1, t)[h, n // BLOCK] = heads_of(c, got, 1, t)[h, n // BLOCK]
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), want):
        assert torch.equal(got, w)


def test_fork_all_layers_truncate_and_device_refusals():
    c = filled([64, 64, 32], [50, 3, 0], layers=3)
    old = state(c)
    c.fork([0], [2])  # 50 tokens do not fit 32
    assert c.device_status() == 3
    c.fork([1], [2], [4])  # sequence 1 holds 3
    assert c.device_status() == 1
    for a, b in zip(old, state(c)):
        assert torch.equal(a, b)
    c.fork([0], [1])
    c.truncate([0], [33])
    assert c.device_status() == 0
    assert c.seq_len.tolist() == [[33, 50, 0]] * 3
    for l in range(3):
        for h in range(2):
            check_summaries(c, l, 0, h, [0, 1, 2], 33)
            check_summaries(c, l, 1, h, [0, 3], 50)


def lists(c, layers, choice):
    """keep tensor from choice[l][pair][head] lists."""
    m = max(len(x) for a in choice for b in a for x in b)
    k = torch.full((layers, len(choice[0]), c.Hkv, max(m, 1) + 1), -1, dtype=torch.int32)
    for l, a in enumerate(choice):
        for i, b in enumerate(a):
            for h, x in enumerate(b):
                k[l, i, h, :len(x)] = torch.tensor(x, dtype=torch.int32)
    return k.cuda()


@pytest.mark.parametrize("d,r,hkv", [(64, 1, 1), (128, 4, 8), (128, 128, 3), (64, 64, 2)])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("kv_memory", ["device", "host"])
def test_compact(d, r, hkv, inplace, kv_memory):
    held = [1999, 640, 5, 700]
    caps = [2048, 640, 64, 1024] * 2
    c = filled(caps, held + [0] * 4, hkv=hkv, d=d, r=r, kv_memory=kv_memory)
    g = torch.Generator().manual_seed(3)

    def pick(n, blocks, last):
        x = sorted(torch.randperm(blocks - 1, generator=g)[:n - last].tolist())
        return x + [blocks - 1] * last
    choice = [[[pick(97, 125, 1) for _ in range(hkv)], [pick(33, 40, 0) for _ in range(hkv)], [[0]] * hkv, [[]] * hkv]
              for _ in range(2)]
    keep = lists(c, 2, choice)
    old = state(c)
    src = [0, 1, 2, 3]
    dst = src if inplace else [4, 5, 6, 7]
    c.compact(keep, src, None if inplace else dst)
    torch.cuda.synchronize()
    assert c.device_status() == 0
    new_len = [96 * 16 + 1999 - 124 * 16, 33 * 16, 5, 0]
    want = [t.clone() for t in old]
    for l in range(2):
        for i in range(4):
            want[5][l, dst[i]] = new_len[i]
            for h in range(hkv):
                for x, o in zip(want[:5], old[:5]):
                    idx = torch.tensor(choice[l][i][h], dtype=torch.long, device=o.device)
                    a, b = heads_of(c, o, l, src[i])[h], heads_of(c, x, l, dst[i])[h]
                    if x.dim() == 3:
                        b.flatten(0, 1)[:new_len[i]] = a[idx].flatten(0, 1)[:new_len[i]]
                    else:
                        b[:len(idx)] = a[idx]
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("bad", [[0, 2, 2], [3, 1], [0, 5], [0, -1, 2], [0, -3], [0, 4]])
def test_compact_refuses_bad_lists(bad):
    # 80 tokens: blocks 0..4; sequence 1's lists are sound and are carried out
    c = filled([96, 96], [73, 73], layers=1)
    ok = [[0, 2, 4, -1], [1, 2, 4, -1]]
    rows = [[0, 1, 3, -1][:4], (bad + [-1] * 4)[:4]]
    keep = torch.tensor([[rows, ok]], dtype=torch.int32, device="cuda")
    old = state(c)
    c.compact(keep)
    assert c.device_status() == 6
    assert c.seq_len.tolist() == [[73, 2 * 16 + 9]]
    for o, n in zip(old[:5], state(c)[:5]):
        assert torch.equal(heads_of(c, o, 0, 0), heads_of(c, n, 0, 0))


def test_compact_refuses_a_destination_that_is_too_small():
    c = filled([96, 32], [73, 5], layers=1)
    old = state(c)
    c.compact(torch.tensor([[[[0, 1, 2]] * 2]], dtype=torch.int32, device="cuda"), [0], [1])
    assert c.device_status() == 3
    for o, n in zip(old, state(c)):
        assert torch.equal(o, n)


# ------------------------------------------------------------------ shared prefix
def shared64(c, layer, q, prefix_seq, prefix_len, lens):
    """(out, sum p |v|) [B, Hq, d] in 64 bits; rows of sequences without a part are None."""
    B, Hkv, G, d = c.batch, c.Hkv, c.G, c.d
    out = torch.zeros(B, Hkv * G, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for s in range(B):
        p = prefix_seq[s]
        if p == -2:
            continue
        for h in range(Hkv):
            kv, vv = c.token_view(layer, s, h)
            n = prefix_len[p] if p >= 0 else 0
            ks, vs = [kv[(n if p == s else 0):lens[s]]], [vv[(n if p == s else 0):lens[s]]]
            if p >= 0:
                kp, vp = c.token_view(layer, p, h)
                ks.insert(0, kp[:n])
                vs.insert(0, vp[:n])
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            if k.shape[0] == 0:
                continue
            w = torch.softmax(q[s, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d), -1)
            out[s, h * G:(h + 1) * G] = w @ v
            mag[s, h * G:(h + 1) * G] = w @ v.abs()
    return out, mag


def check_shared(got, want, mag, take=None):
    # fp32: weights and sums of up to 2^13 keys, added 16 at a time: 2^9 roundings, 2^9 F32 = 3e-5 of sum p |v|;
    # bf16: weights rounded by BF16 each, and the result; logits of bf16 queries are exact up to fp32 sums
    tol = 3e-5 * (mag + want.abs())
    if got.dtype == torch.bfloat16:
        tol = tol + BF16 * (mag + want.abs())
    bad = (got.double() - want).abs() - tol
    if take is not None:
        bad = bad[take]
    assert torch.isfinite(got.float() if take is None else got[take].float()).all()
    assert bad.max().item() <= 0, bad.max().item()


def shared_cache(caps, lens, hkv, g, d, seed=0):
    """Tokens in [0, lens), NaN in every slot behind them."""
    c = make_cache(caps, hkv=hkv, g=g, d=d, fill=float("nan"))
    for s, n in enumerate(lens):
        for h in range(hkv):
            kv, vv = c.token_view(0, s, h)
            kv[:n] = randn(seed + 100 * s + h, n, d)
            vv[:n] = randn(seed + 7000 + 100 * s + h, n, d)
    c.seq_len[0] = torch.tensor(lens, dtype=torch.int32)
    return c


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hkv,g,d", [(2, 4, 64), (8, 4, 128), (1, 8, 128), (3, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("prefix", [0, 1, 16, 127, 128, 129, 1000])
def test_shared_lengths(dtype, hkv, g, d, prefix):
    tails = [3, 0, 1, 130, 16]
    lens = [prefix + tails[0]] + tails[1:]
    c = shared_cache([1024, 16, 16, 144, 32], lens, hkv, g, d)
    q = (2 * randn(5, 5, hkv * g, d)).to(dtype)
    plen = [prefix, 0, 0, 0, 0]
    got = c.attend_shared(0, q, [0] * 5, plen)
    assert c.device_status() == 0
    check_shared(got, *shared64(c, 0, q, [0] * 5, plen, lens))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,hkv,g,d", [(64, 2, 8, 128), (64, 1, 8, 64), (33, 2, 4, 128), (40, 8, 4, 128), (17, 1, 8, 128)])
def test_shared_many_rows(dtype, batch, hkv, g, d):
    lens = [2500] + [(s * 37) % 300 for s in range(1, batch)]
    c = shared_cache([2512] + [304] * (batch - 1), lens, hkv, g, d)
    q = (2 * randn(5, batch, hkv * g, d)).to(dtype)
    plen = [2345] + [0] * (batch - 1)
    got = c.attend_shared(0, q, [0] * batch, plen)
    assert c.device_status() == 0
    check_shared(got, *shared64(c, 0, q, [0] * batch, plen, lens))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hkv,g,d", [(8, 4, 128), (3, 8, 64), (32, 1, 128), (4, 2, 128)])
@pytest.mark.parametrize("prefix", [0, 333])
def test_shared_many_short_sequences(dtype, hkv, g, d, prefix):
    # more sequences x heads than multiprocessors, with few tokens of their own
    lens = [prefix] + [[0, 1, 15, 16, 31, 32, 33, 63, 64, 65, 130][s % 11] for s in range(1, 64)]
    c = shared_cache([max(16, (prefix + 15) // 16 * 16)] + [144] * 63, lens, hkv, g, d)
    q = (2 * randn(5, 64, hkv * g, d)).to(dtype)
    prefix_seq = [0] * 60 + [-1, -1, -2, -1]
    out = torch.full_like(q, 7.0)
    got = c.attend_shared(0, q, prefix_seq, [prefix] + [0] * 63, out=out)
    assert c.device_status() == 0
    take = torch.tensor([p != -2 for p in prefix_seq], device="cuda")
    check_shared(got, *shared64(c, 0, q, prefix_seq, [prefix] + [0] * 63, lens), take)
    assert (out[~take] == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_groups_and_sequences_without_a_part(dtype):
    # two prefixes, one held by a sequence without a part, one by a member of the other; sequences alone; one with nothing
    prefix_seq = [-2, 0, 0, 4, 0, 4, -1, -1, -2, 0]
    prefix_len = [300, 9, 9, 9, 77, 9, 9, 9, 9, 9]
    lens = [310, 20, 0, 5, 200, 128, 0, 650, 33, 129]
    c = shared_cache([320, 32, 16, 16, 208, 128, 16, 656, 48, 144], lens, 2, 4, 128)
    q = (2 * randn(5, 10, 8, 128)).to(dtype)
    out = torch.full((10, 8, 128), 7.0, dtype=dtype, device="cuda")
    got = c.attend_shared(0, q, prefix_seq, prefix_len, out=out)
    assert got is out and c.device_status() == 0
    take = torch.tensor([p != -2 for p in prefix_seq], device="cuda")
    check_shared(got, *shared64(c, 0, q, prefix_seq, prefix_len, lens), take)
    assert (out[~take] == 7).all()
    assert not out[6].any()  # nothing to attend to


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_extreme_logits(dtype):
    # logits that rise by hundreds along the keys, and equal ones: the running maximum changes in every tile
    c = shared_cache([1024, 528], [1000, 520], 1, 2, 64)
    q = torch.zeros(2, 2, 64, device="cuda")
    q[:, 0, 0] = 64.0
    q[:, 1, 1] = -64.0
    for s, n in ((0, 1000), (1, 520)):
        kv, _ = c.token_view(0, s, 0)
        kv[:n, 0] = torch.linspace(-60, 60, n, device="cuda")
        kv[:n, 1] = torch.linspace(-60, 60, n, device="cuda")
    q = q.to(dtype)
    got = c.attend_shared(0, q, [0, 0], [900, 0])
    check_shared(got, *shared64(c, 0, q, [0, 0], [900, 0], [1000, 520]))


def test_shared_nothing_at_all():
    c = shared_cache([64, 64], [0, 0], 1, 8, 128)
    q = randn(5, 2, 8, 128)
    out = torch.full_like(q, 3.0)
    assert not c.attend_shared(0, q, [0, 0], [0, 0], out=out).any()
    out.fill_(3.0)
    assert (c.attend_shared(0, q, [-2, -2], [0, 0], out=out) == 3).all() and c.device_status() == 0


def test_shared_prefix_longer_than_its_holder():
    c = shared_cache([64, 64], [20, 9], 1, 1, 64)
    q = randn(5, 2, 1, 64)
    got = c.attend_shared(0, q, [0, 0], [40, 0])
    assert c.device_status() == 1
    check_shared(got, *shared64(c, 0, q, [0, 0], [20, 0], [20, 9]))


# ------------------------------------------------------------------ refusals
def test_refusals():
    from block_sparse_kv_summary_gb300 import CompKVError
    c = make_cache([64, 64, 64], layers=2)
    width = 12 * 64
    qkv, tab = randn(0, 3, width), table(64, 64)

    def refused(match, fn, *a, **kw):
        with pytest.raises((CompKVError, ValueError), match=match):
            fn(*a, **kw)
    refused("layer", c.rope, 2, qkv, tab)
    refused("rot_dim", c.rope, 0, qkv, table(64, 80))
    refused("rot_dim", c.rope, 0, qkv, table(64, 40))
    refused("qkv", c.rope, 0, qkv[:2], tab)
    refused("qkv", c.rope, 0, qkv.half(), tab)
    refused("qkv", c.rope, 0, qkv.cpu(), tab)
    refused("qkv", c.rope, 0, qkv.t().contiguous().t(), tab)
    refused("qkv_stride", c.rope, 0, randn(0, 3, width + 1)[:, :width], tab)
    refused("aligned", c.rope, 0, randn(0, 3, width + 4)[:, 1:width + 1], tab)
    refused("table", c.rope, 0, qkv, tab.double())
    refused("q_weight", c.rope, 0, qkv, tab, q_weight=torch.ones(32, device="cuda"))
    refused("positions", c.rope, 0, qkv, tab, positions=torch.zeros(3, dtype=torch.int64, device="cuda"))
    refused("q_dtype", c.rope, 0, qkv, tab, q_dtype=torch.float16)
    refused("eps", c.rope, 0, qkv, tab, eps=-1.0)
    refused("eps", c.rope, 0, qkv, tab, eps=float("nan"))
    refused("q:", c.rope, 0, qkv, tab, q=torch.empty(3, 8, 64, dtype=torch.bfloat16, device="cuda"))
    refused("entries", c.prefill_qkv, 0, qkv, [3], tab)
    refused("exceed", c.prefill_qkv, 0, qkv, [3, 0, 0], tab, starts=[62, 0, 0])
    refused("negative", c.prefill_qkv, 0, qkv, [4, -1, 0], tab)
    refused("negative", c.prefill_qkv, 0, qkv, [3, 0, 0], tab, starts=[-1, 0, 0])
    refused("layers", c.fork, [0], [1], layers=(1, 3))
    refused("layers", c.fork, [0], [1], layers=(1, 1))
    refused("pairs", c.fork, [], [])
    refused("outside", c.fork, [0], [3])
    refused("outside", c.fork, [-1], [0])
    refused("another pair", c.fork, [0, 1], [2, 2])
    refused("another pair", c.fork, [0, 1], [1, 2])
    refused("another pair", c.fork, [0, 0], [0, 1])
    refused("below", c.fork, [0], [1], [-2])
    refused("capacity", c.fork, [0], [1], [65])
    refused("one entry", c.fork, [0], [1], [1, 2])
    keep = torch.zeros(2, 3, 2, 1, dtype=torch.int32, device="cuda")
    refused("keep", c.compact, keep[0])
    refused("keep", c.compact, keep.long())
    refused("keep", c.compact, keep, [0], [1])
    refused("keep_blocks", c.compact, torch.zeros(2, 3, 2, 9, dtype=torch.int32, device="cuda"))
    refused("another pair", c.compact, keep, [0, 1, 2], [1, 0, 2])
    q = randn(1, 3, 8, 64)
    refused("entries", c.attend_shared, 0, q, [0, 0], [0, 0, 0])
    refused("prefix_seq", c.attend_shared, 0, q, [0, 3, 0], [0, 0, 0])
    refused("prefix_seq", c.attend_shared, 0, q, [0, -3, 0], [0, 0, 0])
    refused("prefix_len", c.attend_shared, 0, q, [0, 0, 0], [65, 0, 0])
    refused("prefix_len", c.attend_shared, 0, q, [0, 0, 0], [-1, 0, 0])
    refused("q must", c.attend_shared, 0, q.half(), [0, 0, 0], [0, 0, 0])
    refused("out", c.attend_shared, 0, q, [0, 0, 0], [0, 0, 0], out=q.bfloat16())
    refused("device memory", make_cache([64], kv_memory="host").attend_shared, 0, q[:1], [0], [0])
    assert c.device_status() == 0


# ------------------------------------------------------------------ streams, graphs, together
def test_on_another_stream():
    c = shared_cache([512, 64], [500, 40], 2, 4, 64)
    q = randn(5, 2, 8, 64)
    want = c.attend_shared(0, q, [0, 0], [480, 0]).clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = c.attend_shared(0, q, [0, 0], [480, 0])
        c.fork([0], [1], [60])
    st.synchronize()
    assert torch.equal(got, want) and c.seq_len.tolist() == [[500, 60]]


def test_captured_and_replayed():
    # a step captured once and replayed while the sequences grow: norms, decode step and shared attention follow the lengths
    B, hkv, g, d = 3, 2, 4, 64
    c = shared_cache([320] + [64] * 2, [300, 0, 17], hkv, g, d)
    e = shared_cache([320] + [64] * 2, [300, 0, 17], hkv, g, d)
    tab, w = table(1024, d), 1 + 0.1 * randn(9, d)
    for x in (c, e):
        x.prefill(0, [300, 0, 17])
        x.shared_workspace()
    qkv = randn(1, B, (g + 2) * hkv * d).bfloat16()
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(x):
        q, k, v = x.rope(0, qkv, tab, q_weight=w, k_weight=w, positions=pos)
        x.append(0, k, v)
        return x.attend_shared(0, q, [0, 0, 0], [300, 0, 0])
    fresh = make_cache([32])
    with pytest.raises(Exception):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            fresh.attend_shared(0, randn(1, 1, 8, 64), [0], [0])
    torch.cuda.synchronize()
    before = state(c)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(c)
        st.synchronize()
    for t, o in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), before):
        t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for i in range(5):
        qkv.copy_(randn(20 + i, B, (g + 2) * hkv * d))
        pos.fill_(300 + i)
        graph.replay()
        want = step(e)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(c.seq_len, e.seq_len)
    assert c.device_status() == 0 and e.device_status() == 0


def test_a_prompt_shared_and_forked_gives_the_same_step():
    # a prompt prefilled once; its branches step (1) on copies of it, with a budget that selects every block, and (2) on the
    # shared prefix: both are exact attention over the same tokens.  Each is within 2e-3 of it, the decode step's own bound.
    B, hkv, g, d, n = 4, 2, 4, 64, 333
    tab = table(1024, d)
    w = 1 + 0.1 * randn(9, d)
    forked = make_cache([512] * B, hkv=hkv, g=g, d=d, budget=512)
    shared = make_cache([512] + [64] * (B - 1), hkv=hkv, g=g, d=d)
    prompt = randn(1, n, (g + 2) * hkv * d).bfloat16()
    for x in (forked, shared):
        # in two chunks, the second from the middle of a block
        x.prefill_qkv(0, prompt[:200], [200, 0, 0, 0], tab, k_weight=w, q_weight=w)
        x.prefill_qkv(0, prompt[200:], [n - 200, 0, 0, 0], tab, starts=[200, 0, 0, 0], k_weight=w, q_weight=w)
    whole = make_cache([512], hkv=hkv, g=g, d=d)
    whole.prefill_qkv(0, prompt, [n], tab, k_weight=w, q_weight=w)
    for h in range(hkv):
        for a, b in zip(whole.token_view(0, 0, h) + whole.summary_view(0, 0, h), forked.token_view(0, 0, h) + forked.summary_view(0, 0, h)):
            assert torch.equal(a[:336], b[:336])
    forked.fork([0] * 3, [1, 2, 3])
    for i in range(20):
        qkv = randn(50 + i, B, (g + 2) * hkv * d).bfloat16()
        q, k, v = forked.rope(0, qkv, tab, q_weight=w, k_weight=w)
        a = forked.decode(0, q, k, v)
        pos = torch.full((B,), n + i, dtype=torch.int32, device="cuda")
        q2, k2, v2 = shared.rope(0, qkv, tab, q_weight=w, k_weight=w, positions=pos)
        assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, v2)
        shared.append(0, k2, v2)
        b = shared.attend_shared(0, q2, [0] * B, [n, 0, 0, 0])
        assert (a - b).abs().max().item() <= 4e-3
    assert forked.device_status() == 0 and shared.device_status() == 0
    assert shared.seq_len.tolist() == [[n + 20, 20, 20, 20]]


def test_a_selection_compacts_and_decodes_on():
    # the blocks that a step selects become the cache; the next step over all of them is exact attention over those tokens
    hkv, g, d = 2, 4, 64
    c = filled([2048, 2048], [2000, 1500], layers=1, hkv=hkv, g=g, d=d, budget=256)
    q = randn(3, 2, hkv * g, d)
    sel = c.score_select(0, q)
    old = state(c)
    want = c.attend_shared(0, q, [-1, -1], [0, 0])  # before: every token
    c.compact(sel[None])
    torch.cuda.synchronize()
    assert c.device_status() == 0
    assert c.seq_len.tolist() == [[15 * 16 + 2000 - 124 * 16, 15 * 16 + 1500 - 93 * 16]]
    got = c.attend_shared(0, q, [-1, -1], [0, 0])
    lens = c.seq_len[0].tolist()
    check_shared(got, *shared64(c, 0, q, [-1, -1], [0, 0], lens))
    assert not torch.equal(got, want)
    for s in range(2):
        for h in range(hkv):
            a = heads_of(c, old[0], 0, s)[h][sel[s, h].long()].flatten(0, 1)[:lens[s]]
            assert torch.equal(c.token_view(0, s, h)[0][:lens[s]], a)
            check_summaries(c, 0, s, h, range(16), lens[s])


def test_every_layer_reads_its_own_rows():
    # the same tokens in layer 0 and in layer 2 of two caches: each call of layer 2 gives what it gives in layer 0
    hkv, g, d = 2, 4, 128
    one = filled([512, 256], [500, 130], layers=1, hkv=hkv, g=g, d=d, budget=128)
    three = filled([512, 256], [9, 250], layers=3, hkv=hkv, g=g, d=d, seed=50, budget=128)
    rows = one.k.shape[0]
    for x, y in zip(state(three)[:5], (one.k, one.v, one.kbar, one.vbar, one.dbar)):
        assert x.shape[0] == 3 * rows and y.shape[0] == rows
    for x, y in zip((three.k, three.v, three.kbar, three.vbar, three.dbar), (one.k, one.v, one.kbar, one.vbar, one.dbar)):
        x[2 * rows:] = y
    three.seq_len[2] = one.seq_len[0]
    q = randn(3, 2, hkv * g, d)
    new = [randn(s, 2, hkv, d, dtype=torch.bfloat16) for s in (4, 5)]
    a, b = (c.attend_shared(l, q, [0, 0], [400, 0]) for c, l in ((one, 0), (three, 2)))
    assert torch.equal(a, b)
    a, b = (c.decode(l, q, *new) for c, l in ((one, 0), (three, 2)))
    assert torch.equal(a, b)
    qkv, tab = randn(6, 40, (g + 2) * hkv * d), table(600, d)
    a, b = (c.prefill_qkv(l, qkv, [3, 37], tab, starts=[500, 0]) for c, l in ((one, 0), (three, 2)))
    assert torch.equal(a, b)
    one.fork([0], [1], [200])
    three.fork([0], [1], [200], layers=(2, 3))
    keep = torch.tensor([[[0, 2, 5, 12]] * hkv], dtype=torch.int32, device="cuda")[None]
    one.compact(keep, [1])
    three.compact(keep, [1], layers=(2, 3))
    for x, y in zip((three.k, three.v, three.kbar, three.vbar, three.dbar), (one.k, one.v, one.kbar, one.vbar, one.dbar)):
        assert torch.equal(x[2 * rows:], y)
    assert torch.equal(three.seq_len[2], one.seq_len[0]) and one.device_status() == 0 and three.device_status() == 0


def test_rows_far_into_a_large_cache():
    # 5 GB of keys: rows whose byte offsets pass 32 bits give what they give in a small cache
    hkv, g, d = 8, 1, 128
    big = make_cache([131072] * 20, hkv=hkv, g=g, d=d)
    small = make_cache([1024] * 2, hkv=hkv, g=g, d=d)
    assert big.k.numel() * 2 > 2 ** 32
    qkv, tab = randn(1, 700, (g + 2) * hkv * d).bfloat16(), table(1024, d)
    q = randn(2, 20, hkv * g, d)
    counts = [0] * 19 + [700]
    a = big.prefill_qkv(0, qkv, counts, tab)
    b = small.prefill_qkv(0, qkv, [0, 700], tab)
    assert torch.equal(a, b)
    prefix_len = [0] * 19 + [650]
    a = big.attend_shared(0, q, [-2] * 18 + [19, 19], prefix_len)
    b = small.attend_shared(0, q[18:].contiguous(), [1, 1], [0, 650])
    # pieces end elsewhere (other items come before): the same numbers, added in another order
    assert (a[18:] - b).abs().max().item() <= 1e-5
    keep = torch.tensor([[[0, 3, 9, 43]] * hkv], dtype=torch.int32, device="cuda")[None]
    big.fork([19], [18], [690])
    small.fork([1], [0], [690])
    big.compact(keep, [18])
    small.compact(keep, [0])
    for s, t in ((18, 0), (19, 1)):
        for h in range(hkv):
            for x, y in zip(big.token_view(0, s, h) + big.summary_view(0, s, h), small.token_view(0, t, h) + small.summary_view(0, t, h)):
                assert torch.equal(x[:40], y[:40])
    assert big.seq_len[0, 18:].tolist() == small.seq_len[0].tolist() == [3 * 16 + 2, 700]
    assert big.device_status() == 0 and small.device_status() == 0
