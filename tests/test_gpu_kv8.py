"""K and V in 8 bits against plain 64-bit restatements: what is stored for which tokens, what is read back, attention
over everything and over a selection, the fused decode step; alone at the sizes where they can go wrong, refused where
they must be, on streams and in graphs, and together as a server would use them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 16
F32 = 2.0 ** -24   # largest relative error of one fp32 rounding
BF16 = 2.0 ** -8   # and of one bf16 rounding
KV8 = [torch.int8, torch.float8_e4m3fn]
MOST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_sparse_kv_summary_gb300 as P
    P.build()
    P.lib()


def make_cache(caps, kv=torch.int8, *, layers=1, hkv=2, g=4, d=64, r=4, budget=128, variant=0):
    from block_sparse_kv_summary_gb300 import CompKVCache
    return CompKVCache(num_layers=layers, batch=len(caps), num_kv_heads=hkv, group_size=g, head_dim=d, r=r, budget_tokens=budget,
                       capacity_tokens=list(caps), kv_dtype=kv, variant=variant)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=gen(seed)).to(dtype)


def table(positions, rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def bits(t):
    return t.view(torch.int8) if t.element_size() == 1 else t.view(torch.int32) if t.dtype == torch.float32 else t


def quantised(x, kv):
    """Codes and scales of blocks x [..., 16, d] of fp32 values, by the definition."""
    m = x.abs().amax((-1, -2))
    most = torch.full_like(m, MOST[kv])
    held = m >= 2.0 ** -100
    inv = torch.where(held, most / m, 0.0)
    y = x * inv[..., None, None]
    return (y.round() if kv == torch.int8 else y).to(kv), torch.where(held, m / most, 0.0)


def values(c):
    """(K, V) of every row in 64 bits."""
    return [t.float().double() * s.double()[:, None, None] for t, s in ((c.k, c.kscale), (c.v, c.vscale))]


def fill(c, seed, lens, wide=True):
    """Random codes, scales and summaries in every row of the cache's layers; each layer's sequences hold lens tokens."""
    rows, d = c.k.shape[0], c.d
    k = randn(seed, rows, 1, d) + 0.4 * randn(seed + 1, rows, BLOCK, d)
    if wide:
        k[..., 3] *= 5
    v = randn(seed + 2, rows, BLOCK, d)
    for t, s, x in ((c.k, c.kscale, k), (c.v, c.vscale, v)):
        codes, s[:] = quantised(x.bfloat16().float(), c.kv_dtype)
        t.copy_(codes)
    c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32, device="cuda").expand(c.num_layers, -1))
    for l in range(c.num_layers):
        for s, n in enumerate(lens):
            for h in range(c.Hkv):
                r0, cap = c.rows(l, s, h)
                for b in range((n + BLOCK - 1) // BLOCK):
                    m = min(BLOCK, n - b * BLOCK)
                    x, y = k[r0 + b, :m].bfloat16().double(), v[r0 + b, :m].bfloat16().double()
                    c.kbar[r0 + b], c.vbar[r0 + b] = x.mean(0), y.mean(0)
                    c.dbar[r0 + b] = x.var(0, unbiased=False).view(c.r, -1).mean(-1)


def own_tokens(c, layer, s, h, n):
    r0, cap = c.rows(layer, s, h)
    return [t[r0:r0 + cap].reshape(-1, c.d)[:n] for t in values(c)]


def attention(c, layer, q, s, h, n, sel=None):
    """(output, bound on the fp32 kernel's error) of the query heads of unit (s, h), in 64 bits.  sel: the selected
    blocks; the others stand for their tokens with mean key and mean value."""
    d, G = c.d, c.G
    x = q[s, h * G:(h + 1) * G].double()
    out = torch.zeros(G, d, dtype=torch.float64, device="cuda")
    if not n:
        return out, out
    k, v = own_tokens(c, layer, s, h, n)
    z = x @ k.T / d ** 0.5
    # int8 codes enter the products 128 too large, which these start from: what a logit and an output add up
    r0, cap = c.rows(layer, s, h)
    bias = [(128.0 if c.kv_dtype == torch.int8 else 0.0) * t[r0:r0 + cap].double().repeat_interleave(BLOCK)[:n, None] for t in (c.kscale, c.vscale)]
    size = x.abs() @ (k.abs() + bias[0]).T / d ** 0.5
    vsize = v.abs() + bias[1]
    w = torch.ones(n, dtype=torch.float64, device="cuda")
    N = (n + BLOCK - 1) // BLOCK
    removed = 0.0
    if sel is not None:
        r0, _ = c.rows(layer, s, h)
        kb, vb = c.kbar[r0:r0 + N].double(), c.vbar[r0:r0 + N].double()
        count = torch.tensor([min(BLOCK, n - b * BLOCK) for b in range(N)], dtype=torch.float64, device="cuda")
        taken = torch.zeros(N, dtype=torch.bool, device="cuda")
        taken[sel] = True
        tok = taken.repeat_interleave(BLOCK)[:n]
        if c.variant & 4:  # no compensation
            k, v, z, size, w, vsize = k[tok], v[tok], z[:, tok], size[:, tok], w[tok], vsize[tok]
        else:
            zb, sb = x @ kb.T / d ** 0.5, x.abs() @ kb.abs().T / d ** 0.5
            if not taken.all():
                # the sums over all blocks are formed first, and the selected blocks' shares come off again
                removed = (count * torch.exp(zb - z.amax(-1, keepdim=True))) @ vb.abs()
            z = torch.cat([z[:, tok], zb[:, ~taken]], 1)
            size = torch.cat([size[:, tok], sb[:, ~taken]], 1)
            v = torch.cat([v[tok], vb[~taken]])
            vsize = torch.cat([vsize[tok], vb[~taken].abs()])
            w = torch.cat([w[tok], count[~taken]])
            if not taken.all():
                removed = (count * torch.exp(zb - z.amax(-1, keepdim=True))) @ vb.abs()
    p = w * torch.exp(z - z.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    out = p @ v / total
    # relative error of a weight: the logit's products and their sum (11 steps of 2^-22 of what it adds up: two parts of a
    # query, 8 products in a row whose accumulator truncates, the bias's own sum), its three factors and the distance from
    # the reference (each 2^-24 of up to |z| + 20 in log2 units), the exponential (2^-22), the weight's two parts (2^-22)
    span = z.abs().amax() + 20
    eps = 12 * 4 * F32 * size.amax() + 8 * F32 * span + 8 * F32
    # sums: at most one rounding a token in the denominator, two truncations and a rounding a block in the numerator,
    # and some 60 in the joins; a stream of means adds as many again
    eps = eps + (4 * n / BLOCK + n + 60) * F32 if n < 4096 else eps + (n / 64 + 300) * F32
    mag = p @ vsize / total + out.abs() + removed / total
    return out, 2 * eps * mag


def check(c, got, layer, q, lens, sel=None):
    for s, n in enumerate(lens):
        for h in range(c.Hkv):
            pick = None if sel is None else [b for b in sel[s, h].tolist() if b >= 0]
            want, tol = attention(c, layer, q, s, h, n, pick)
            y = got[s, h * c.G:(h + 1) * c.G].double()
            if got.dtype == torch.bfloat16:
                tol = tol * (1 + BF16) + BF16 * want.abs()
            bad = ((y - want).abs() - tol).max().item()
            assert bad <= 0, (s, h, n, bad, (y - want).abs().max().item())


# ------------------------------------------------------------------ what is stored
def write(c, lens_from_to, seed, hkv, g, d, layer=0):
    """One prefill_qkv of the tokens [a, b) of every sequence, from a projection that depends on the seed."""
    starts, counts = [a for a, _ in lens_from_to], [b - a for a, b in lens_from_to]
    qkv = randn(seed, sum(counts), (g + 2) * hkv * d, dtype=torch.bfloat16)
    return c.prefill_qkv(layer, qkv, counts, table(4096, d), starts=starts, k_weight=1 + 0.1 * randn(9, d), q_weight=None)


def check_stored(c8, c16, lens, layer=0):
    """Codes and scales are those of the bf16 cache's tokens, to the bit; summaries are the same."""
    for s, n in enumerate(lens):
        for h in range(c8.Hkv):
            r0, _ = c8.rows(layer, s, h)
            N = (n + BLOCK - 1) // BLOCK
            for t8, sc, t16 in ((c8.k, c8.kscale, c16.k), (c8.v, c8.vscale, c16.v)):
                x = t16[r0:r0 + N].float()
                x.view(-1, c8.d)[n:] = 0
                codes, scale = quantised(x, c8.kv_dtype)
                assert torch.equal(bits(sc[r0:r0 + N]), bits(scale)), (s, h)
                assert torch.equal(bits(t8[r0:r0 + N]).view(-1, c8.d)[:n], bits(codes).view(-1, c8.d)[:n]), (s, h)
            for a, b in ((c8.kbar, c16.kbar), (c8.vbar, c16.vbar), (c8.dbar, c16.dbar)):
                assert torch.equal(bits(a[r0:r0 + N]), bits(b[r0:r0 + N])), (s, h)
    assert c8.seq_len[layer].tolist() == list(lens)


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g,r", [(64, 2, 4, 4), (128, 8, 4, 64), (128, 1, 8, 1), (64, 5, 1, 32), (128, 3, 2, 128)])
def test_prefill_stores_the_codes_of_its_tokens(kv, d, hkv, g, r):
    # one token, a full block, a block and one, odd ones; none; then more, from inside a block, over one and several
    # block ends (where the last block's tail replaces the one that the first block reads), and from a block's end
    caps = [64, 64, 64, 96, 64, 208]
    steps = [[(0, 1), (0, 16), (0, 17), (0, 45), (0, 0), (0, 33)],
             [(1, 2), (16, 16), (17, 40), (45, 90), (0, 3), (33, 200)],
             [(2, 17), (16, 33), (40, 64), (90, 90), (3, 48), (200, 208)]]
    c8, c16 = make_cache(caps, kv, hkv=hkv, g=g, d=d, r=r), make_cache(caps, torch.bfloat16, hkv=hkv, g=g, d=d, r=r)
    for i, step in enumerate(steps):
        q8, q16 = write(c8, step, 50 + i, hkv, g, d), write(c16, step, 50 + i, hkv, g, d)
        assert torch.equal(q8, q16)
        check_stored(c8, c16, [b for _, b in step])
    assert c8.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 8), (128, 11)])
def test_append_stores_the_codes_of_its_tokens(kv, d, hkv):
    caps = [64, 48, 64]
    c8, c16 = make_cache(caps, kv, hkv=hkv, d=d), make_cache(caps, torch.bfloat16, hkv=hkv, d=d)
    start = [(0, 0), (0, 15), (0, 32)]
    for c in (c8, c16):
        write(c, start, 3, hkv, 4, d)
    lens = [b for _, b in start]
    for t in range(20):
        # sizes go up and down, so that some tokens widen their block's scale and others do not
        k = randn(100 + t, 3, hkv, d, dtype=torch.bfloat16) * (0.5 + (t * 7 % 5))
        v = randn(200 + t, 3, hkv, d, dtype=torch.bfloat16) * (0.5 + (t * 5 % 7))
        for c in (c8, c16):
            c.append(0, k, v)
        lens = [n + 1 for n in lens]
        check_stored(c8, c16, lens)
    assert c8.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("append", [False, True])
def test_a_cut_into_an_older_block_goes_on_from_its_codes(kv, append):
    hkv, d = 2, 64
    c = make_cache([96], kv, hkv=hkv, d=d)
    write(c, [(0, 50)], 1, hkv, 4, d)
    old = [x.clone() for x in values(c)]
    cut = 21  # inside block 1, while the tail holds block 3
    if append:
        c.seq_len.fill_(cut)
        new = [randn(5 + i, 1, hkv, d, dtype=torch.bfloat16) for i in range(2)]
        c.append(0, *new)
    else:
        write(c, [(cut, cut + 1)], 7, hkv, 4, d)
        twin = make_cache([96], torch.bfloat16, hkv=hkv, d=d)
        write(twin, [(cut, cut + 1)], 7, hkv, 4, d)
        new = [torch.stack([t[twin.rows(0, 0, h)[0] + 1, cut - 16] for h in range(hkv)])[None] for t in (twin.k, twin.v)]
    for h in range(hkv):
        r = c.rows(0, 0, h)[0] + 1
        for x, codes, scale, y in zip(old, (c.k, c.v), (c.kscale, c.vscale), new):
            block = torch.zeros(BLOCK, d, device="cuda")
            block[:cut - 16] = x[r, :cut - 16].float().bfloat16().float()
            block[cut - 16] = y[0, h].float()
            want, s = quantised(block, kv)
            assert torch.equal(bits(codes[r])[:cut - 15], bits(want)[:cut - 15]) and scale[r] == s
    assert c.seq_len.item() == cut + 1
    # and within the last block, the tail holds the tokens as they came
    write(c, [(cut, cut + 4)], 8, hkv, 4, d)
    tail = c.tail.clone()
    write(c, [(cut + 2, cut + 4)], 9, hkv, 4, d)
    unit = torch.arange(hkv, device="cuda")
    place = (c.tail_len == cut + 4).int().argmax(1)
    assert (c.tail_len[unit, place] == cut + 4).all()
    assert torch.equal(c.tail[unit, place][:, :, :cut - 14], tail[unit, place][:, :, :cut - 14])
    assert not torch.equal(c.tail[unit, place][:, :, cut - 14:cut - 12], tail[unit, place][:, :, cut - 14:cut - 12])


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("append", [False, True])
def test_cuts_into_blocks_that_the_tail_holds(kv, append):
    # a call that began inside a block is taken back, to where it began and to a place before, and its block goes on with
    # other tokens; what was written over it since does not come back
    hkv, d = 3, 128
    c8, c16 = make_cache([160], kv, hkv=hkv, d=d), make_cache([160], torch.bfloat16, hkv=hkv, d=d)

    def both(a, b, seed):
        for c in (c8, c16):
            if append and b == a + 1:
                c.seq_len.fill_(a)
                c.append(0, *(randn(seed + i, 1, hkv, d, dtype=torch.bfloat16) * (1 + seed % 3) for i in range(2)))
            else:
                write(c, [(a, b)], seed, hkv, 4, d)
        check_stored(c8, c16, [b])

    both(0, 40, 1)
    both(40, 100, 2)    # began inside block 2
    both(100, 101, 3)   # goes on behind it
    both(40, 41, 4)     # taken back to where it began
    both(41, 90, 5)
    both(38, 39, 6)     # and to a place before, in the same block
    both(39, 77, 7)
    both(77, 130, 8)    # began inside block 4
    both(70, 71, 9)     # block 4 goes on with other tokens
    both(71, 100, 10)
    both(64, 120, 11)   # block 4 from its start, with others again: what the tail had of it is gone
    assert (c8.tail_len > 64).sum().item() == hkv and (c8.tail_len == 120).sum().item() == hkv
    both(120, 121, 12)  # the last block goes on, wherever it stands
    both(121, 127, 13)
    both(127, 150, 14)  # from inside the last block into the next two
    both(127, 160, 15)  # and again, longer
    both(125, 126, 16)  # back into the block that the call began inside
    both(16, 17, 17)    # far back, at a block's start


def test_many_writes_keep_the_tail_in_order():
    # random cuts and writes of two sequences: wherever the tail has the tokens in front, codes are those of the tokens in
    # bf16; elsewhere the bf16 cache first takes over what the codes stand for
    import random
    rng = random.Random(5)
    hkv, d, cap = 5, 64, 192
    c8, c16 = make_cache([cap, cap], torch.int8, hkv=hkv, d=d), make_cache([cap, cap], torch.bfloat16, hkv=hkv, d=d)
    lens = [0, 0]
    for step in range(60):
        span = []
        for s in range(2):
            a = lens[s] if rng.random() < 0.5 else rng.randrange(max(0, lens[s] - 40), lens[s] + 1)
            span.append((a, min(cap, a + rng.choice([0, 1, 3, 16, 30, 50]))))
        for s, (a, b) in enumerate(span):
            if b > a and a % BLOCK:
                held = c8.tail_len[s * hkv].tolist()
                if not any(BLOCK * (a // BLOCK) < x <= BLOCK * (a // BLOCK + 1) and x >= a for x in held):
                    vk, vv = values(c8)
                    for h in range(hkv):
                        r = c8.rows(0, s, h)[0] + a // BLOCK
                        for t, x in ((c16.k, vk), (c16.v, vv)):
                            t[r, :a % BLOCK] = x[r, :a % BLOCK].float().bfloat16()
        for c in (c8, c16):
            write(c, span, 1000 + step, hkv, 4, d)
        lens = [b if b > a else n for (a, b), n in zip(span, lens)]
        # (a block behind the end of a shorter write may be out of date in either cache: the first `lens` tokens count)
        check_stored(c8, c16, lens)
        if max(lens) > cap - 20:
            for c in (c8, c16):
                c.seq_len.fill_(0)
            lens = [0, 0]


@pytest.mark.parametrize("kv", KV8)
def test_a_call_again_stores_the_same(kv):
    hkv, d = 2, 64
    c = make_cache([64, 320, 96], kv, hkv=hkv, d=d)
    write(c, [(0, 20), (0, 77), (0, 33)], 1, hkv, 4, d)
    held = None
    for _ in range(3):
        write(c, [(20, 41), (77, 300), (33, 40)], 2, hkv, 4, d)
        now = [bits(t).clone() for t in (c.k, c.v, c.kscale, c.vscale, c.kbar, c.vbar, c.dbar)]
        now.append(c.tail_len.sort(1).values)  # (which place of the tail holds which block may change)
        assert held is None or all(torch.equal(a, b) for a, b in zip(held, now))
        held = now


@pytest.mark.parametrize("kv", KV8)
def test_blocks_of_nothing_infinities_and_tiny_values(kv):
    hkv, d = 1, 128
    c = make_cache([16] * 7, kv, hkv=hkv, g=1, d=d)
    k = randn(1, 7, hkv, d, dtype=torch.bfloat16)
    v = randn(2, 7, hkv, d, dtype=torch.bfloat16)
    k[0] = 0
    k[1], v[1] = 2.0 ** -101, 2.0 ** -99
    k[2, 0, 5] = float("inf")
    v[3, 0, 6] = float("nan")
    k[4], v[4] = 3.0e38, -3.0e38
    v[5, 0, 7] = float("-inf")
    c.append(0, k, v)
    gk, gv = c.read(0, None, [1] * 7, dtype=torch.float32)
    assert (gk[0] == 0).all() and (gk[1] == 0).all()
    assert torch.equal(gv[1], v[1].float()) and torch.equal(gk[4], k[4].float()) and torch.equal(gv[4], v[4].float())
    assert gk[2].isnan().all() and gv[3].isnan().all() and gv[5].isnan().all()
    assert gv[2].isfinite().all() and gk[3].isfinite().all() and gk[6].isfinite().all()
    # a NaN reaches the rows of its own sequence and no other (the logits of sequence 4, some 3e38 times log2 e, are beyond
    # what the call takes)
    out = c.attend_all(0, randn(3, 7, 1, d))
    for s in (2, 3, 5):
        assert out[s].isnan().all()
    assert out[[0, 1, 6]].isfinite().all()


# ------------------------------------------------------------------ read back
@pytest.mark.parametrize("kv", [*KV8, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 8)])
def test_read(kv, dtype, d, hkv):
    caps, lens = [48, 16, 112, 16, 32], [47, 16, 100, 0, 32]
    c = make_cache(caps, kv, hkv=hkv, d=d, layers=2)
    if kv == torch.bfloat16:
        c.k.copy_(randn(1, *c.k.shape))
        c.v.copy_(randn(2, *c.v.shape))
        c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32).expand(2, -1))
        vals = [c.k.double(), c.v.double()]
    else:
        fill(c, 1, lens)
        # one fp32 rounding, then the output's
        vals = [(t.float() * s[:, None, None]).double() for t, s in ((c.k, c.kscale), (c.v, c.vscale))]
    for starts, counts in ((None, lens), ([3, 0, 15, 0, 31], [1, 16, 35, 0, 1]), ([0, 15, 16, 0, 5], [0, 1, 84, 0, 27])):
        k, v = c.read(1, starts, counts, dtype=dtype)
        for got, x in ((k, vals[0]), (v, vals[1])):
            parts = []
            for s, n in enumerate(counts):
                a = 0 if starts is None else starts[s]
                heads = [x[c.rows(1, s, h)[0]:c.rows(1, s, h)[0] + caps[s] // BLOCK].reshape(-1, d)[a:a + n] for h in range(hkv)]
                parts.append(torch.stack(heads, 1))
            assert torch.equal(got, torch.cat(parts).to(dtype))
    assert c.device_status() == 0


def test_read_leaves_what_the_sequence_does_not_hold():
    c = make_cache([64, 64])
    fill(c, 1, [20, 64])
    k = torch.full((60, 2, 64), 7.0, device="cuda")
    v = torch.full((60, 2, 64), 8.0, device="cuda")
    c.read(0, [10, 5], [30, 30], torch.float32, k, v)
    assert (k[10:30] == 7).all() and (v[10:30] == 8).all()
    want = c.read(0, [10, 5], [10, 30], torch.float32)
    assert torch.equal(torch.cat([k[:10], k[30:]]), want[0]) and torch.equal(torch.cat([v[:10], v[30:]]), want[1])
    from block_sparse_kv_summary_gb300 import compkv as C
    assert c.device_status() == 1 and "sequence 0" in C.compkv_last_error()
    assert c.device_status() == 0


def test_read_from_host_memory():
    from block_sparse_kv_summary_gb300 import CompKVCache
    c = CompKVCache(num_layers=1, batch=2, num_kv_heads=2, group_size=4, head_dim=64, r=4, budget_tokens=128, capacity_tokens=[48, 64],
                    kv_memory="host")
    c.k.copy_(randn(1, *c.k.shape).bfloat16())
    c.v.copy_(randn(2, *c.v.shape).bfloat16())
    c.seq_len.copy_(torch.tensor([[40, 64]], dtype=torch.int32))
    k, v = c.read(0, [1, 0], [39, 64])
    for s, n, a, at in ((0, 39, 1, 0), (1, 64, 0, 39)):
        for h in range(2):
            tk, tv = c.token_view(0, s, h)
            assert torch.equal(k[at:at + n, h].cpu(), tk[a:a + n]) and torch.equal(v[at:at + n, h].cpu(), tv[a:a + n])


# ------------------------------------------------------------------ attention over everything
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,hkv,g", [(64, 2, 4), (128, 8, 8), (128, 1, 1), (64, 3, 2), (64, 1, 8)])
def test_attend_all(kv, dtype, d, hkv, g):
    # none, one, a block less one, a block, one more; two blocks and one; more blocks than a CTA's warps take at once
    lens = [0, 1, 15, 16, 17, 33, 300, 0, 1000]
    caps = [16, 16, 16, 16, 32, 48, 304, 16, 1008]
    c = make_cache(caps, kv, hkv=hkv, g=g, d=d, layers=2)
    fill(c, 10, lens)
    q = randn(20, len(lens), hkv * g, d, dtype=dtype)
    out = torch.full_like(q, 9.0)
    assert c.attend_all(1, q, out) is out
    check(c, out, 1, q, lens)
    assert torch.equal(out, c.attend_all(1, q)) and c.device_status() == 0


@pytest.mark.parametrize("kv,d,hkv,g,lens", [
    (torch.int8, 128, 1, 4, [40000]),             # one unit over every CTA
    (torch.float8_e4m3fn, 64, 2, 8, [9999, 20]),  # cut at odd places
    (torch.int8, 128, 8, 4, [2049, 1, 4097, 700, 0, 333, 5000, 16]),
    (torch.float8_e4m3fn, 128, 4, 2, [777] * 64),
])
def test_attend_all_over_many_ctas(kv, d, hkv, g, lens):
    c = make_cache([max(16, (n + 15) // 16 * 16) for n in lens], kv, hkv=hkv, g=g, d=d)
    for seed, t in ((1, c.k), (2, c.v)):  # any sign, magnitudes up to 120 (which e4m3 has as numbers)
        x = torch.randint(0, 121, t.shape, device="cuda", generator=gen(seed)) * torch.randint(0, 2, t.shape, device="cuda", generator=gen(seed)).mul(2).sub(1)
        t.view(torch.int8).copy_(x if kv == torch.int8 else x.abs() - 128 * (x < 0))
    c.kscale.uniform_(0.005, 0.02, generator=gen(3))
    c.vscale.uniform_(0.01, 0.02, generator=gen(4))
    c.seq_len.copy_(torch.tensor([lens], dtype=torch.int32))
    q = randn(5, len(lens), hkv * g, d)
    out = c.attend_all(0, q)
    check(c, out, 0, q, lens)
    for _ in range(3):
        assert torch.equal(out, c.attend_all(0, q))  # the parts are joined in one order


def test_attend_all_large_and_small_numbers():
    # heads of very different size, scales that differ by far, one logit that carries everything
    c = make_cache([64], torch.int8, hkv=1, g=8, d=128)
    fill(c, 3, [64], wide=False)
    c.kscale.mul_(torch.tensor([1.0, 3.0, 1e-6, 10.0], device="cuda"))
    c.vscale.mul_(torch.tensor([1e-8, 1.0, 1e6, 1.0], device="cuda"))
    q = randn(4, 1, 8, 128) * torch.tensor([1.0, 1e-20, 1e-38, 0.0, 10.0, 1e-3, 30.0, 1e-5], device="cuda")[:, None]
    check(c, c.attend_all(0, q), 0, q, [64])


# ------------------------------------------------------------------ attention over a selection
def selection(seed, c, lens, K):
    sel = torch.full((c.batch, c.Hkv, K), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(seed)
    for s, n in enumerate(lens):
        N = (n + BLOCK - 1) // BLOCK
        for h in range(c.Hkv):
            m = min(K, N)
            sel[s, h, :m] = torch.randperm(N, generator=g)[:m].sort().values.int()
    return sel


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g,r", [(64, 2, 4, 4), (128, 8, 8, 128), (128, 2, 1, 1), (64, 1, 2, 64)])
@pytest.mark.parametrize("variant", [0, 4])
def test_attend_a_selection(kv, d, hkv, g, r, variant):
    lens = [1, 0, 130, 16, 1200, 129]
    caps = [16, 16, 144, 16, 1200, 144]
    c = make_cache(caps, kv, hkv=hkv, g=g, d=d, r=r, budget=128, variant=variant)
    fill(c, 30, lens)
    q = randn(31, len(lens), hkv * g, d)
    for seed in (0, 1):
        sel = selection(seed, c, lens, 8)
        if seed:  # fewer than the budget, and none at all: every block stands for its tokens
            sel[2, :, 3:] = -1
            sel[4, 0] = -1
        out = c.attend(0, q, sel)
        if variant and seed:
            assert (out[4, :g] == 0).all()  # no token and no mean
            sel[4, 0, 0] = 0
            out = c.attend(0, q, sel)
        check(c, out, 0, q, lens, sel)
    assert c.device_status() == 0


def test_a_bad_selection_is_reported():
    c = make_cache([256, 256], torch.int8)
    fill(c, 1, [250, 250])
    q = randn(2, 2, 8, 64)
    sel = selection(3, c, [250, 250], 8)
    good = c.attend(0, q, sel)
    sel[1, 1, 3] = sel[1, 1, 2]
    out = c.attend(0, q, sel)
    assert torch.equal(out[0], good[0]) and torch.equal(out[1, :4], good[1, :4])
    assert c.device_status() == 6
    sel[1, 1, 3] = 16  # as many blocks as there are
    c.attend(0, q, sel)
    assert c.device_status() == 6 and c.device_status() == 0


# ------------------------------------------------------------------ the fused step
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g,r,budget", [(64, 2, 4, 4, 128), (128, 8, 4, 4, 256), (128, 2, 8, 128, 48)])
def test_decode(kv, d, hkv, g, r, budget):
    # selections are those of the same tokens in bf16 (the summaries are the same); outputs are those of the codes
    lens = [0, 1, 100, 1007, 640]
    caps = [32, 32, 128, 1024, 656]
    c8, c16 = (make_cache(caps, t, hkv=hkv, g=g, d=d, r=r, budget=budget) for t in (kv, torch.bfloat16))
    for c in (c8, c16):
        write(c, [(0, n) for n in lens], 3, hkv, g, d)
    for t in range(18):
        q = randn(300 + t, len(lens), hkv * g, d)
        k, v = (randn(400 + 10 * t + i, len(lens), hkv, d, dtype=torch.bfloat16) for i in range(2))
        sel = c8.new_sel()
        out = c8.decode(0, q, k, v, sel=sel)
        lens = [n + 1 if n < cap else n for n, cap in zip(lens, caps)]
        c16.append(0, k, v)
        want = c16.score_select(0, q)
        assert torch.equal(sel, want)
        assert torch.equal(c8.score_select(0, q), want)
        check_stored(c8, c16, lens)
        check(c8, out, 0, q, lens, sel)
        if t < 2:
            assert torch.equal(c8.attend(0, q, sel)[0], out[0])
    from block_sparse_kv_summary_gb300 import compkv as C
    assert c8.device_status() == 3 and "sequence 4" in C.compkv_last_error()  # 640 + 16 tokens were all that it holds


def test_decode_host():
    c, d = make_cache([128, 64], torch.int8), 64
    twin = make_cache([128, 64], torch.int8)
    for x in (c, twin):
        write(x, [(0, 100), (0, 40)], 3, 2, 4, d)
    for pinned in (False, True):
        host = [torch.randn(2, 8, d), torch.randn(2, 2, d).bfloat16(), torch.randn(2, 2, d).bfloat16(), torch.empty(2, 8, d),
                torch.empty(2, 2, 8, dtype=torch.int32)]
        if pinned:
            host = [t.pin_memory() for t in host]
        out = c.decode_host(0, *host[:4], sel=host[4])
        sel = twin.new_sel()
        want = twin.decode(0, *(t.cuda() for t in host[:3]), sel=sel)
        assert torch.equal(out, want.cpu()) and torch.equal(host[4], sel.cpu())


# ------------------------------------------------------------------ refusals
def test_refusals():
    from block_sparse_kv_summary_gb300 import CompKVCache
    from block_sparse_kv_summary_gb300 import compkv as C
    c = make_cache([64, 32], torch.int8)
    q = randn(1, 2, 8, 64)
    for call in (lambda: c.prefill(0, [1, 1]), lambda: c.fork([0], [1]), lambda: c.truncate([0], [1]),
                 lambda: c.compact(torch.zeros(1, 2, 2, 1, dtype=torch.int32, device="cuda")),
                 lambda: C.compkv_attend_shared(c.ctx, 0, q.data_ptr(), 1, [-1, -1], [0, 0], q.data_ptr(), q.data_ptr(), 1 << 30, 0),
                 lambda: C.compkv_trace(c.ctx, q.data_ptr(), 4096)):
        with pytest.raises(C.CompKVError, match="8 bits"):
            call()
    with pytest.raises(C.CompKVError, match="attend_shared"):
        make_cache([64, 32], torch.bfloat16).attend_all(0, q)
    with pytest.raises(ValueError, match="kv_dtype"):
        make_cache([64], torch.float16)
    with pytest.raises(ValueError, match="GPU memory"):
        CompKVCache(num_layers=1, batch=1, num_kv_heads=2, group_size=4, head_dim=64, r=4, budget_tokens=128, capacity_tokens=64,
                    kv_memory="host", kv_dtype=torch.int8)
    for args, msg in (((0, [0], [1, 1]), "entries"), ((0, None, [1]), "entries"), ((0, None, [-1, 2]), "negative"),
                      ((0, None, [1, 1], torch.float16), "dtype")):
        with pytest.raises(ValueError, match=msg):
            c.read(*args)
    for args, msg in (((0, [-1, 0], [1, 1]), "negative"), ((0, [60, 0], [5, 1]), "capacity"), ((2, None, [1, 1]), "layer"),
                      ((0, [70, 0], [0, 1]), None)):
        if msg is None:  # nothing is read of a sequence with no count
            c.seq_len.fill_(1)
            c.read(*args)
            continue
        with pytest.raises(C.CompKVError, match=msg):
            c.read(*args)
    k = torch.empty(2 * 2 * 64 + 8, device="cuda")
    with pytest.raises(C.CompKVError, match="32-byte"):
        C.compkv_read(c.ctx, 0, None, [1, 1], 1, k.data_ptr() + 16, k.data_ptr(), 0)
    for bad, msg in ((q[:1], "q"), (q.half(), "float32 or"), (q.cpu(), "q"), (q.transpose(0, 1), "q")):
        with pytest.raises(ValueError, match=msg):
            c.attend_all(0, bad)
    with pytest.raises(ValueError, match="out"):
        c.attend_all(0, q, q.bfloat16())
    with pytest.raises(C.CompKVError, match="type"):
        C.compkv_attend_all(c.ctx, 0, q.data_ptr(), 2, q.data_ptr(), 0)
    assert c.device_status() == 0


# ------------------------------------------------------------------ streams, graphs, together
def test_in_place_over_the_queries():
    c = make_cache([512, 64], torch.int8)
    fill(c, 1, [500, 64])
    for dtype in (torch.float32, torch.bfloat16):
        q = randn(2, 2, 8, 64, dtype=dtype)
        want = c.attend_all(0, q)
        assert torch.equal(c.attend_all(0, q, q), want)


def test_streams_and_graphs():
    hkv, g, d = 2, 4, 64
    caps = [256, 96]
    c, twin = make_cache(caps, torch.int8, hkv=hkv, g=g, d=d), make_cache(caps, torch.int8, hkv=hkv, g=g, d=d)
    for x in (c, twin):
        write(x, [(0, 200), (0, 61)], 3, hkv, g, d)
    torch.cuda.synchronize()
    q = randn(1, 2, hkv * g, d)
    k, v = (randn(2 + i, 2, hkv, d, dtype=torch.bfloat16) for i in range(2))
    dense, out, sel = torch.empty_like(q), torch.empty_like(q), c.new_sel()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            c.decode(0, q, k, v, out=out, sel=sel)
            c.attend_all(0, q, dense)
    for t in range(20):  # over a block's end, lengths that only the device knows
        q.copy_(randn(50 + t, *q.shape))
        k.copy_(randn(90 + t, *k.shape))
        v.copy_(randn(130 + t, *v.shape))
        graph.replay()
        s2 = twin.new_sel()
        assert torch.equal(twin.decode(0, q, k, v, sel=s2), out) and torch.equal(s2, sel)
        assert torch.equal(twin.attend_all(0, q), dense)
    assert c.seq_len.tolist() == [[220, 81]] and c.device_status() == 0


def test_two_caches_on_two_streams():
    caches = [make_cache([4096, 1024], t, hkv=4, d=128) for t in KV8]
    for i, c in enumerate(caches):
        fill(c, 7 * i, [4001, 1000])
    q = [randn(70 + i, 2, 16, 128) for i in range(2)]
    want = [c.attend_all(0, x) for c, x in zip(caches, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(caches[i].attend_all(0, q[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("kv", KV8)
def test_a_conversation(kv):
    """A prompt in two chunks, read back for their attention; sparse steps with a dense one now and then; a new prompt in a
    used sequence."""
    hkv, g, d = 2, 4, 128
    caps = [512, 256, 64]
    c, twin = (make_cache(caps, t, layers=2, hkv=hkv, g=g, d=d, budget=96) for t in (kv, torch.bfloat16))
    lens = [300, 131, 40]
    for layer in range(2):
        for x in (c, twin):
            write(x, [(0, n // 2) for n in lens], layer, hkv, g, d, layer)
            write(x, [(n // 2, n) for n in lens], 10 + layer, hkv, g, d, layer)
        check_stored(c, twin, lens, layer)
        k, v = c.read(layer, None, lens, torch.float32)
        kk, vv = twin.read(layer, None, lens, torch.float32)
        for a, b in ((k, kk), (v, vv)):
            # half a step of the block's scale, or half of e4m3's last bit of the value (and of its smallest number)
            half = a.abs().max() / 127 / 2 if kv == torch.int8 else b.abs() * 2.0 ** -4 + a.abs().max() / 448 * 2.0 ** -10
            # (and five fp32 roundings of the value, which is up to 127 steps)
            assert ((a - b).abs() <= half * (1 + 2048 * F32)).all()
    for t in range(6):
        for layer in range(2):
            q = randn(t, 3, hkv * g, d)
            k, v = (randn(1000 + 10 * t + layer + 5 * i, 3, hkv, d, dtype=torch.bfloat16) for i in range(2))
            sel = c.new_sel()
            out = c.decode(layer, q, k, v, sel=sel)
            now = [n + t + 1 for n in lens]
            check(c, out, layer, q, now, sel)
            check(c, c.attend_all(layer, q), layer, q, now)
    write(c, [(0, 20), (137, 137), (46, 50)], 77, hkv, g, d, 1)
    q = randn(99, 3, hkv * g, d)
    check(c, c.attend_all(1, q), 1, q, [20, 137, 50])
    assert c.seq_len[1].tolist() == [20, 137, 50] and c.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
def test_far_into_a_large_cache(kv):
    # the codes of the last layer start behind 4 GB: every call gives what it gives in a small cache
    hkv, g, d, layers = 8, 4, 128, 34
    big, small = make_cache([131072], kv, layers=layers, hkv=hkv, g=g, d=d), make_cache([1024], kv, hkv=hkv, g=g, d=d)
    assert big.rows(layers - 1, 0, 0)[0] * BLOCK * d > 2 ** 32
    got = []
    for c, layer in ((big, layers - 1), (small, 0)):
        q = write(c, [(0, 700)], 1, hkv, g, d, layer)
        c.append(layer, *(randn(5 + i, 1, hkv, d, dtype=torch.bfloat16) for i in range(2)))
        write(c, [(701, 760)], 2, hkv, g, d, layer)
        q = randn(9, 1, hkv * g, d)
        sel = c.new_sel()
        out = c.decode(layer, q, *(randn(7 + i, 1, hkv, d, dtype=torch.bfloat16) for i in range(2)), sel=sel)
        got.append([out, sel, *c.read(layer, None, [761]), c.attend_all(layer, q), c.attend(layer, q, sel)])
        assert c.device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not big.k[:big.rows_per_layer].view(torch.int8).any()


def test_wide_batches():
    # 64 sequences of 32 heads: more units than CTAs, several heads of a sequence in one run, units without tokens
    lens = [(s * 37) % 90 for s in range(64)]
    c = make_cache([96] * 64, torch.int8, hkv=32, g=1, d=64)
    fill(c, 4, lens)
    q = randn(5, 64, 32, 64)
    check(c, c.attend_all(0, q), 0, q, lens)
    sel = selection(6, c, lens, 8)
    sel[::3, :, 4:] = -1
    check(c, c.attend(0, q, sel), 0, q, lens, sel)
    assert c.device_status() == 0


def test_queries_from_another_stream():
    # queries written on another stream are waited for by the caller's events, as for any call
    c = make_cache([2048], torch.float8_e4m3fn, hkv=4, d=128)
    fill(c, 3, [2000])
    side = torch.cuda.Stream()
    q = randn(1, 1, 16, 128)
    want = c.attend_all(0, q)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            x = q.clone()
            ready = side.record_event()
        torch.cuda.current_stream().wait_event(ready)
        assert torch.equal(c.attend_all(0, x), want)
    with pytest.raises(ValueError):
        c.attend_all(0, torch.stack([q, q], -1)[..., 0])


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d", [64, 128])
def test_what_stands_behind_the_tokens_is_never_read_as_such(kv, d):
    # codes of NaN behind the last token of a block, and rows of NaN behind the last block
    hkv, g, lens, caps = 2, 4, [1, 17, 40, 0, 100, 31], [64, 64, 64, 16, 128, 32]
    c = make_cache(caps, kv, hkv=hkv, g=g, d=d)
    write(c, [(0, n) for n in lens], 3, hkv, g, d)
    q = randn(4, len(lens), hkv * g, d)
    sel = selection(5, c, lens, 8)
    sel[4, :, 3:] = -1

    def results():
        return [c.attend_all(0, q), c.attend(0, q, sel), *c.read(0, None, lens, torch.float32)]

    want = results()
    for s, n in enumerate(lens):
        for h in range(hkv):
            r0, cap = c.rows(0, s, h)
            N = (n + BLOCK - 1) // BLOCK
            for t, x in ((c.k, c.kscale), (c.v, c.vscale)):
                t[r0:r0 + cap].view(torch.int8).view(-1, d)[n:] = 127
                x[r0 + N:r0 + cap] = float("nan")
            for t in (c.kbar, c.vbar, c.dbar):
                t[r0 + N:r0 + cap] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    # and tokens that come later make blocks of their own
    k, v = (randn(6 + i, len(lens), hkv, d, dtype=torch.bfloat16) for i in range(2))
    twin = make_cache(caps, torch.bfloat16, hkv=hkv, g=g, d=d)
    write(twin, [(0, n) for n in lens], 3, hkv, g, d)
    for x in (c, twin):
        x.append(0, k, v)
    check_stored(c, twin, [n + 1 for n in lens])
    assert c.attend_all(0, q).isfinite().all()


def test_a_sequence_copied_by_the_caller():
    # rows, summaries and length of one sequence into another that held something else, its tail_len zeroed
    hkv, d, n = 2, 64, 37
    c = make_cache([64, 64], torch.float8_e4m3fn, hkv=hkv, d=d)
    write(c, [(0, n), (0, 41)], 3, hkv, 4, d)
    for h in range(hkv):
        a, b = c.rows(0, 0, h)[0], c.rows(0, 1, h)[0]
        for t in (c.k.view(torch.int8), c.v.view(torch.int8), c.kscale, c.vscale, c.kbar, c.vbar, c.dbar):
            t[b:b + 4] = t[a:a + 4]
    c.seq_len[0, 1] = n
    c.tail_len.view(2, hkv, 3)[1] = 0
    q = randn(4, 1, hkv * 4, d).expand(2, -1, -1).contiguous()
    out = c.attend_all(0, q)
    assert torch.equal(out[0], out[1])
    before = values(c)
    k, v = (randn(6 + i, 2, hkv, d, dtype=torch.bfloat16) for i in range(2))
    c.append(0, k, v)
    for h in range(hkv):
        r = c.rows(0, 1, h)[0] + n // BLOCK
        for x, codes, scale, y in zip(before, (c.k, c.v), (c.kscale, c.vscale), (k, v)):
            block = torch.zeros(BLOCK, d, device="cuda")
            block[:n % BLOCK] = x[r, :n % BLOCK].float().bfloat16().float()
            block[n % BLOCK] = y[1, h].float()
            want, s = quantised(block, c.kv_dtype)
            assert torch.equal(bits(codes[r]), bits(want)) and scale[r] == s
