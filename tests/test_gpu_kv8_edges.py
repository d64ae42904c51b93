"""K and V in 8 bits at the edges of what the calls promise."""
import ctypes

import pytest
import torch

from block_sparse_kv_summary_gb300 import compkv as C
from block_sparse_kv_summary_gb300 import lib

from test_gpu_kv8 import (BLOCK, F32, KV8, MOST, _built, check, check_stored, fill, gen, make_cache, randn, selection,  # noqa: F401
                          values, write)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the tail
# What is done to a sequence, and where it stands then: a prefill from the place on where it stands ("p"), tokens one
# after another ("a"), a cut ("c").  Every write goes on from the block that the sequence ended in or from the one that its
# last prefill began inside, so all of it is quantised from tokens as they came.
TAIL = {
    # a call inside one block, tokens over the block's end, and back: by either call
    "short call": [("p", 20), ("p", 25), ("a", 33), ("c", 20), ("p", 24), ("a", 35), ("c", 20), ("a", 23)],
    # the same where the tokens go on for several blocks
    "short call, far": [("p", 7), ("p", 9), ("a", 70), ("c", 7), ("p", 50), ("c", 7), ("a", 12)],
    # a call over several blocks, taken back by tokens that go past its first block, and once more
    "long call": [("p", 40), ("p", 100), ("c", 40), ("a", 50), ("c", 40), ("p", 41), ("a", 66), ("c", 40), ("p", 90)],
    # into the block's front, and on from there
    "in front of the beginning": [("p", 40), ("p", 100), ("a", 115), ("c", 37), ("a", 52), ("c", 37), ("p", 38)],
    # a short call in the block that a long one ended in, then back to the short one
    "short behind long": [("p", 5), ("p", 75), ("p", 77), ("a", 99), ("c", 75), ("p", 120), ("c", 75), ("a", 81)],
    # calls of one token each, from a block's start and over its end
    "single tokens": [("p", 32), ("p", 33), ("p", 34), ("a", 51), ("c", 33), ("p", 34), ("p", 35), ("a", 36)],
}


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("name", list(TAIL))
def test_the_block_that_a_call_began_inside_is_kept(kv, name):
    hkv, d = 3, 64
    c8, c16 = make_cache([160], kv, hkv=hkv, d=d), make_cache([160], torch.bfloat16, hkv=hkv, d=d)
    at = 0
    for i, (op, to) in enumerate(TAIL[name]):
        if op == "p":
            for c in (c8, c16):
                write(c, [(at, to)], 1 + i, hkv, 4, d)
        elif op == "a":
            for t in range(at, to):
                # sizes go up and down, so that a block's scale does as well
                new = [randn(1000 * i + 10 * t + j, 1, hkv, d, dtype=torch.bfloat16) * (0.5 + t * (5 + j) % 7) for j in range(2)]
                for c in (c8, c16):
                    c.append(0, *new)
        else:
            for c in (c8, c16):
                c.seq_len.fill_(to)
        at = to
        if op != "c":
            check_stored(c8, c16, [at])
    assert c8.device_status() == 0


# ------------------------------------------------------------------ the range of values
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g", [(64, 2, 4), (128, 1, 8)])
def test_values_near_the_end_of_fp32(kv, d, hkv, g):
    # keys of ordinary size, values up to bf16's largest: what the call sums up stays within fp32 where the result does
    lens = [1, 17, 40, 300]
    caps = [16, 32, 48, 304]
    c = make_cache(caps, kv, hkv=hkv, g=g, d=d, budget=128)
    for seed, size, sparse in ((1, 2.0 ** 127, False), (2, 2.0 ** 112, True)):
        fill(c, seed, lens)
        c.vscale.mul_(size / MOST[kv] / c.vscale.max())
        v = values(c)[1]
        assert size / 2 < v.abs().max() < size * 1.01
        for s, n in enumerate(lens):
            for h in range(hkv):
                r0, _ = c.rows(0, s, h)
                for b in range((n + 15) // 16):
                    c.vbar[r0 + b] = v[r0 + b, :n - 16 * b].mean(0)
        for dtype in (torch.float32, torch.bfloat16):
            q = randn(seed + 7, len(lens), hkv * g, d, dtype=dtype)
            out = c.attend_all(0, q)
            assert out.isfinite().all()
            check(c, out, 0, q, lens)
        if sparse:  # (with Mean compensation the sums of a row's mean values are formed first, at their own size)
            q = randn(seed + 9, len(lens), hkv * g, d)
            sel = selection(3, c, lens, 8)
            out = c.attend(0, q, sel)
            assert out.isfinite().all()
            check(c, out, 0, q, lens, sel)


@pytest.mark.parametrize("kv", KV8)
def test_values_near_the_least(kv):
    c = make_cache([48], kv, hkv=1, g=4, d=64)
    fill(c, 5, [40])
    c.vscale.mul_(2.0 ** -80 / MOST[kv] / c.vscale.max())
    q = randn(6, 1, 4, 64)
    check(c, c.attend_all(0, q), 0, q, [40])


# ------------------------------------------------------------------ channels of very different size
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("sparse", [False, True])
def test_one_channel_far_wider_in_the_keys(kv, sparse):
    # a channel that the queries do not look at takes the whole range of the codes; those that they look at, all with one
    # sign, are codes of one unit
    d, g, n = 128, 4, 64
    c = make_cache([n], kv, hkv=1, g=g, d=d, budget=128)
    fill(c, 1, [n], wide=False)
    k = torch.randint(0, 2, c.k.shape, device="cuda", generator=gen(3)) * 2.0 - 1
    k[..., 3] = 127.0
    c.k.copy_(k.to(kv))
    c.kscale.fill_(8.0)
    q = randn(2, 1, g, d).abs()
    q[..., 3] = 0
    sel = torch.tensor([[[0, 1, 2, 3, -1, -1, -1, -1]]], dtype=torch.int32, device="cuda")
    out = c.attend(0, q, sel) if sparse else c.attend_all(0, q)
    kk, vv = values(c)
    z = q[0].double() @ kk.view(n, d).T / d ** 0.5
    p = torch.exp(z - z.amax(-1, keepdim=True))
    want = p @ vv.view(n, d) / p.sum(-1, keepdim=True)
    # Relative error of a weight: the two parts of a query's coordinate
    # (2^-23), eight products in a row (2^-22 of the sum each, as they truncate), three factors and the distance from the
    # reference (2^-24 each of up to |z| + 20 in log2 units, times log 2), the exponential and its two parts (2^-21); sums of
    # 64 tokens, the block's products (three steps of 2^-22) and the join of up to 12 parts add 64 + 12 + 40 roundings.
    size = 8 * q.sum(-1).max().item() / d ** 0.5
    eps = (8 * 4 + 2) * F32 * size + 5 * F32 * (z.abs().max().item() + 20) + 8 * F32 + 116 * F32
    tol = 2 * eps * (p @ vv.view(n, d).abs() / p.sum(-1, keepdim=True) + want.abs())
    assert ((out[0].double() - want).abs() <= tol).all(), ((out[0].double() - want).abs() / tol).max()


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d", [64, 128])
def test_one_channel_far_wider_in_the_values(kv, d):
    # one block, logits of one product each, values of one unit beside a channel of the whole range
    g, n = 4, 16
    c = make_cache([n], kv, hkv=1, g=g, d=d)
    fill(c, 1, [n], wide=False)
    c.k.zero_()
    c.k[0, :, 0] = torch.arange(-8, 8, device="cuda").to(kv)
    c.kscale.fill_(0.25)
    v = torch.randint(0, 2, (1, n, d), device="cuda", generator=gen(4)) * 2.0 - 1
    v[..., 5] = 127.0
    c.v.copy_(v.to(kv))
    c.vscale.fill_(0.3)
    q = torch.zeros(1, g, d, device="cuda")
    q[0, :, 0] = torch.tensor([1.0, -1.7, 3.1, 0.3], device="cuda")
    out = c.attend_all(0, q)
    kk, vv = values(c)
    z = q[0].double() @ kk[0].T / d ** 0.5
    p = torch.exp(z - z.amax(-1, keepdim=True))
    want = p @ vv[0] / p.sum(-1, keepdim=True)
    # A logit (below 1) has five roundings of 2^-24; its distance from the reference, below 16 in log2 units, one of 2^-24
    # of that; the exponential 2^-22, the weight's parts 2^-23; sums of 16 tokens 16 roundings, the block's products three
    # truncations of 2^-22, joins and the division some 14 more.
    eps = (5 + 16 + 4 + 2 + 16 + 12 + 14) * F32
    tol = 2 * eps * (p @ vv[0].abs() / p.sum(-1, keepdim=True) + want.abs())
    assert ((out[0].double() - want).abs() <= tol).all(), ((out[0].double() - want).abs() / tol).max()


# ------------------------------------------------------------------ a wait that runs out
def stages_of(lens, hkv, warps, sel_blocks=None):
    """(unit of every stage, stages of a run): the attention's row of stages, where it is not a short one."""
    units = []
    for s, n in enumerate(lens):
        blocks = (n + BLOCK - 1) // BLOCK
        st = ((blocks if sel_blocks is None else min(blocks, sel_blocks)) + 1) // 2
        units += [(s, h) for h in range(hkv) for _ in range(st)]
    ctas = min(160, torch.cuda.get_device_properties(0).multi_processor_count)
    return units, (len(units) + ctas - 1) // ctas


def lose(c, stage):
    lib().compkv_internal_lose_stage(ctypes.c_void_p(c.ctx), stage)


@pytest.mark.parametrize("kv", KV8)
def test_a_copy_that_never_comes_is_reported(kv):
    # long and short sequences in turn, several heads a run: behind the stage that never comes, its warp's ring still names
    # blocks that the next, shorter sequence does not have.  The call ends, says so, and every unit that has nothing of that
    # warp's stages is what it is anyway; so is everything in the next call.
    hkv, warps, lens = 32, 8, [128, 1] * 32
    c = make_cache([max(BLOCK, n) for n in lens], kv, hkv=hkv, g=1, d=128, budget=128)
    fill(c, 1, lens)
    q = randn(2, len(lens), hkv, 128)
    sel = selection(3, c, lens, 8)
    units, per = stages_of(lens, hkv, warps, 8)
    assert per > 2 * warps  # (then every run has `per` stages)
    run = next(r for r in range(len(units) // per) if units[r * per][0] % 2 == 0 and units[(r + 1) * per - 1][0] != units[r * per][0])
    mine = [units[i] for i in range(run * per, (run + 1) * per, warps)]
    assert len(mine) > 3 and mine[0][0] % 2 == 0 and mine[-1][0] == mine[0][0] + 1
    want = c.attend(0, q, sel)
    lose(c, run * per)
    out = c.attend(0, q, sel)
    lose(c, -1)
    assert c.device_status() == 5 and "sequence %d, head %d, site 71" % mine[0] in C.compkv_last_error()
    other = torch.ones(len(lens), hkv, dtype=torch.bool, device="cuda")
    for s, h in mine:
        other[s, h] = False
    assert torch.equal(out[other], want[other])
    assert torch.equal(c.attend(0, q, sel), want) and c.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d", [64, 128])
def test_a_copy_that_never_comes_in_a_dense_call(kv, d):
    # one unit over many CTAs: the parts of all of them are still joined and the counters end at zero
    c = make_cache([4096, 64], kv, hkv=2, g=4, d=d)
    fill(c, 1, [4000, 50])
    q = randn(2, 2, 8, d)
    want = c.attend_all(0, q)
    lose(c, 40)
    out = c.attend_all(0, q)
    lose(c, -1)
    assert c.device_status() == 5 and "sequence 0, head 0" in C.compkv_last_error()
    assert torch.equal(out[0, 4:], want[0, 4:]) and torch.equal(out[1], want[1])
    for _ in range(2):
        assert torch.equal(c.attend_all(0, q), want)
    assert c.device_status() == 0
