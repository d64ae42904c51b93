"""K and V in 8 bits at the edges of what the calls promise."""
import pytest
import torch

from test_gpu_kv8 import KV8, MOST, _built, check, check_stored, fill, make_cache, randn, selection, values, write  # noqa: F401

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
