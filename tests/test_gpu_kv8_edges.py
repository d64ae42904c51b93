"""K and V in 8 bits at the edges of what the calls promise."""
import pytest
import torch

from test_gpu_kv8 import KV8, _built, check_stored, make_cache, randn, write  # noqa: F401

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
