"""Numerics of the attention over a shared prefix: the bits that each type keeps, infinities and NaN among a
sequence's tokens, and logits that rise and jump while a piece of a long item is walked."""
import math

import pytest
import torch

from test_gpu_around_decode import (BF16, F32, _built, check_shared, make_cache, randn, shared64,  # noqa: F401
                                    shared_cache)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bits
def test_bf16_weights_and_their_sum_are_the_same():
    # 99 of 100 keys share a weight of which rounding takes or adds up to 2^-8, and all values are alike: the weights' sum
    # must be that of the rounded ones for the value to come back (sums are off by less than 100 F32, the rounding of
    # the result is exact)
    d, n, batch, hkv, g = 64, 100, 64, 2, 4
    c = make_cache([112] * batch, hkv=hkv, g=g, d=d, fill=0.0)
    q = torch.zeros(batch, hkv * g, d, device="cuda")
    q[..., 0] = torch.linspace(0, 40, batch * hkv * g, device="cuda").view(batch, hkv * g)
    for s in range(batch):
        for h in range(hkv):
            kv, vv = c.token_view(0, s, h)
            kv[n - 1, 0] = 1.0
            vv[:n] = torch.linspace(-3, 3, d, device="cuda")
    c.seq_len.fill_(n)
    want = c.token_view(0, 0, 0)[1][0]
    out = c.attend_shared(0, q.bfloat16(), [-1] * batch, [0] * batch)
    assert c.device_status() == 0
    assert torch.equal(out, want.expand_as(out))


def two_keys(z_lo, z_hi, d=64, batch=64, hkv=2, g=4):
    """Two tokens a sequence: key e_0 and key 0, so that the first one's logit is q_0 / sqrt(d) to the last bit."""
    c = make_cache([16] * batch, hkv=hkv, g=g, d=d, fill=0.0)
    u = torch.rand(batch, hkv * g, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    q = torch.zeros(batch, hkv * g, d, device="cuda")
    q[..., 0] = (z_lo + (z_hi - z_lo) * u) * math.sqrt(d)
    for s in range(batch):
        for h in range(hkv):
            kv, vv = c.token_view(0, s, h)
            kv[0, 0] = 1.0
            vv[0, :d // 2] = 1.0   # first half of the coordinates: the first key's share
            vv[1, d // 2:] = 1.0   # second half: the other's
    c.seq_len.fill_(2)
    return c, q


def test_fp32_queries_and_weights_keep_24_bits():
    # z = q_0 / 8 in [1, 3]; in powers of two x = z log2(e) <= 4.33.  The scores are exact: one product a part, and
    # parts that add up to a value of 24 bits.  One weight is 1 up to the rounding of its argument, the other 2^-x: an
    # argument is off by two roundings of x (the constant, the reference), 2 x ln 2 F32 of the weight, and the power by
    # 2 ulp (4 F32) each.
    c, q = two_keys(1.0, 3.0)
    out = c.attend_shared(0, q, [-1] * 64, [0] * 64).double()
    assert c.device_status() == 0
    share = torch.sigmoid(q[..., 0].double() / 8)[..., None]
    ratio = (2 * 4.33 * math.log(2) + 2 * 4) * F32
    # the sum's, the product's (truncated: 2 F32) and the quotient's roundings
    rest = 4 * F32
    first, second = out[..., :32], out[..., 32:]
    # a query of 16 bits is off by up to 2^-18 z / share of the ratio, ten times this
    assert ((first - share).abs() <= share * ((1 - share) * ratio + rest)).all()
    # a weight of 16 bits is off by up to 2^-18 = 64 F32, four times this
    assert ((second - (1 - share)).abs() <= (1 - share) * (share * ratio + rest)).all()


def test_fp32_sums_of_a_long_prefix_lose_nothing():
    # values of 1 behind 128K keys: the result is the weights' sum over itself
    n, hkv, g, d = 131072, 8, 4, 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = make_cache([n, 16], hkv=hkv, g=g, d=d)
    c.k.copy_(randn(1, *c.k.shape))
    c.v.fill_(1.0)
    c.seq_len[0] = torch.tensor([n, 3], dtype=torch.int32)
    out = c.attend_shared(0, randn(2, 2, hkv * g, d), [0, 0], [n, 0])
    tiles = n // 128 * hkv // sms + 2   # of a CTA at most, and as many additions; pieces of a head:
    pieces = sms // hkv + 4
    # denominator: 10 roundings in a thread's 32 keys, one a tile, 3 across threads; numerator: 8 truncations (2 F32
    # each) of a tile's last part, the earlier parts' a 2^-8 of that, one rounding a tile; joining: two a piece for each
    bound = (10 + tiles + 3 + 17 + tiles + 4 * pieces + 1) * F32
    assert c.device_status() == 0
    assert (out.double() - 1).abs().max().item() <= bound


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_the_same_call_gives_the_same_bits(dtype, d):
    # sums are dealt and joined by a plan of the lengths alone, whatever runs first and whatever stood in the workspace
    hkv, g, batch = 4, 4, 40
    lens = [9000] + [(s * 53) % 700 for s in range(1, batch)]
    c = shared_cache([9008] + [704] * (batch - 1), lens, hkv, g, d)
    q = (2 * randn(5, batch, hkv * g, d)).to(dtype)
    plen = [8999] + [0] * (batch - 1)
    want = c.attend_shared(0, q, [0] * batch, plen).clone()
    for i in range(20):
        c.shared_workspace().fill_(255 * (i & 1))
        c.attend_shared(0, randn(i, batch, hkv * g, d).to(dtype), [-1] * batch, plen)
        assert torch.equal(c.attend_shared(0, q, [0] * batch, plen), want)
    assert c.device_status() == 0


# ------------------------------------------------------------------ infinities and NaN
def plain64(k, v, q):
    """Softmax attention of one head by the definition, products one by one: q [g, d], k, v [n, d] -> (out, sum p |v|)."""
    k, v, q = k.double(), v.double(), q.double()
    z = (q[:, None] * k[None]).sum(-1) / math.sqrt(q.shape[-1])
    w = (z - z.amax(-1, keepdim=True)).exp()
    w = w / w.sum(-1, keepdim=True)
    return (w[..., None] * v).sum(1), (w[..., None] * v.abs()).sum(1)


INF, NAN = math.inf, math.nan
# (which buffer, token slice, coordinate, value), on the holder's tokens; the prefix has 300 of its 330
PLANTS = {
    "a key of infinity": [("k", slice(77, 78), 5, INF)],
    "keys of both infinities": [("k", slice(3, 4), 5, INF), ("k", slice(290, 291), 9, -INF)],
    "an infinite key among own tokens": [("k", slice(310, 311), 5, -INF)],
    "infinite keys in the whole first tile": [("k", slice(0, 128), 5, INF)],
    "infinite keys everywhere": [("k", slice(0, 330), 5, INF)],
    "a value of infinity": [("v", slice(10, 11), 7, INF)],
    "values of both infinities": [("v", slice(10, 11), 7, INF), ("v", slice(200, 201), 7, -INF), ("v", slice(5, 6), 0, -INF)],
    "a value of NaN": [("v", slice(299, 300), 63, NAN)],
    "a key of NaN": [("k", slice(128, 129), 1, NAN)],
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("plant", PLANTS)
def test_infinities_and_nan_among_the_tokens(dtype, d, plant):
    hkv, g = 2, 4
    lens, plen = [330, 9, 0, 140], [300, 0, 0, 0]
    c = shared_cache([336, 16, 16, 144], lens, hkv, g, d)
    q = 1.5 * randn(5, 4, hkv * g, d)
    q[:, :, 5] = q[:, :, 5].abs() + 0.25
    q[:, 0::2, 5] *= -1   # every other query turns the other way
    q[1, 1, 5] = 0.0      # and one is orthogonal
    q = q.to(dtype)
    for name, at, x, value in PLANTS[plant]:
        for h in range(hkv):
            c.token_view(0, 0, h)[name == "v"][at, x] = value
    prefix_seq = [0, 0, 0, -1]
    out = c.attend_shared(0, q, prefix_seq, plen)
    assert c.device_status() == 0
    for s in range(4):
        for h in range(hkv):
            (kp, vp), (ko, vo) = c.token_view(0, 0, h), c.token_view(0, s, h)
            k, v = ko[:lens[s]], vo[:lens[s]]
            if s == 1 or s == 2:
                k, v = torch.cat([kp[:300], k]), torch.cat([vp[:300], v])
            want, mag = plain64(k, v, q[s, h * g:(h + 1) * g])
            got = out[s, h * g:(h + 1) * g].double()
            assert torch.equal(got.isnan(), want.isnan()), (s, h)
            inf = want.isinf()
            assert torch.equal(got[inf], want[inf]), (s, h)
            ok = want.isfinite()
            tol = 3e-5 * (mag + want.abs()) + (BF16 * (mag + want.abs()) if dtype == torch.bfloat16 else 0)
            assert ((got - want).abs() <= tol)[ok].all(), (s, h)
    if plant == "a key of infinity":  # half of the rows are finite
        assert out[1].isfinite().all(-1).sum().item() == 4
    if "value" in plant:
        assert out[1].isfinite().sum().item() > 0.9 * out[1].numel()
    assert out[3].isfinite().all()


def test_infinities_behind_a_long_prefix():
    # pieces of many tiles in many CTAs: a row whose first tiles have no weight at all, one with an infinite value
    n, hkv, g, d = 20000, 8, 1, 128
    c = shared_cache([20000, 16], [n, 2], hkv, g, d)
    q = randn(5, 2, hkv * g, d)
    q[..., 3], q[..., 4] = -1.0, 0.0
    for h in range(hkv):
        kv, vv = c.token_view(0, 0, h)
        kv[:9000, 3] = INF
        vv[15000, 2] = -INF
        vv[7000, 9] = 5.0
    out = c.attend_shared(0, q, [0, 0], [n, 0])
    for s in range(2):
        for h in range(hkv):
            (kp, vp), (ko, vo) = c.token_view(0, 0, h), c.token_view(0, 1, h)
            k, v = (kp, vp) if s == 0 else (torch.cat([kp, ko[:2]]), torch.cat([vp, vo[:2]]))
            want, mag = plain64(k, v, q[s, h:h + 1])
            got = out[s, h:h + 1].double()
            assert (got[:, 2] == -INF).all() and (want[:, 2] == -INF).all()
            got[:, 2] = want[:, 2] = mag[:, 2] = 0
            assert ((got - want).abs() <= 3e-5 * (mag + want.abs())).all()
    assert c.device_status() == 0


# ------------------------------------------------------------------ a reference that is raised on the way
def rising_cache(n, batch, hkv, g, d, own=16):
    """Keys whose logits, in powers of two, make the sum of a tile's 128 weights pass 2^30 now and then.

    Coordinate 0, tiles in fives: 0, three of 22.8 the last of which has one key at 30.4, 0.  Coordinates 1 and 2 the
    same in fours, and 30.4 higher from each four to the next.  Whatever stood before a jump keeps as much weight as
    the jump.  Coordinates from 8 on are random.  All scores are exact in fp32."""
    a0, a1 = (16.0, 14.875) if d == 128 else (11.3125, 10.5)
    c = make_cache([(n + 15) // 16 * 16] + [own] * (batch - 1), hkv=hkv, g=g, d=d, fill=float("nan"))
    tile = torch.arange(n, device="cuda") // 128
    at = torch.arange(n, device="cuda") % 128
    last = tile == tile[-1]
    for h in range(hkv):
        k = torch.zeros(n, d, device="cuda")
        k[:, 8:] = randn(h, n, d - 8)
        spot = at == torch.where(last, at[-1] // 2, (tile * 37 + 11 * h) % 128)  # the key of a tile that jumps
        k[:, 0] = torch.where((tile % 5 == 3) & spot | last & spot, 14.875, torch.where((tile % 5 >= 1) & (tile % 5 <= 3), 11.1875, 0.0))
        k[:, 1] = 16.0 * (tile // 4)
        k[:, 2] = torch.where((tile % 4 == 3) & spot | last & spot, 14.875, torch.where(tile % 4 >= 1, 11.1875, 0.0))
        kv, vv = c.token_view(0, 0, h)
        kv[:n], vv[:n] = k, randn(900 + h, n, d)
        for s in range(1, batch):
            kv, vv = c.token_view(0, s, h)
            kv[:own], vv[:own] = randn(100 * s + h, own, d), randn(5000 + 100 * s + h, own, d)
    lens = [n] + [own - s % 3 for s in range(1, batch)]
    c.seq_len[0] = torch.tensor(lens, dtype=torch.int32)
    q = torch.zeros(batch, hkv * g, d, device="cuda")
    kind = (torch.arange(batch, device="cuda")[:, None] * g + torch.arange(hkv * g, device="cuda")[None] % g) % 5
    q[..., 0] = a0 * ((kind == 0).float() - (kind == 3).float())  # jumps; the same downwards
    q[..., 1] = a1 * (kind == 1)
    q[..., 2] = a0 * (kind == 1)
    q[..., 8:] = 2 * randn(7, batch, hkv * g, d - 8) * ((kind == 2) | (kind == 4))[..., None]
    return c, q, lens


@pytest.mark.parametrize("dtype,batch", [(torch.float32, 16), (torch.float32, 40), (torch.bfloat16, 16), (torch.bfloat16, 40),
                                         (torch.bfloat16, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_logits_that_jump_in_the_middle_of_a_piece(dtype, batch, d):
    n, hkv, g = 32768 + 57, 8, 4
    c, q, lens = rising_cache(n, batch, hkv, g, d)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # a CTA's run of equal costs has this many tiles of one or two heads: pieces of at least four tiles everywhere
    assert (n // 128) * hkv // sms >= 12
    z = (q[0].double().view(hkv, g, d) @ torch.stack([c.token_view(0, 0, h)[0][:n].double() for h in range(hkv)]).transpose(1, 2))
    z = z[..., :n // 128 * 128].unflatten(-1, (-1, 128)) * (math.log2(math.e) / math.sqrt(d))
    # of the rows that jump, four tiles in a row: the reference of the first is passed by 2^30 in one of the others
    base = z[..., :-3, :].amax(-1)
    passed = [(torch.logsumexp((z[..., i:z.shape[-2] - 3 + i, :] - base[..., None]) * math.log(2), -1) / math.log(2) > 30) for i in (1, 2, 3)]
    assert (passed[0] | passed[1] | passed[2])[:, 1].float().mean().item() > 0.4
    q = q.to(dtype)
    got = c.attend_shared(0, q, [0] * batch, [n] + [0] * (batch - 1))
    assert c.device_status() == 0
    check_shared(got, *shared64(c, 0, q, [0] * batch, [n] + [0] * (batch - 1), lens))
