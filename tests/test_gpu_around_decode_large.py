"""The calls around the decode step at sizes where their kernels take other paths: several KV heads to a CTA of the
prefill, copies of long runs and many work items, long lists; one block's summary from every call that forms it; and
calls at once on other streams and in graphs."""
import pytest
import torch

from test_gpu_around_decode import (BLOCK, _built, check_k, check_q, check_summaries, filled, heads_of, make_cache,  # noqa: F401
                                    randn, rope64, shared_cache, split_heads, state, table)

pytestmark = pytest.mark.gpu


def multiprocessors():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("hkv,g,d,r,heads,counts", [
    (8, 4, 128, 4, 4, [9000, 0, 1701, 37]),     # four heads to a CTA
    (5, 2, 64, 64, 4, [11000, 301, 0, 37]),     # four and one
    (3, 1, 128, 128, 2, [700, 12001, 0, 9]),    # two and one
    (3, 8, 64, 1, 3, [19995, 1, 16, 700]),      # all three
    (8, 1, 64, 16, 2, [5003, 0, 64, 900]),      # two of eight
])
def test_prefill_with_several_heads_to_a_cta(hkv, g, d, r, heads, counts):
    starts = [0, 5, 16, 77]
    caps = [(a + n + 31) // BLOCK * BLOCK for a, n in zip(starts, counts)]
    blocks = sum((a + n - 1) // BLOCK - a // BLOCK + 1 for a, n in zip(starts, counts) if n)
    # heads are halved from four until every multiprocessor has eight CTAs
    want = min(hkv, 4)
    while want > 1 and blocks * -(-hkv // want) < 8 * multiprocessors():
        want = (want + 1) // 2
    if multiprocessors() == 152:
        assert want == heads
    rot, w = d // 2, [1 + 0.2 * randn(x, d) for x in (2, 3)]
    one, many = (make_cache(caps, hkv=hkv, g=g, d=d, r=r) for _ in range(2))
    for c in (one, many):
        c.k.copy_(randn(1, *c.k.shape))
        c.v.copy_(randn(2, *c.v.shape))
    T = sum(counts)
    qkv, tab = randn(5, T, (g + 2) * hkv * d).bfloat16(), table(max(caps), rot)
    kw = dict(q_weight=w[0], k_weight=w[1], eps=1e-5)
    q = one.prefill_qkv(0, qkv, counts, tab, starts=starts, **kw)
    # the same in pieces of up to 500 tokens: one head to a CTA, which the small tests check against 64 bits
    at = 0
    for s, (a, n) in enumerate(zip(starts, counts)):
        for i in range(0, n, 500):
            m = min(500, n - i)
            part = many.prefill_qkv(0, qkv[at + i:at + i + m], [m * (x == s) for x in range(4)], tab, starts=[(a + i) * (x == s) for x in range(4)], **kw)
            assert torch.equal(part, q[at + i:at + i + m]), (s, i)
        at += n
    for x, y in zip(state(one), state(many)):
        assert torch.equal(x, y)
    assert one.device_status() == 0 and many.device_status() == 0
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).cuda()
    xq, xk, xv = split_heads(qkv, hkv, g, d)
    check_q(q, *rope64(xq, w[0], tab, pos, rot, False, 1e-5))
    k64 = rope64(xk, w[1], tab, pos, rot, False, 1e-5)[0]
    at = 0
    for s, (a, n) in enumerate(zip(starts, counts)):
        for h in range(hkv if n else 0):
            kv, vv = one.token_view(0, s, h)
            check_k(kv[a:a + n], k64[at:at + n, h])
            assert torch.equal(vv[a:a + n], xv[at:at + n, h])
            check_summaries(one, 0, s, h, {a // BLOCK, (a + n // 2) // BLOCK, (a + n - 1) // BLOCK}, a + n)
        at += n


# ------------------------------------------------------------------ copies
def expected_fork(c, old, pairs, layers):
    """Buffers after the copies (src, dst, tokens), but for the summaries of cut blocks, which are taken from c."""
    want = [t.clone() for t in old]
    for l in layers:
        for s, t, n in pairs:
            held = old[5][l, s].item()
            n = held if n < 0 else n
            want[5][l, t] = n
            for x, o in zip(want[:2], old[:2]):
                heads_of(c, x, l, t).flatten(1, 2)[:, :n] = heads_of(c, o, l, s).flatten(1, 2)[:, :n]
            whole = n // BLOCK + (n % BLOCK > 0 and n == held)
            for x, o in zip(want[2:5], old[2:5]):
                heads_of(c, x, l, t)[:, :whole] = heads_of(c, o, l, s)[:, :whole]
            if n % BLOCK and n < held:
                for h in range(c.Hkv):
                    check_summaries(c, l, t, h, [n // BLOCK], n)
                    for x, got in zip(want[2:5], (c.kbar, c.vbar, c.dbar)):
                        heads_of(c, x, l, t)[h, n // BLOCK] = heads_of(c, got, l, t)[h, n // BLOCK]
    return want


@pytest.mark.parametrize("d,r,hkv", [(128, 1, 8), (128, 128, 8), (64, 2, 5), (64, 64, 8), (128, 4, 3)])
def test_fork_of_long_sequences(d, r, hkv):
    # three sources of very different lengths; copies of one source end at different places: inside a run of 16 blocks,
    # at its end, inside a 32 KB stage, inside a block
    n0, n1 = 11211, 7001
    caps = [11216, 7008, 48, 11216, 11216, 11216, 11216, 7008, 7024, 16, 32]
    held = [n0, n1, 40] + [0] * 8
    c = filled(caps, held, hkv=hkv, d=d, r=r)
    pairs = [(0, 3, -1), (0, 4, 256 * 40), (1, 7, -1), (0, 5, 256 * 40 + 128 + 5), (2, 9, 16), (0, 6, 256 * 21 + 33), (1, 8, 6400 + 256 - 1),
             (2, 10, 31)]
    assert 2 * hkv * -(-n0 // 64) > 2 * multiprocessors()                                # items of 16 blocks
    assert 2 * hkv * (-(-n0 // 256) + -(-n1 // 256) + 1) > 2 * multiprocessors()         # more than one for a CTA
    old = state(c)
    c.fork(*zip(*pairs))
    torch.cuda.synchronize()
    assert c.device_status() == 0
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), expected_fork(c, old, pairs, range(2))):
        assert torch.equal(got, w)


@pytest.mark.parametrize("d,r,hkv", [(128, 4, 8), (64, 64, 3)])
def test_long_fork_beside_cuts_and_refused_pairs(d, r, hkv):
    # of one source: a whole copy, one that its destination has no room for, one of more than it holds; cuts beside them
    caps = [20480, 20480, 9008, 20480, 6400, 4096]
    held = [20001, 0, 0, 0, 6390, 4000]
    c = filled(caps, held, hkv=hkv, d=d, r=r)
    old = state(c)
    c.fork([0, 0, 0, 4, 5], [1, 2, 3, 4, 5], [-1, -1, 20002, 1234, 0])
    torch.cuda.synchronize()
    assert c.device_status() in (1, 3) and c.device_status() == 0
    want = expected_fork(c, old, [(0, 1, -1), (4, 4, 1234), (5, 5, 0)], range(2))
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), want):
        assert torch.equal(got, w)


# ------------------------------------------------------------------ long lists
def check_compact(c, old, choice, src, dst):
    """choice[l][pair][head] lists; buffers after the call against the moved blocks."""
    want = [t.clone() for t in old]
    for l, of in enumerate(choice):
        for i, heads in enumerate(of):
            held = old[5][l, src[i]].item()
            N = -(-held // BLOCK)
            n = len(heads[0]) * BLOCK - (N * BLOCK - held if heads[0] and heads[0][-1] == N - 1 else 0)
            want[5][l, dst[i]] = n
            for h, x in enumerate(heads):
                idx = torch.tensor(x, dtype=torch.long, device="cuda")
                for w, o in zip(want[:5], old[:5]):
                    a, b = heads_of(c, o, l, src[i])[h], heads_of(c, w, l, dst[i])[h]
                    if w.dim() == 3:
                        b.flatten(0, 1)[:n] = a[idx].flatten(0, 1)[:n]
                    else:
                        b[:len(x)] = a[idx]
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar, c.seq_len), want):
        assert torch.equal(got, w)


def random_lists(c, layers, sizes, g):
    """sizes[pair] = (kept, blocks of the source, with its last); a list of its own for each layer and head."""
    def pick(n, blocks, last):
        x = sorted(torch.randperm(blocks - 1, generator=g)[:n - last].tolist())
        return x + [blocks - 1] * last
    choice = [[[pick(*s) for _ in range(c.Hkv)] for s in sizes] for _ in range(layers)]
    m = max(s[0] for s in sizes)
    keep = torch.full((layers, len(sizes), c.Hkv, m), -1, dtype=torch.int32)
    for l in range(layers):
        for i in range(len(sizes)):
            for h in range(c.Hkv):
                keep[l, i, h, :sizes[i][0]] = torch.tensor(choice[l][i][h], dtype=torch.int32)
    return choice, keep.cuda()


@pytest.mark.parametrize("d,r,hkv,kept", [(128, 4, 8, 300), (64, 64, 8, 256), (64, 1, 8, 257), (128, 128, 3, 683)])
def test_long_lists_into_other_sequences(d, r, hkv, kept):
    # lists of 2048 entries a pair and below are checked where the blocks are moved, longer ones before
    caps = [16000, 12800, 16, 11200, 11200, 11200]
    c = filled(caps, [15991, 12800, 9, 0, 0, 0], hkv=hkv, d=d, r=r)
    choice, keep = random_lists(c, 2, [(kept, 1000, 1), (kept - 1, 800, 0), (1, 1, 1)], torch.Generator().manual_seed(kept))
    old = state(c)
    c.compact(keep, [0, 1, 2], [3, 4, 5])
    assert c.device_status() == 0
    check_compact(c, old, choice, [0, 1, 2], [3, 4, 5])


@pytest.mark.parametrize("d,r,hkv", [(64, 1, 2), (128, 64, 8)])
def test_pairs_in_place_and_others_in_one_call(d, r, hkv):
    c = filled([4000, 3200, 2000, 4000, 1600], [3991, 3200, 1777, 5, 0], hkv=hkv, d=d, r=r)
    src, dst = [0, 1, 2], [0, 4, 2]
    choice, keep = random_lists(c, 2, [(97, 250, 1), (33, 200, 0), (60, 112, 1)], torch.Generator().manual_seed(9))
    old = state(c)
    c.compact(keep, src, dst)
    assert c.device_status() == 0
    check_compact(c, old, choice, src, dst)


def test_a_bad_long_list_changes_nothing():
    c = filled([16000, 8000, 16000, 8000], [15991, 7999, 0, 3], layers=1, hkv=8)
    choice, keep = random_lists(c, 1, [(300, 1000, 1), (290, 500, 1)], torch.Generator().manual_seed(1))
    keep[0, 0, 7, 299] = 1000  # one behind the last block, in the last place of the last head
    old = state(c)
    c.compact(keep, [0, 1], [2, 3])
    assert c.device_status() == 6
    want = [t.clone() for t in old]
    assert torch.equal(c.seq_len, torch.tensor([[15991, 7999, 0, 289 * 16 + 15]], dtype=torch.int32, device="cuda"))
    for got, w in zip((c.k, c.v, c.kbar, c.vbar, c.dbar), want[:5]):
        assert torch.equal(heads_of(c, got, 0, 2), heads_of(c, w, 0, 2))


# ------------------------------------------------------------------ one summary
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("r", [1, 2, 16, 64])
def test_every_call_forms_the_same_summary(d, r):
    # tokens prefilled from the projection, prefilled in place, appended one by one (from the one-token rotation) and cut
    # back to: the same bits, complete blocks and the last one
    hkv, g, n = 2, 2, 37
    tab, w = table(64, d), 1 + 0.2 * randn(9, d)
    qkv = randn(4, n, (g + 2) * hkv * d).bfloat16()
    cs = [make_cache([64, 64], hkv=hkv, g=g, d=d, r=r) for _ in range(4)]
    a, b, e, f = cs
    q = a.prefill_qkv(0, qkv, [n, 0], tab, q_weight=w, k_weight=w)
    b.k.copy_(a.k)
    b.v.copy_(a.v)
    b.prefill(0, [n, 0])
    for i in range(n):
        rows = torch.stack([qkv[i], qkv[i]])
        qi, k, v = e.rope(0, rows, tab, q_weight=w, k_weight=w)
        assert torch.equal(qi[0], q[i])
        e.append(0, k, v)
    f.prefill_qkv(0, torch.cat([qkv, qkv[:9]]), [n + 9, 0], tab, q_weight=w, k_weight=w)
    f.fork([0], [1], [n])
    f.truncate([0], [n])
    for h in range(hkv):
        want = a.token_view(0, 0, h) + a.summary_view(0, 0, h)
        for c, s in ((b, 0), (e, 0), (e, 1), (f, 0), (f, 1)):
            got = c.token_view(0, s, h) + c.summary_view(0, s, h)
            for x, y in zip(got[:2], want[:2]):
                assert torch.equal(x[:n], y[:n])
            for x, y in zip(got[2:], want[2:]):
                assert torch.equal(x[:3], y[:3])
    assert all(c.device_status() == 0 for c in cs)


# ------------------------------------------------------------------ at once
def test_two_caches_on_two_streams_at_once():
    # each call of the attention takes every multiprocessor and waits for its own CTAs; two of them, and a third stream
    # with decode steps and copies, give what they give alone
    hkv, g, d, batch, n = 4, 4, 128, 8, 5000
    cs = [shared_cache([5008] + [304] * (batch - 1), [n] + [(s * 37) % 300 for s in range(1, batch)], hkv, g, d, seed=x) for x in (1, 50)]
    qs = [2 * randn(x, batch, hkv * g, d) for x in (8, 9)]
    plen = [n - 3] + [0] * (batch - 1)
    want = [c.attend_shared(0, q, [0] * batch, plen).clone() for c, q in zip(cs, qs)]
    busy, idle = (filled([4096, 4096], [3000, 0], layers=1, hkv=8, d=128) for _ in range(2))
    q, k, v = randn(1, 2, 32, 128), randn(2, 2, 8, 128).bfloat16(), randn(3, 2, 8, 128).bfloat16()

    def other(c):
        c.fork([0], [1])
        out = c.decode(0, q, k, v)
        c.truncate([0], [3000])
        return out
    alone = [other(idle) for _ in range(3)][-1].clone()
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(3)]
    outs, steps = [[], []], []
    for i in range(50):
        for j in range(2):
            with torch.cuda.stream(st[j]):
                outs[j].append(cs[j].attend_shared(0, qs[j], [0] * batch, plen))
        with torch.cuda.stream(st[2]):
            steps.append(other(busy))
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j]) for o in outs[j])
    assert all(torch.equal(o, alone) for o in steps)
    assert [c.device_status() for c in cs + [busy, idle]] == [0] * 4


def test_two_graphs_share_a_workspace_and_a_query_is_overwritten():
    hkv, g, d, lens = 2, 4, 64, [1500, 40, 0]
    c = shared_cache([1504, 48, 16], lens, hkv, g, d)
    plans = [([0, 0, 0], [1400, 0, 0]), ([-1, 0, -2], [700, 0, 0])]
    qs = [randn(x, 3, hkv * g, d) for x in (1, 2)]
    want = [c.attend_shared(0, q, *p, out=torch.zeros_like(q)).clone() for q, p in zip(qs, plans)]
    graphs, outs = [], [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for q, p, o in zip(qs, plans, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.attend_shared(0, q, *p, out=o)
    for i in range(6):
        for j in (0, 1) if i % 2 else (1, 0):
            outs[j].zero_()
            graphs[j].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    q = qs[0].clone()  # the result in the place of the queries
    assert torch.equal(c.attend_shared(0, q, *plans[0], out=q), want[0])
    assert c.device_status() == 0
