"""K and V in 8 bits: selections whose rows are dealt to many CTAs, every form of the prefill, the binding's own calls."""
import pytest
import torch

from block_sparse_kv_summary_gb300 import compkv as C

from test_gpu_kv8 import BLOCK, KV8, _built, check, check_stored, fill, make_cache, randn, selection, table  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selections over many CTAs
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g,r,K,lens", [
    # a short row of stages, padded: 3, 4 and 8 CTAs a unit, each with its share of the stream's records
    (128, 1, 4, 4, 33, [3000]),
    (64, 2, 8, 4, 64, [5003, 2049]),
    (128, 2, 1, 64, 128, [9001]),
    (64, 1, 1, 1, 128, [7777, 600]),
    # runs that cut units at odd places, several units a run, rows of a few blocks and of none between long ones
    (128, 8, 4, 4, 128, [4500, 2100, 0, 2049, 17, 3333, 2500, 4100]),
    (64, 8, 8, 16, 64, [1100, 5, 2000, 0, 1030, 1500, 3001, 700, 1200, 40, 2222, 1025]),
    (128, 4, 8, 128, 65, [1041, 2300, 1500, 16, 0, 1999, 3100, 1100, 2600, 1042]),
])
def test_attend_a_selection_over_many_ctas(kv, d, hkv, g, r, K, lens):
    c = make_cache([max(BLOCK, (n + 15) // 16 * 16) for n in lens], kv, hkv=hkv, g=g, d=d, r=r, budget=BLOCK * K)
    fill(c, 40, lens)
    q = randn(41, len(lens), hkv * g, d)
    full = selection(5, c, lens, K)
    part = full.clone()
    part[0, 0, 3:] = -1              # fewer than the budget: most CTAs of the unit have nothing but records
    part[-1, hkv - 1, K // 2 + 1:] = -1
    part[0, hkv - 1] = -1 if hkv > 1 else part[0, hkv - 1]
    for sel in (full, part):
        out = c.attend(0, q, sel)
        check(c, out, 0, q, lens, sel)
        for _ in range(3):
            assert torch.equal(c.attend(0, q, sel), out)
    assert c.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g,r,K,lens", [(128, 2, 4, 4, 128, [5000, 2050]), (64, 4, 1, 4, 33, [2000, 527, 0, 528, 529, 1600]),
                                              (128, 8, 8, 16, 64, [1500, 1023, 1024, 2100, 3000])])
def test_decode_over_many_ctas(kv, d, hkv, g, r, K, lens):
    # the selection is that of the same tokens in bf16; some rows fit the budget, one just no longer does
    caps = [(n + 15) // 16 * 16 + 32 for n in lens]
    c8, c16 = (make_cache(caps, t, hkv=hkv, g=g, d=d, r=r, budget=BLOCK * K) for t in (kv, torch.bfloat16))
    for c in (c8, c16):
        for a in range(0, max(lens), 2500):  # (the table of angles has 4096 rows)
            span = [(min(n, a), min(n, a + 2500)) for n in lens]
            qkv = randn(a + 3, sum(y - x for x, y in span), (g + 2) * hkv * d, dtype=torch.bfloat16)
            c.prefill_qkv(0, qkv, [y - x for x, y in span], table(8192, d), starts=[x for x, _ in span])
    for t in range(3):
        q = randn(300 + t, len(lens), hkv * g, d)
        k, v = (randn(400 + 10 * t + i, len(lens), hkv, d, dtype=torch.bfloat16) for i in range(2))
        sel = c8.new_sel()
        out = c8.decode(0, q, k, v, sel=sel)
        lens = [n + 1 for n in lens]
        c16.append(0, k, v)
        assert torch.equal(sel, c16.score_select(0, q))
        check(c8, out, 0, q, lens, sel)
        assert torch.equal(c8.attend(0, q, sel), c8.attend(0, q, sel))
    assert c8.device_status() == 0


# ------------------------------------------------------------------ forms of the prefill
@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,g", [(64, 3, 2), (128, 2, 4)])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [1, 2])
def test_every_form_of_the_projection(kv, d, hkv, g, fp32, interleaved, rot):
    # fp32 and bf16 projections, both kinds of pairs, whole and partial rotation, with and without norms, positions of their
    # own, both types of q; chunks that begin inside blocks whose tokens come from the tail, and from codes
    caps, lens = [96, 64, 160], [0, 0, 0]
    c8, c16 = make_cache(caps, kv, hkv=hkv, g=g, d=d), make_cache(caps, torch.bfloat16, hkv=hkv, g=g, d=d)
    for i, counts in enumerate([[21, 1, 33], [9, 16, 50], [3, 0, 14], [40, 5, 1]]):
        rows = sum(counts)
        qkv = randn(7 + i, rows, (g + 2) * hkv * d, dtype=torch.float32 if fp32 else torch.bfloat16)
        kw = dict(starts=lens, interleaved=interleaved, q_dtype=torch.bfloat16 if i % 2 else torch.float32)
        if i != 1:
            kw.update(q_weight=1 + 0.1 * randn(1, d), k_weight=1 + 0.1 * randn(2, d), eps=1e-5)
        if i >= 2:
            kw.update(positions=torch.randint(0, 300, (rows,), device="cuda", dtype=torch.int32))
        tab = table(300, d // rot)
        a, b = (c.prefill_qkv(0, qkv, counts, tab, **kw) for c in (c8, c16))
        assert torch.equal(a, b)
        lens = [n + m for n, m in zip(lens, counts)]
        check_stored(c8, c16, lens)
    # back into a block that only its codes are left of: the bf16 cache takes over what they stand for
    cut = [5, 3, 37]
    for s, n in enumerate(cut):
        for h in range(hkv):
            r = c8.rows(0, s, h)[0] + n // BLOCK
            for t, codes, scale in ((c16.k, c8.k, c8.kscale), (c16.v, c8.v, c8.vscale)):
                t[r, :n % BLOCK] = (codes[r].float() * scale[r])[:n % BLOCK].bfloat16()
    c8.tail_len.zero_()
    counts = [30, 2, 70]
    qkv = randn(70, sum(counts), (g + 2) * hkv * d, dtype=torch.float32 if fp32 else torch.bfloat16)
    for c in (c8, c16):
        c.prefill_qkv(0, qkv, counts, table(300, d // rot), starts=cut, interleaved=interleaved)
    check_stored(c8, c16, [n + m for n, m in zip(cut, counts)])
    assert c8.device_status() == 0


@pytest.mark.parametrize("kv", KV8)
@pytest.mark.parametrize("d,hkv,tokens", [(64, 8, 9900), (128, 8, 5200), (64, 6, 10000), (64, 3, 20000), (128, 4, 20000)])
def test_several_heads_to_a_cta(kv, d, hkv, tokens):
    # enough blocks that a CTA of the prefill takes two to four heads, the last one of a row fewer; then chunks and tokens
    # that go on from the tails of all of them
    share = [tokens // 2 + 7, tokens // 4 + 5, 0, tokens - tokens // 2 - tokens // 4 - 12]
    caps = [(n + 15) // 16 * 16 + 160 for n in share]
    c8, c16 = make_cache(caps, kv, hkv=hkv, g=1, d=d), make_cache(caps, torch.bfloat16, hkv=hkv, g=1, d=d)
    first = [7, 20, 0, 33]
    tab = table(caps[0], d)

    def both(starts, counts, seed):
        qkv = randn(seed, sum(counts), 3 * hkv * d, dtype=torch.bfloat16)
        a, b = (c.prefill_qkv(0, qkv, counts, tab, starts=starts) for c in (c8, c16))
        assert torch.equal(a, b)

    both([0] * 4, first, 1)
    for seed in (2, 9):                                     # (on from what a small call left open; and the same again)
        both(first, [n - m for n, m in zip(share, first)], seed)
        check_stored(c8, c16, share)
    lens = share
    both(lens, [3, 20, 4, 50], 3)                           # (and from what a large one did)
    lens = [n + m for n, m in zip(lens, [3, 20, 4, 50])]
    check_stored(c8, c16, lens)
    for t in range(3):
        new = [randn(50 + 2 * t + i, 4, hkv, d, dtype=torch.bfloat16) * (1 + t) for i in range(2)]
        for c in (c8, c16):
            c.append(0, *new)
    check_stored(c8, c16, [n + 3 for n in lens])
    assert c8.device_status() == 0


# ------------------------------------------------------------------ the binding
def test_the_binding_s_calls():
    # the functions of the library's own names, on valid arguments: what the cache's methods give
    hkv, g, d, caps = 2, 4, 64, [64, 96]
    a, b = make_cache(caps, torch.int8, hkv=hkv, g=g, d=d), make_cache(caps, torch.int8, hkv=hkv, g=g, d=d)
    counts, starts = [20, 41], [0, 0]
    qkv = randn(1, sum(counts), (g + 2) * hkv * d, dtype=torch.bfloat16)
    tab = table(128, d)
    for _ in range(2):
        want = a.prefill_qkv(0, qkv, counts, tab, starts=starts)
        q = torch.empty_like(want)
        args = C.compkv_rope_args(qkv.data_ptr(), C.COMPKV_BF16, qkv.stride(0), tab.data_ptr(), 128, d, 0, None, None, 1e-6, None,
                                  C.COMPKV_F32)
        C.compkv_prefill_qkv(b.ctx, 0, args, starts if any(starts) else None, counts, q.data_ptr(), 0)
        assert torch.equal(q, want) and torch.equal(a.k, b.k) and torch.equal(a.vscale, b.vscale)
        starts = [20, 41]
    for starts in (None, [3, 17]):
        want = a.read(0, starts, [7, 30])
        k, v = torch.empty_like(want[0]), torch.empty_like(want[1])
        C.compkv_read(b.ctx, 0, starts, [7, 30], C.COMPKV_BF16, k.data_ptr(), v.data_ptr(), 0)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    q = randn(4, 2, hkv * g, d)
    out = torch.empty_like(q)
    C.compkv_attend_all(b.ctx, 0, q.data_ptr(), C.COMPKV_F32, out.data_ptr(), 0)
    assert torch.equal(out, a.attend_all(0, q)) and a.device_status() == 0 and b.device_status() == 0
