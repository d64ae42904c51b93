"""Host-side checks of the calls on a cache in 8 bits that need no GPU."""
import ctypes

import pytest

import block_sparse_kv_summary_gb300 as P
from block_sparse_kv_summary_gb300 import compkv as C


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P.lib()


def config(**kw):
    base = dict(num_layers=2, batch=2, num_kv_heads=8, group_size=4, head_dim=128, r=4, budget_tokens=2048, max_tokens=4096)
    base.update(kw)
    return C.make_config(**base)


def test_null_context(lib):
    assert lib.compkv_read(None, 0, None, None, 0, None, None, None) == 1
    assert "context" in C.compkv_last_error()
    assert lib.compkv_attend_all(None, 0, None, 0, None, None) == 1


def test_scratch_of_a_cache_in_8_bits(lib):
    # that of a bf16 cache stays as it is; behind it stand a counter a unit and two parts of every CTA
    for kw in (dict(), dict(group_size=8), dict(head_dim=64), dict(batch=64)):
        c = config(**kw)
        more = C.compkv_scratch_bytes_kv8(c) - C.compkv_scratch_bytes(c)
        assert more >= c.batch * c.num_kv_heads * 4 + 2 * 152 * c.group_size * (c.head_dim + 2) * 4
        assert C.compkv_scratch_bytes_kv8(c) % 256 == 0
    assert C.compkv_scratch_bytes_kv8(config(group_size=3)) == 0 and "group_size" in C.compkv_last_error()


@pytest.mark.parametrize("bad,msg", [
    (dict(type=0), "kv8 type"), (dict(type=1), "kv8 type"), (dict(type=4), "kv8 type"),
    (dict(kscale=0), "kscale is NULL"), (dict(vscale=8), "vscale must be 16-byte aligned"),
    (dict(tail=0), "tail is NULL"), (dict(tail=24), "tail must be"), (dict(tail_len=0), "tail_len is NULL"),
    (dict(tail_len=258), "tail_len must be"),
])
def test_init_rejects_bad_buffers(lib, bad, msg):
    c = config()
    fields = dict(type=C.COMPKV_INT8, kscale=256, vscale=256, tail=256, tail_len=256)
    fields.update(bad)
    kv8 = C.compkv_kv8(*(fields[n] for n, _ in C.compkv_kv8._fields_))
    bufs = C.compkv_buffers(256, 256, 256, 256, 256, 256, 256, C.compkv_scratch_bytes_kv8(c))
    with pytest.raises(C.CompKVError, match=msg):
        C.compkv_init_kv8(c, bufs, kv8)


def test_init_wants_its_scratch_and_its_arguments(lib):
    c = config()
    kv8 = C.compkv_kv8(C.COMPKV_E4M3, 256, 256, 256, 256)
    with pytest.raises(C.CompKVError, match="scratch_bytes"):
        C.compkv_init_kv8(c, C.compkv_buffers(256, 256, 256, 256, 256, 256, 256, C.compkv_scratch_bytes(c)), kv8)
    ctx = ctypes.c_void_p()
    bufs = C.compkv_buffers(256, 256, 256, 256, 256, 256, 256, C.compkv_scratch_bytes_kv8(c))
    assert lib.compkv_init_kv8(ctypes.byref(c), ctypes.byref(bufs), None, ctypes.byref(ctx)) == 1
    assert "kv8 is NULL" in C.compkv_last_error() and not ctx.value
    with pytest.raises(C.CompKVError, match="group_size"):
        C.compkv_init_kv8(config(group_size=3), bufs, kv8)
