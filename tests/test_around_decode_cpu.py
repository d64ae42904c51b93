"""Host-side checks of the calls around the decode step that need no GPU."""
import pytest

import block_sparse_kv_summary_gb300 as P
from block_sparse_kv_summary_gb300 import compkv as C


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P.lib()


def test_null_context(lib):
    assert lib.compkv_rope(None, 0, None, None, None, None, None) == 1
    assert "context" in C.compkv_last_error()
    assert lib.compkv_prefill_qkv(None, 0, None, None, None, None, None) == 1
    assert lib.compkv_fork(None, 0, 1, 1, None, None, None, None) == 1
    assert lib.compkv_compact(None, 0, 1, 1, None, None, None, 1, None) == 1
    assert lib.compkv_attend_shared(None, 0, None, 0, None, None, None, None, 0, None) == 1


def test_shared_workspace_size(lib):
    def size(**kw):
        base = dict(num_layers=1, batch=2, num_kv_heads=8, group_size=4, head_dim=128, r=4, budget_tokens=2048, max_tokens=4096)
        base.update(kw)
        return C.compkv_attend_shared_bytes(C.make_config(**base))
    assert size() > 0
    assert size(batch=64) > size()
    assert size(group_size=3) == 0 and "group_size" in C.compkv_last_error()


@pytest.mark.parametrize("typecode", "bBhHiIlLqQ")
def test_host_lists_arrive_as_int32(typecode):
    # whatever holds the integers, the library reads int32
    from array import array
    import ctypes
    for x in (array(typecode, [3, 5, 7]), [3, 5, 7], (3, 5, 7), range(3, 8, 2)):
        a = C.ints(x)
        assert a.itemsize == ctypes.sizeof(ctypes.c_int) and len(a) == 3
        assert list((ctypes.c_int * 3).from_address(C._at(a))) == [3, 5, 7]
    same = array("i", [1, 2])
    assert C.ints(same) is same and C.ints(None) is None  # int32 already: no copy
    assert C.ints(bytes([3, 5, 7, 9])).tolist() == C.ints(bytearray([3, 5, 7, 9])).tolist() == [3, 5, 7, 9]


@pytest.mark.parametrize("bad", [("f", [1.0, 2.0]), ("d", [1.0]), ("q", [2 ** 31]), ("I", [2 ** 32 - 1])])
def test_host_lists_that_are_no_int32_are_refused(bad):
    from array import array
    with pytest.raises((TypeError, OverflowError)):
        C.ints(array(*bad))


def test_numpy_and_tensor_lists():
    import numpy as np
    import torch
    for x in (np.array([9, 50]), np.array([9, 0, 50, 0])[::2], np.array([9, 50], dtype=np.int16), torch.tensor([9, 50])):
        assert C.ints(x).tolist() == [9, 50]
    for x in (np.array([9.5]), torch.tensor([1.5]), "12"):
        with pytest.raises(TypeError):
            C.ints(x)
