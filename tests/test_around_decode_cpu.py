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
