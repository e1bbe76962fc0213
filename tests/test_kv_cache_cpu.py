"""What KVCache hands to the library, on tensors that stand in for CUDA ones: no GPU."""
import ctypes

import pytest
import torch

from tests.test_attention_cpu import _problem, misa  # noqa: F401  (the fixture that builds the library)


class _OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)


def _cuda_like(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnGpu)


@pytest.mark.parametrize("table", [torch.zeros(2, 0, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)[:, :0],
                                   torch.zeros(0, 5, dtype=torch.int32)])
def test_a_page_table_without_entries_stays_a_paged_cache(misa, table):
    """An empty tensor's address is NULL, which the library reads as a packed cache."""
    k = _cuda_like(4, 16, 2, 128)
    cache = misa.KVCache(k, _cuda_like(4, 16, 2, 128), table)
    assert cache.c.page_table, "the library would take this cache for a packed one"
    assert cache.c.pages_per_seq == table.shape[1] and cache.c.page_table_stride >= table.shape[1]
    assert misa.lib.misa_attention_workspace_size(ctypes.byref(_problem(misa)), ctypes.byref(cache.c), 8, 0, None) > 0


def test_a_packed_cache_has_no_page_table(misa):
    assert not misa.KVCache(_cuda_like(40, 2, 128)).c.page_table


def test_strides_that_nothing_is_multiplied_by_may_differ(misa):
    """One head: its stride is whatever the view it comes from had."""
    k = _cuda_like(4, 16, 1, 128)
    v = _cuda_like(4, 1, 16, 128).transpose(1, 2)
    assert k.stride() != v.stride()
    c = misa.KVCache(k, v, torch.zeros(2, 5, dtype=torch.int32)).c
    assert (c.page_stride, c.token_stride) == (16 * 128, 128)
    for bad in (_cuda_like(4, 16, 2, 128), _cuda_like(4, 16, 1, 136)[..., :128], _cuda_like(8, 16, 1, 128)[::2]):
        with pytest.raises(ValueError, match="strides"):
            misa.KVCache(k, bad, torch.zeros(2, 5, dtype=torch.int32))
