"""Copied and pickled host objects of the calls around the attention (CPU only)."""
import copy
import ctypes
import gc
import pickle

import pytest


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as pf
    from paged_fp8_kv_02_gb300 import _build
    _build.build_pfkv()
    return pf


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))], ids=["copy", "deepcopy", "pickle"])
def test_a_copied_rotary_passes_its_own_description(pf, how):
    """The address that a copy hands to a call is that of the description it
    holds, also when the original is gone and its memory used again."""
    first = pf.Rotary([1.0 / (1 + i) for i in range(64)], axes=[0, 1] * 32)
    want = bytes(first._struct)
    other = how(first)
    del first
    gc.collect()
    rest = [pf.Rotary([0.5] * 8, first=16) for _ in range(50)]
    assert other._ptr == ctypes.addressof(other._struct) and other.num_axes == 2
    assert ctypes.string_at(ctypes.addressof(other._struct), len(want)) == want
    assert len({r._ptr for r in rest} | {other._ptr}) == 51


def test_a_changed_copy_leaves_the_original(pf):
    first = pf.Rotary([1.0] * 8)
    other = copy.deepcopy(first)
    other._struct.turns[0] = 0
    assert first._struct.turns[0] != 0 and first._ptr != other._ptr


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, pickle.dumps], ids=["copy", "deepcopy", "pickle"])
def test_a_page_pool_is_not_copied(pf, how):
    """Two objects of one pool would both free it."""
    pool = pf.PagePool(4, 4)
    with pytest.raises(TypeError):
        how(pool)
    assert pool.num_free() == 4


def test_a_changed_list_of_tensors_changes_no_call(pf, monkeypatch):
    """copy_pages passes as many descriptions as were made, whatever is done to
    the list of tensors that keeps them alive."""
    import torch

    class Tensor:
        shape, dtype, nbytes, device = (9, 64), torch.uint8, 9 * 64, "cuda:0"

        def get_device(self):
            return 0

        def dim(self):
            return 2

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 0x10000

    class Pairs(Tensor):
        shape, dtype = (1, 2), torch.int32

    calls = []

    class Lib:
        def pfkv_copy_pages(self, *a):
            calls.append(a)
            return 0

    monkeypatch.setattr(pf, "_lib", Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    arrays = pf.PagedArrays([Tensor(), Tensor()])
    arrays.tensors.append(Tensor())
    pf.copy_pages(arrays, Pairs())
    assert calls[0][:2] == (ctypes.addressof(arrays._arrays), 2)
