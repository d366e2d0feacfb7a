"""Host side of the block-sparse calls without a GPU: limits, a process without
a device, and the device that a workspace is sized for (CPU only)."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def without_device(code):
    """Run code in a process that sees no GPU, so that no launch can happen."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    head = f"""
        import ctypes, sys
        sys.path.insert(0, {ROOT!r})
        import paged_fp8_kv_02_gb300 as pf
        from paged_fp8_kv_02_gb300 import _build
        _build.build_pfkv()
        lib = pf.load(build_if_missing=False)
        fake = ctypes.c_void_p(0x10000)
        i64 = ctypes.c_int64
    """
    return subprocess.run([sys.executable, "-c", textwrap.dedent(head) + textwrap.dedent(code)], env=env, cwd=ROOT,
                          capture_output=True, text=True, timeout=600)


SELECT = """
    def select(Hkv, pages, maxp=9000):
        return lib.pfkv_select_pages(fake, fake, fake, fake, None, fake, maxp, fake, 2, Hkv, Hkv, 128, 16, i64(pages), 4, 1,
                                     1, fake, 1 << 30, None, None)
"""


@pytest.mark.parametrize("maxp", [8, 9000])
def test_select_without_a_device_is_an_error(maxp):
    r = without_device(SELECT + f"""
    rc = select(2, 64, {maxp})
    print(rc, lib.pfkv_last_error().decode())
    """)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert r.stdout.startswith("-3 select_pages"), r.stdout


def test_the_other_calls_without_a_device_are_errors():
    r = without_device("""
    print(lib.pfkv_kv_append_fp8_block(fake, fake, fake, fake, fake, fake, fake, 8, fake, fake, 2, 4, 2, 2, 128, 16,
                                       i64(64), None))
    print(lib.pfkv_page_key_bounds(fake, fake, fake, fake, 8, fake, fake, 2, 2, 2, 128, 16, i64(64), None))
    print(lib.pfkv_paged_sparse_decode_attn(fake, fake, fake, fake, 3, fake, fake, fake, 4, fake, 8, fake, 2, 16, 2, 128,
                                            16, i64(64), 0.1, None, None, None))
    for maxp in (8, 9000):
        print(lib.pfkv_paged_decode_attn_scaled(fake, fake, fake, fake, 3, fake, fake, fake, maxp, fake, 2, 16, 2, 128, 16,
                                                i64(64), 0.1, 0, fake, 1 << 30, None, None))
    """)
    assert r.returncode == 0 and r.stdout.split() == ["-3"] * 5, (r.returncode, r.stdout, r.stderr)


def test_select_takes_every_pool_below_two_to_the_31_pairs():
    """Up to 2^31 - 1 (page, KV head) pairs, also where the heads do not divide
    2^31; -3 is the missing device."""
    r = without_device(SELECT + """
    for heads in (1, 2, 3, 5, 7, 8, 48):
        most = (2 ** 31 - 1) // heads
        print(select(heads, most), select(heads, most + 1))
    """)
    assert r.returncode == 0 and r.stdout.splitlines() == ["-3 -2"] * 7, (r.returncode, r.stdout, r.stderr)


class FakeTensor:
    """Shape, type and place of a tensor on a device that is not there."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self._device = tuple(shape), dtype, device
        self.device = f"cuda:{device}"

    def get_device(self):
        return self._device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


@pytest.mark.parametrize("current", [0, 1])
def test_select_sizes_its_workspace_on_the_tensors_device(monkeypatch, current):
    """A device with other SMs than the current one needs another workspace."""
    import contextlib

    import torch

    import paged_fp8_kv_02_gb300 as pf
    state = {"device": current}
    calls = []

    @contextlib.contextmanager
    def device(d):
        before, state["device"] = state["device"], d
        yield
        state["device"] = before

    class Lib:
        @staticmethod
        def pfkv_select_pages_workspace_size(*args):
            calls.append(("size", state["device"], args))
            return 512 << state["device"]

        @staticmethod
        def pfkv_select_pages(*args):
            calls.append(("call", state["device"], args))
            return 0

    monkeypatch.setattr(pf, "_lib", Lib)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 77 + d, raising=False)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: FakeTensor((n,), dtype, int(device[5:])))
    T = lambda dt, *s: FakeTensor(s, dt, 1)
    ws = pf.select_pages(T(torch.int32, 2, 4, 8), T(torch.bfloat16, 2, 16, 128), T(torch.int8, 9, 4, 2, 128),
                         T(torch.float32, 9, 4), T(torch.int32, 2, 9000), T(torch.int32, 2), 16)
    assert [c[:2] for c in calls] == [("size", 1), ("call", 1)] and state["device"] == current
    assert ws.numel() == 1024 and calls[0][2] == (2, 4, 9000) and calls[1][2][-1] == 78 and 1024 in calls[1][2]


def test_counts_beyond_32_bits_are_not_cut(monkeypatch):
    """A bound on the new tokens may be as large as one likes; other counts that
    do not fit are refused.  ctypes alone would pass their low bits."""
    import torch

    import paged_fp8_kv_02_gb300 as pf
    calls = {}

    class Lib:
        @staticmethod
        def pfkv_kv_append_fp8_block(*args):
            calls["append"] = args
            return 0

        @staticmethod
        def pfkv_page_key_bounds(*args):
            calls["bounds"] = args
            return 0

        @staticmethod
        def pfkv_select_pages(*args):
            calls["select"] = args
            return 0

    monkeypatch.setattr(pf, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    T = lambda dt, *s: FakeTensor(s, dt, 0)
    x, cache, scales = T(torch.bfloat16, 5, 2, 128), T(torch.uint8, 9, 2, 16, 128), T(torch.float32, 9, 2)
    bt, ctx, start = T(torch.int32, 3, 7), T(torch.int32, 3), T(torch.int32, 4)
    bnd = T(torch.int8, 9, 2, 2, 128)
    for given, passed in ((5, 5), (0, 0), (-3, -3), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1),
                          (2 ** 64 + 1, 2 ** 31 - 1)):
        pf.kv_append_fp8_block(x, x, cache, cache, scales, scales, bt, ctx, start, given)
        pf.page_key_bounds(bnd, scales, cache, bt, ctx, start, given)
        assert calls["append"][12] == passed and calls["bounds"][8] == passed
    select = lambda **kw: pf.select_pages(T(torch.int32, 3, 2, 4), T(torch.bfloat16, 3, 8, 128), bnd, scales, bt, ctx,
                                          **{"page_size": 16, "workspace": T(torch.uint8, 512), **kw})
    select()
    assert calls["select"][12] == 16
    for name in ("page_size", "sink_pages", "recent_pages"):
        with pytest.raises(ValueError, match=name):
            select(**{name: 2 ** 32 + 1})
    with pytest.raises(ValueError, match="max_new_len"):
        pf.page_key_bounds(bnd, scales, cache, bt, ctx, start, -2 ** 32)
