"""Host side of the rotary, copy and verify calls: what they refuse, before
anything is launched (CPU only: the calls that are in order fail for want of a
device, in a process that sees none)."""
import ctypes

import numpy as np
import pytest

from test_block_host import FakeTensor, without_device


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as pf
    from paged_fp8_kv_02_gb300 import _build
    _build.build_pfkv()
    return pf


CALLS = """
    NO, BAD, UNS = -3, -1, -2     # no device; a bad argument; one that is not supported
    big = 1 << 40
    rot = pf.Rotary([1.0] * 64)
    def embed(out=0x100000, os=1024, x=0x10000, xs=1024, pos=0x10000, r=rot._ptr, T=3, H=8, D=128):
        return lib.pfkv_rotary_embed(out, os, x, xs, pos, r, T, H, D, None)
    def append(qo=0x100000, qos=1024, q=0x10000, qs=1024, k=0x10000, ks=256, v=0x10000, vs=256, kc=0x10000, vc=0x10000,
               sl=0x10000, pos=0x10000, r=rot._ptr, T=3, Hq=8, H=2, D=128, P=16, pages=5, gran=0, sk=0x10000, sv=0x10000):
        return lib.pfkv_rotary_append_fp8(qo, qos, q, qs, k, ks, v, vs, kc, vc, sl, pos, r, T, Hq, H, D, P, i64(pages), gran,
                                          sk, sv, None)
    def verify(nx=0x10000, acc=0x10000, p=0x10000, ps=1000, q=0x10000, qs=1000, dt=0, tok=0x10000, u=0x10000, st=0x10000, B=2,
               T=5, V=1000, ctx=None, rs=None):
        return lib.pfkv_verify_drafts(nx, acc, p, ps, q, qs, dt, tok, u, st, B, T, V, ctx, rs, None)
    def copy(arrays=((0x10000, 4096, 4096),), n=None, pairs=0x10000, np=2, pages=9, st=None):
        a = (pf._PagedArrayStruct * max(1, len(arrays)))(*[pf._PagedArrayStruct(*x) for x in arrays])
        return lib.pfkv_copy_pages(ctypes.addressof(a), len(arrays) if n is None else n, pairs, np, i64(pages), st, None)
    def expect(f, want, **kw):
        got = f(**kw)
        assert got == want, (f.__name__, kw, got, want, lib.pfkv_last_error())
        assert want == 0 or f.__name__ in lib.pfkv_last_error().decode() or f in (embed, append), lib.pfkv_last_error()
"""


def refuses(code):
    r = without_device(CALLS + code + "\n    print('done')\n")
    assert r.returncode == 0 and r.stdout.split() == ["done"], (r.returncode, r.stdout, r.stderr)


def test_rotary_calls():
    refuses("""
    for f in (embed, append):
        expect(f, NO)
        expect(f, 0, T=0)
        for kw in (dict(T=-1), dict(D=0), dict(D=-16), dict(pos=None), dict(pos=0x10002), dict(r=None), dict(D=112)):
            expect(f, BAD, **kw)
        expect(f, UNS, D=120)
        expect(f, UNS, D=4112)
    for kw in (dict(H=0), dict(out=None), dict(x=None), dict(out=0x100008), dict(x=0x10008), dict(os=1016), dict(xs=1028), dict(xs=-1024),
               dict(os=big), dict(xs=1 << 31)):
        expect(embed, BAD, **kw)
    expect(embed, UNS, H=1 << 23)
    # in place, beside and across each other
    expect(embed, NO, out=0x10000)
    expect(embed, BAD, out=0x10000, os=2048)
    expect(embed, NO, out=0x10000, os=2048, T=1)
    expect(embed, BAD, out=0x10000 + 16)
    expect(embed, NO, out=0x10000 + 3 * 2048)
    expect(embed, BAD, out=0x10000 + 3 * 2048 - 16)
    for kw in (dict(Hq=0), dict(H=0), dict(P=0), dict(pages=0), dict(pages=1 << 62), dict(qo=None), dict(q=None), dict(k=None), dict(kc=None),
               dict(v=None), dict(vc=None), dict(sv=None), dict(sk=None), dict(sl=None), dict(sl=0x10004), dict(k=0x10004),
               dict(kc=0x10004), dict(v=0x10004), dict(vc=0x10004), dict(sk=0x10002), dict(sv=0x10001), dict(ks=255), dict(ks=248),
               dict(vs=260), dict(gran=3), dict(gran=4), dict(gran=-1)):
        expect(append, BAD, **kw)
    assert "kv_append_fp8_block" in (append(gran=3), lib.pfkv_last_error().decode())[1]
    expect(append, UNS, D=528, ks=2000, vs=2000, qs=5000, qos=5000, gran=2)
    expect(append, NO, D=528, ks=2000, vs=2000, qs=5000, qos=5000, qo=0x10000000)
    expect(append, NO, qo=None, q=None, Hq=-5)
    expect(append, NO, v=None, vc=None, sv=None, vs=0)
    expect(append, UNS, H=1 << 22, ks=1 << 30, vs=1 << 30)
    """)


def test_rotary_descriptions(pf):
    import ctypes
    for kw in (dict(frequencies=[1.0] * 7), dict(frequencies=[]), dict(frequencies=[1.0] * 136), dict(frequencies=[1.0] * 8, first=8),
               dict(frequencies=[1.0] * 8, first=-16), dict(frequencies=[1.0] * 8, num_axes=0), dict(frequencies=[1.0] * 8, num_axes=9),
               dict(frequencies=[1.0] * 7 + [float("nan")]), dict(frequencies=[float("inf")] * 8),
               dict(frequencies=[1.0] * 8, axes=[0] * 7 + [2], num_axes=2)):
        with pytest.raises(pf.PfkvError):
            pf.Rotary(**kw)
    for kw in (dict(frequencies=[[1.0] * 8]), dict(frequencies=[1.0] * 8, axes=[0] * 7), dict(frequencies=[1.0] * 8, axes=[0.5] * 8),
               dict(frequencies=[1.0] * 8, axes=[-1] * 8), dict(frequencies=[1.0] * 8, axes=[2 ** 32] * 8),
               dict(frequencies=[1.0] * 8, num_axes=2 ** 32 + 1), dict(frequencies=[1.0] * 8, first=2 ** 32)):
        with pytest.raises(ValueError):
            pf.Rotary(**kw)
    assert pf.Rotary([1.0] * 8, axes=[0, 1, 2, 0, 1, 2, 0, 1]).num_axes == 3
    lib = pf.load()
    s = pf._RotaryStruct()
    f = (ctypes.c_double * 8)(*[1.0] * 8)
    assert lib.pfkv_rotary_init(None, f, None, 8, 1, 0, 0) == -1 and lib.pfkv_rotary_init(ctypes.byref(s), None, None, 8, 1, 0, 0) == -1
    # the struct of the header
    assert ctypes.sizeof(s) == 16 + 128 * 8 + 128


def test_turns_are_the_frequencies(pf):
    """turns[i] / 2^64 is the fraction of a turn per position, to the rounding
    of one double division (2^-53 of the whole) and the step of 2^-64."""
    f = np.concatenate([10000.0 ** (-np.arange(32) / 32), [0.0, 2 * np.pi, 7.5, 1e-30, 123456.789, -1.0, -0.25, 1e9]])
    r = pf.Rotary(f)
    for v, t in zip(f, r._struct.turns):
        whole = abs(v) / (2 * np.pi)
        frac = (whole - np.floor(whole)) * (1 if v >= 0 else -1) % 1.0
        off = abs(t / 2.0 ** 64 - frac)
        assert min(off, 1 - off) <= whole * 2.0 ** -52 + 2.0 ** -64, v
    assert (r._struct.turns[37] + pf.Rotary([1.0] * 8)._struct.turns[0]) % 2 ** 64 == 0


def test_a_description_that_nobody_filled():
    refuses("""
    for change in (dict(num_pairs=0), dict(num_pairs=12), dict(num_pairs=136), dict(first=8), dict(first=-16), dict(num_axes=0),
                   dict(num_axes=9)):
        r = pf.Rotary([1.0] * 64)
        for name, v in change.items():
            setattr(r._struct, name, v)
        expect(embed, BAD, r=r._ptr)
        expect(append, BAD, r=r._ptr)
    r = pf.Rotary([1.0] * 64)
    r._struct.axis[5] = 1
    expect(embed, BAD, r=r._ptr)
    """)


def test_verify_calls():
    refuses("""
    verify.__name__ = "verify_drafts"
    expect(verify, NO)
    expect(verify, NO, q=None, qs=0)
    expect(verify, NO, dt=2, p=0x10002, q=0x10006)
    expect(verify, 0, B=0, acc=None)
    expect(verify, NO, T=0, nx=None, p=None, tok=None, u=None, q=None)
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(dt=3), dict(dt=-1), dict(nx=None), dict(acc=None), dict(p=None), dict(tok=None),
               dict(u=None), dict(st=None), dict(p=0x10002), dict(q=0x10002), dict(dt=1, p=0x10001), dict(ps=999), dict(qs=999),
               dict(ps=-1000), dict(ps=big + 1), dict(nx=0x10002), dict(acc=0x10001), dict(tok=0x10002), dict(u=0x10002),
               dict(st=0x10002), dict(ctx=0x10002), dict(rs=0x10002)):
        expect(verify, BAD, **kw)
    expect(verify, UNS, V=(1 << 20) + 1, ps=1 << 21, qs=1 << 21)
    expect(verify, UNS, B=(1 << 24) + 1)
    """)


def test_copy_calls():
    refuses("""
    copy.__name__ = "copy_pages"
    ok = (0x10000, 4096, 4096)
    expect(copy, NO)
    expect(copy, NO, arrays=[ok] * 300)
    expect(copy, NO, arrays=[(0x10001, 3, 5)])
    expect(copy, 0, np=0, pairs=None)
    expect(copy, 0, n=0)
    for kw in (dict(n=-1), dict(np=-1), dict(pages=0), dict(pairs=None), dict(pairs=0x10004), dict(st=0x10002),
               dict(arrays=[ok, (None, 4096, 4096)]), dict(arrays=[(0x10000, 0, 4096)]), dict(arrays=[(0x10000, 4096, 4095)]),
               dict(arrays=[(0x10000, -1, 4096)]), dict(arrays=[(0x10000, 4096, 1 << 62)]), dict(np=0, arrays=[(0x10000, 0, 0)])):
        expect(copy, BAD, **kw)
    expect(copy, UNS, arrays=[(0x10000, 1 << 31, 1 << 31)])
    assert lib.pfkv_copy_pages(None, 1, 0x10000, 1, i64(4), None, None) == -1
    """)


def test_python_checks(monkeypatch, pf):
    """Types, shapes and places that the binding refuses, on fake tensors."""
    import torch
    bf, u8, i32, i64, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32

    class T(FakeTensor):
        def __init__(self, dtype, *shape, device=0):
            super().__init__(shape, dtype, device)

        def dim(self):
            return len(self.shape)

        def stride(self, i=None):
            return () if i is None else 1

    calls = []

    class Lib:
        def __getattr__(self, name):
            if name == "pfkv_last_error":
                return lambda: b""
            return lambda *a: calls.append((name, a)) or 0

    rot, rot3 = pf.Rotary([1.0] * 64), pf.Rotary([1.0] * 64, num_axes=3)
    monkeypatch.setattr(pf, "_lib", Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d, raising=False)
    x, pos = T(bf, 5, 8, 128), T(i32, 5)
    pf.rotary_embed(x, x, pos, rot)
    pf.rotary_embed(x, x, T(i32, 1, 5), rot)
    pf.rotary_embed(x, x, T(i32, 3, 5), rot3)
    assert [c[0] for c in calls] == ["pfkv_rotary_embed"] * 3
    for args in ((T(f32, 5, 8, 128), x, pos, rot), (x, T(f32, 5, 8, 128), pos, rot), (T(bf, 5, 7, 128), x, pos, rot), (x, x, T(i64, 5), rot),
                 (x, x, T(i32, 6), rot), (x, x, pos, rot3), (x, x, T(i32, 2, 5), rot), (T(bf, 5, 8, 128, device=1), x, pos, rot),
                 (x, x, T(i32, 5, device=1), rot)):
        with pytest.raises(ValueError):
            pf.rotary_embed(*args)
    k, cache, slots = T(bf, 5, 2, 128), T(u8, 9, 2, 16, 128), T(i64, 5)
    one, head, token = T(f32, 1), T(f32, 2), T(f32, 9, 2, 16)
    good = [x, x, k, k, cache, cache, slots, pos, rot, pf.SCALE_TENSOR, one, one]
    pf.rotary_append_fp8(*good)
    pf.rotary_append_fp8(None, None, k, None, cache, None, slots, pos, rot, pf.SCALE_HEAD, head)
    pf.rotary_append_fp8(*good[:9], pf.SCALE_TOKEN, token, token)
    assert calls[-1][0] == "pfkv_rotary_append_fp8" and calls[-2][1][:4] == (0, 0, 0, 0) and calls[-1][1][-1] == 70
    for at, bad in ((0, None), (1, None), (2, T(f32, 5, 2, 128)), (3, None), (3, T(bf, 5, 2, 64)), (4, T(i32, 9, 2, 16, 128)),
                    (5, None), (5, T(u8, 9, 2, 32, 128)), (6, T(i32, 5)), (7, T(i32, 4)), (10, head), (11, token), (11, None),
                    (10, T(f32, 1, device=1))):
        with pytest.raises(ValueError):
            pf.rotary_append_fp8(*good[:at], bad, *good[at + 1:])
    p, B = T(f32, 7, 100), T(i32, 2)
    good = [T(i32, 7), B, p, p, T(i32, 7), T(f32, 7), T(i32, 3), B, B]
    pf.verify_drafts(*good)
    pf.verify_drafts(*good[:3], None, *good[4:7])
    assert calls[-1][0] == "pfkv_verify_drafts" and calls[-1][1][4] is None and calls[-2][1][10:13] == (2, 7, 100)
    for at, bad in ((0, T(i64, 7)), (0, T(i32, 6)), (1, T(i32, 3)), (2, T(torch.float64, 7, 100)), (3, T(bf, 7, 100)), (3, T(f32, 7, 99)),
                    (4, T(i64, 7)), (5, T(bf, 7)), (6, T(i64, 3)), (7, T(i32, 3)), (8, T(i32, 1)), (8, T(i32, 2, device=1))):
        with pytest.raises(ValueError):
            pf.verify_drafts(*good[:at], bad, *good[at + 1:])
    with pytest.raises(ValueError):
        pf.PagedArrays([])
    with pytest.raises(ValueError):
        pf.PagedArrays([torch.zeros(4, 8)])   # not on a GPU
