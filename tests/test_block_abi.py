"""Host-side argument checks of the block-scale and block-sparse calls, and of
their 64-bit reference's own parts (CPU only)."""
import ctypes

import numpy as np
import pytest

import block_reference as ref
import oracle

i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    import paged_fp8_kv_02_gb300 as pf
    from paged_fp8_kv_02_gb300 import _build
    _build.build_pfkv()
    return pf.load(build_if_missing=False)


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


def _err(lib):
    return lib.pfkv_last_error().decode()


def test_append_block_host_validation(lib):
    def call(B=2, T=4, mx=2, H=2, D=128, P=16, pages=64, maxp=8, k=_fake(), v=_fake(), vc=_fake(), vs=_fake(),
             ks=_fake(), bt=_fake(), st=_fake()):
        return lib.pfkv_kv_append_fp8_block(k, v, _fake(), vc, ks, vs, bt, maxp, _fake(), st, B, T, mx, H, D, P,
                                            i64(pages), None)

    for bad in (dict(B=-1), dict(T=-1), dict(mx=-1), dict(H=0), dict(P=0), dict(pages=0), dict(maxp=0)):
        assert call(**bad) == -1 and "bad sizes" in _err(lib), bad
    assert call(D=24) == -2
    assert call(maxp=1 << 27) == -2 and "too long" in _err(lib)
    assert call(P=1 << 25, maxp=1) == -2
    assert call(B=0) == 0 and call(T=0) == 0 and call(mx=0) == 0
    assert call(k=None) == -1 and call(st=None) == -1 and "null" in _err(lib)
    assert call(v=None) == -1 and call(vc=None) == -1 and call(vs=None) == -1 and "all" in _err(lib)
    assert call(ks=_fake(0x10002)) == -1 and "misaligned" in _err(lib)
    assert call(v=_fake(0x10008)) == -1 and call(bt=_fake(0x10001)) == -1
    assert call(B=1 << 20, T=1 << 20, mx=1 << 20, maxp=1 << 20, H=64) == -2 and "too many" in _err(lib)


def test_bounds_host_validation(lib):
    def call(B=2, mx=2, H=2, D=128, P=16, pages=64, maxp=8, bnd=_fake(), sc=_fake(), k=_fake()):
        return lib.pfkv_page_key_bounds(bnd, sc, k, _fake(), maxp, _fake(), _fake(), B, mx, H, D, P, i64(pages), None)

    for bad in (dict(B=-1), dict(mx=-1), dict(H=0), dict(P=0), dict(pages=0), dict(maxp=0)):
        assert call(**bad) == -1 and "bad sizes" in _err(lib), bad
    assert call(D=64) == -2 and call(maxp=1 << 27) == -2
    assert call(B=0) == 0 and call(mx=0) == 0
    assert call(bnd=None) == -1 and "null" in _err(lib)
    assert call(bnd=_fake(0x10008)) == -1 and call(sc=_fake(0x10002)) == -1 and "misaligned" in _err(lib)
    assert call(B=1 << 20, mx=1 << 20, maxp=1 << 20, H=64) == -2 and "too many" in _err(lib)


def test_select_host_validation(lib):
    def call(B=2, Hq=16, Hkv=2, D=128, P=16, pages=64, maxp=9000, top=4, sink=1, recent=1, sel=_fake(), ks=None, st=None,
             q=_fake(), ws=_fake(), wsb=1 << 20):
        return lib.pfkv_select_pages(sel, q, _fake(), _fake(), ks, _fake(), maxp, _fake(), B, Hq, Hkv, D, P, i64(pages),
                                     top, sink, recent, ws, wsb, st, None)

    for bad in (dict(B=-1), dict(Hkv=0), dict(P=0), dict(pages=0), dict(maxp=0), dict(top=0), dict(sink=-1),
                dict(recent=-1)):
        assert call(**bad) == -1 and "bad sizes" in _err(lib), bad
    assert call(Hkv=3) == -1
    assert call(sink=3, recent=2) == -1 and "top_pages" in _err(lib)
    assert call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == -1
    assert call(Hq=34) == -2 and call(D=64) == -2
    assert call(maxp=1 << 28) == -2 and call(B=1 << 30) == -2
    assert call(pages=1 << 30) == -2 and "2^31" in _err(lib)
    need = lib.pfkv_select_pages_workspace_size(2, 2, 9000)
    assert need >= 2 * 2 * 9000 * 4
    assert call(wsb=need - 1) == -5 and "too small" in _err(lib)
    assert call(ws=None) == -1 and call(ws=_fake(0x10080)) == -1
    assert lib.pfkv_select_pages_workspace_size(2, 0, 8) == 0
    assert lib.pfkv_select_pages_workspace_size(0, 2, 8) >= 0
    assert lib.pfkv_select_pages_workspace_size(64, 8, 1 << 20) >= 64 * 8 * (4 << 20)
    assert call(B=0) == 0
    assert call(sel=None) == -1 and "null" in _err(lib)
    assert call(q=_fake(0x10008)) == -1 and call(ks=_fake(0x10001)) == -1 and call(st=_fake(0x10002)) == -1


def test_sparse_host_validation(lib):
    def call(B=2, Hq=16, Hkv=2, D=128, P=16, pages=64, maxp=8, top=4, gran=3, sm=0.1, out=_fake(), ks=_fake(),
             lse=None, st=None, sel=_fake()):
        return lib.pfkv_paged_sparse_decode_attn(out, _fake(), _fake(), _fake(), gran, ks, _fake(), sel, top, _fake(),
                                                 maxp, _fake(), B, Hq, Hkv, D, P, i64(pages), sm, lse, st, None)

    for bad in (dict(B=-1), dict(Hkv=0), dict(P=0), dict(pages=0), dict(maxp=0), dict(top=0)):
        assert call(**bad) == -1 and "bad sizes" in _err(lib), bad
    assert call(Hkv=3) == -1 and call(Hq=34) == -2 and call(D=64) == -2 and call(P=24) == -2
    assert call(gran=2) == -2 and "per token" in _err(lib)
    assert call(gran=7) == -1 and "granularity" in _err(lib)
    assert call(pages=1 << 26) == -2 and "2^31" in _err(lib)
    assert call(maxp=1 << 27) == -2 and call(B=1 << 28) == -2
    assert call(sm=0.0) == -1 and call(sm=float("inf")) == -1 and call(sm=float("nan")) == -1
    assert call(B=0) == 0
    assert call(out=None) == -1 and call(sel=None) == -1 and call(ks=None) == -1 and "null" in _err(lib)
    assert call(out=_fake(0x10008)) == -1 and call(lse=_fake(0x10001)) == -1 and call(st=_fake(0x10002)) == -1


def test_block_granularity_of_the_scaled_calls(lib):
    """Decode takes it like the others; the slot-mapped append cannot."""
    rc = lib.pfkv_kv_append_fp8_scaled(_fake(), None, _fake(), None, _fake(), 4, 2, 128, 16, i64(8), 3, _fake(), None, None)
    assert rc == -1 and "kv_append_fp8_block" in _err(lib)
    rc = lib.pfkv_paged_decode_attn_scaled(_fake(), _fake(), _fake(), _fake(), 3, None, _fake(), _fake(), 8, _fake(), 2,
                                           16, 2, 128, 16, i64(64), 0.088, 0, _fake(), 1 << 24, None, None)
    assert rc == -1 and "null scale" in _err(lib)


# ------------------------------------------------- the reference's own parts
def test_reference_encoder_is_the_oracles():
    x = np.concatenate([np.random.default_rng(0).standard_normal(4096) * 2.0 ** e for e in range(-12, 9, 3)] +
                       [np.array([0.0, -0.0, 448, 464, 1e9, 2.0 ** -10, 1.5 * 2.0 ** -9, -2.0 ** -9])]).astype(np.float32)
    assert np.array_equal(ref.encode(x), oracle.e4m3_encode(x))


def test_block_scale_holds_the_largest_and_no_smaller_power_does():
    for a in (0.0, 1e-45, 2.0 ** -118, 448.0, 448.5, 1.0, 1.75, 1.7578125, 3.0e38):
        s = ref.block_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 448 * s / 2) and np.log2(s) == int(np.log2(s))


def test_scores_bound_the_products_of_every_key():
    """Up to the query's 8 bits: |rounding| <= 1/2 of a step per channel."""
    rng = np.random.default_rng(3)
    q = rng.standard_normal((4, 128))
    keys = ref.VALUES[rng.integers(0, 0x70, (1, 1, 32, 128))] * np.where(rng.random((1, 1, 32, 128)) < 0.5, -1, 1)
    codes = ref.encode(keys)
    bnd, bs = np.zeros((1, 1, 2, 128), np.int8), np.zeros((1, 1), np.float32)
    ref.bounds(codes, bnd, bs, np.zeros((1, 2), np.int32), [32], [0, 32], 32)
    lo, hi = bnd[0, 0].astype(np.float64) * bs[0, 0]
    assert np.all(lo <= keys[0, 0]) and np.all(hi >= keys[0, 0])
    Q = ref.group_query(q).astype(np.float64)
    step = np.abs(np.minimum(q, 0).sum(0)).max() / np.abs(Q[0]).max()
    bound = (Q[0] * lo + Q[1] * hi).sum() * step
    best = (q @ keys[0, 0].T).sum(0).max()
    # half a step per part and channel, and the step itself known to half a unit of its largest
    slack = step * (np.abs(lo).sum() + np.abs(hi).sum()) * 0.5 + abs(bound) * 0.5 / np.abs(Q[0]).max()
    assert best <= bound + slack
