"""rotary_embed and rotary_append_fp8 against a 64-bit reference."""
import itertools

import numpy as np
import pytest

from around_reference import BF16_HALF, e4m3_half_step, e4m3_values, turn_slack, turned
from guard_helpers import Guarded

pytestmark = pytest.mark.gpu

FREQ = lambda n, base=10000.0: base ** (-np.arange(n) / n)


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(T, H, D, seed, wide=0, big=1.0):
    """bf16 rows; wide > 0: part of rows that are `wide` elements longer."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, H * D + wide, device="cuda", generator=g) * big).bfloat16()
    at = wide // 16 * 8   # the call wants rows on 16 bytes
    return x[:, at:at + H * D].unflatten(1, (H, D))


# T, H, D, pairs, first, neighbours, axes, extra elements between tokens, span
EMBED = [
    (1, 1, 16, 8, 0, False, 1, 0, 1), (1, 64, 128, 64, 0, False, 1, 0, 100), (3, 7, 128, 64, 0, False, 3, 0, 1 << 20),
    (64, 64, 128, 64, 0, False, 3, 2048, 32768), (5, 12, 64, 32, 0, True, 2, 16, 9000), (300, 5, 80, 16, 48, False, 1, 0, 70000),
    (310, 3, 96, 40, 16, True, 2, 32, 1 << 20), (17, 128, 576, 32, 512, True, 1, 0, 65536), (700, 2, 256, 128, 0, False, 8, 0, 5000),
    (1300, 4, 128, 32, 0, True, 1, 8, 131072), (2, 3, 4096, 128, 256, False, 1, 0, 777), (640, 1, 48, 8, 32, False, 1, 0, 50),
]


@pytest.mark.parametrize("T,H,D,n,first,near,axes,wide,span", EMBED)
@pytest.mark.parametrize("in_place", [False, True])
def test_embed(pf, T, H, D, n, first, near, axes, wide, span, in_place):
    import torch
    rng = np.random.default_rng(T * 31 + D)
    x = make(T, H, D, T + D, wide)
    want_in = f64(x)
    pos = rng.integers(-span, span, (axes, T)).astype(np.int32)
    ax = rng.integers(0, axes, n).astype(np.int32)
    rot = pf.Rotary(FREQ(n), axes=ax, first=first, neighbours=near, num_axes=axes)
    out = x if in_place else Guarded((T, H, D), torch.bfloat16, "cuda")
    around = x.storage_offset(), (x._base if x._base is not None else x).clone()
    pf.rotary_embed(out if in_place else out.t, x, torch.from_numpy(pos).cuda(), rot)
    if not in_place:
        out.check()
        assert torch.equal(x, x) and np.array_equal(f64(x), want_in)
    got = f64(out if in_place else out.t)
    ref, size, far = turned(want_in, pos, FREQ(n), ax, first, near)
    bound = np.abs(ref) * BF16_HALF + 2 * turn_slack(size, far)
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) - bound)
    stays = np.ones(D, bool)
    stays[first:first + 2 * n] = False
    assert np.array_equal(got[..., stays], want_in[..., stays])
    if in_place and wide:   # nothing beside the rows changed
        base = x._base
        mask = torch.ones_like(base, dtype=torch.bool)
        flat = mask.view(-1).as_strided(x.shape, x.stride(), x.storage_offset())
        flat.fill_(False)
        assert torch.equal(base[mask], around[1][mask])


def test_far_positions(pf):
    """Angles at the ends of 32 bits, from whole-number arithmetic: the
    fraction of a turn is position * floor(f / 2 pi 2^64) / 2^64."""
    import torch
    n, pos = 64, np.array([[2 ** 31 - 1, -2 ** 31, 1234567890, -1, 0, 1]], np.int32)
    f = FREQ(n, 500000.0)
    x = torch.zeros(pos.shape[1], 1, 128, dtype=torch.bfloat16, device="cuda")
    x[..., :64] = 1.0
    out = torch.empty_like(x)
    pf.rotary_embed(out, x, torch.from_numpy(pos).cuda(), pf.Rotary(f))
    turns = [int(np.ldexp(v / (2 * np.pi) - np.floor(v / (2 * np.pi)), 64)) for v in f]
    frac = np.array([[(int(p) * t % (1 << 64)) / 2.0 ** 64 for t in turns] for p in pos[0]])
    ref = np.concatenate([np.cos(2 * np.pi * frac), np.sin(2 * np.pi * frac)], 1)[:, None]
    got = f64(out)
    assert np.all(np.abs(got - ref) <= np.abs(ref) * BF16_HALF + 2 * turn_slack(np.ones_like(ref), 0 * ref))


def test_negative_frequency_turns_back(pf):
    import torch
    pos = torch.arange(-8, 9, dtype=torch.int32, device="cuda")
    x = make(17, 2, 128, 5)
    a, b = torch.empty_like(x), torch.empty_like(x)
    pf.rotary_embed(a, x, pos, pf.Rotary(FREQ(64)))
    pf.rotary_embed(b, x, -pos, pf.Rotary(-FREQ(64)))
    assert torch.equal(a, b)


# T, Hq, Hkv, D, pairs, first, neighbours, axes, page, gran, with V, extra
APPEND = [
    (1, 8, 2, 128, 64, 0, False, 1, 16, "tensor", True, 0), (64, 64, 8, 128, 64, 0, False, 3, 16, "head", True, 0),
    (64, 64, 8, 128, 64, 0, False, 3, 64, "token", True, 24), (333, 7, 1, 128, 32, 16, True, 2, 48, "token", True, 0),
    (1501, 20, 4, 128, 64, 0, False, 3, 32, "tensor", True, 8), (90, 12, 6, 80, 16, 48, False, 1, 96, "token", True, 0),
    (7, 16, 1, 576, 32, 512, True, 1, 64, "tensor", False, 0), (700, 3, 1, 576, 32, 512, True, 1, 64, "head", False, 64),
    (50, 0, 5, 64, 32, 0, True, 1, 16, "token", True, 0), (650, 4, 2, 512, 128, 0, False, 1, 16, "token", True, 0),
    (2, 5, 3, 16, 8, 0, False, 1, 1, "token", True, 0), (40, 4, 2, 272, 64, 144, False, 2, 16, "token", False, 0),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,n,first,near,axes,P,gran,has_v,wide", APPEND)
def test_append(pf, T, Hq, Hkv, D, n, first, near, axes, P, gran, has_v, wide):
    import torch
    rng = np.random.default_rng(T * 7 + D + Hkv)
    kind = {"tensor": pf.SCALE_TENSOR, "head": pf.SCALE_HEAD, "token": pf.SCALE_TOKEN}[gran]
    pages = -(-T // P) + 2
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    if T > 2:
        slots[1], slots[-1] = -1, pages * P   # skipped
    pos = rng.integers(0, 40000, (axes, T)).astype(np.int32)
    ax = rng.integers(0, axes, n).astype(np.int32)
    rot = pf.Rotary(FREQ(n), axes=ax, first=first, neighbours=near, num_axes=axes)
    d = lambda a: torch.from_numpy(a).cuda()
    q = make(T, Hq, D, 1, wide) if Hq else None
    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") if Hq else None
    new = {"k": make(T, Hkv, D, 2, wide), "v": make(T, Hkv, D, 3, wide)}
    if T > 3:
        new["k"][3, 0] = 0   # an all-zero row
        new["v"][3, 0] = 0
    shape = {"tensor": (1,), "head": (Hkv,), "token": (pages, Hkv, P)}[gran]
    cache = {x: Guarded((pages, Hkv, P, D), torch.uint8, "cuda") for x in "kv"}
    scale = {x: Guarded(shape, torch.float32, "cuda") for x in "kv"}
    for x in "kv":
        if gran != "token":
            scale[x].t.copy_(torch.rand(shape, device="cuda") * 0.02 + 0.004)
    before = {x: (cache[x].t.clone(), scale[x].t.clone()) for x in "kv"}
    v = (new["v"], cache["v"].t, scale["v"].t) if has_v else (None, None, None)
    pf.rotary_append_fp8(q_out, q, new["k"], v[0], cache["k"].t, v[1], d(slots), d(pos), rot, kind, scale["k"].t, v[2])
    torch.cuda.synchronize()
    for x in "kv":
        cache[x].check(x)
        scale[x].check(x)
    if Hq:
        embedded = torch.empty_like(q_out)
        pf.rotary_embed(embedded, q, d(pos), rot)
        assert torch.equal(embedded, q_out)
    # values: the bytes of kv_append_fp8_scaled
    other = {x: (before[x][0].clone(), before[x][1].clone()) for x in "kv"}
    pf.kv_append_fp8_scaled(new["k"].contiguous(), new["v"].contiguous(), other["k"][0], other["v"][0], d(slots), kind,
                            other["k"][1], other["v"][1])
    if has_v:
        assert torch.equal(other["v"][0], cache["v"].t)
        assert torch.equal(other["v"][1].view(torch.int32), scale["v"].t.view(torch.int32))
    else:
        assert torch.equal(before["v"][0], cache["v"].t)
    # keys: rows that were appended, and no others
    ok = (slots >= 0) & (slots < pages * P)
    page, off = slots[ok] // P, slots[ok] % P
    touched = np.zeros((pages, P), bool)
    touched[page, off] = True
    rest = d(~touched)[:, None, :].expand(pages, Hkv, P)
    assert torch.equal(cache["k"].t[rest], before["k"][0][rest])
    ref, size, far = turned(f64(new["k"]), pos, FREQ(n), ax, first, near)
    ref, slack = ref[ok], turn_slack(size, far)[ok]
    codes = cache["k"].t.cpu().numpy()[page, :, off]
    got = e4m3_values()[codes]
    if gran == "token":
        s = f64(scale["k"].t)[page, :, off]
        assert torch.equal(scale["k"].t[rest].view(torch.int32), before["k"][1][rest].view(torch.int32))
        amax = np.abs(ref).max(2)
        # the division rounds once more (2^-24)
        assert np.all(np.abs(s * 448 - amax) <= slack.max(2) + amax * 2.0 ** -23)
        s = s[..., None]
    else:
        s = np.broadcast_to(f64(scale["k"].t)[:, None], (Hkv, 1))
    live = np.broadcast_to(s > 0, got.shape)
    assert not np.any(codes[~live])
    r = np.divide(ref, s, out=np.zeros_like(ref), where=live)
    slack = np.divide(slack, s, out=np.zeros_like(ref), where=live) + np.abs(r) * 2.0 ** -23
    r = np.clip(r, -448, 448)
    # a value near a border of the format's binades may be rounded by either's step
    bound = np.maximum(e4m3_half_step(r), e4m3_half_step(np.clip(np.abs(r) + slack, 0, 448))) + slack
    assert np.all(np.abs(got - r)[live] <= bound[live])


def test_position_zero_is_the_plain_append(pf):
    import torch
    T, H, D, P = 200, 4, 128, 16
    rot = pf.Rotary(FREQ(64))
    for kind, shape in ((pf.SCALE_HEAD, (H,)), (pf.SCALE_TOKEN, (13, H, P))):
        k, v = make(T, H, D, 8), make(T, H, D, 9)
        slots = torch.randperm(13 * P, device="cuda")[:T]
        a = [torch.zeros(13, H, P, D, dtype=torch.uint8, device="cuda") for _ in range(4)]
        s = [torch.full(shape, 0.01, device="cuda") for _ in range(4)]
        pf.kv_append_fp8_scaled(k, v, a[0], a[1], slots, kind, s[0], s[1])
        pf.rotary_append_fp8(None, None, k, v, a[2], a[3], slots, torch.zeros(T, dtype=torch.int32, device="cuda"), rot, kind,
                             s[2], s[3])
        assert all(torch.equal(x, y) for x, y in ((a[0], a[2]), (a[1], a[3]), (s[0], s[2]), (s[1], s[3])))


def test_on_a_stream_and_in_a_graph(pf):
    """Captured with one rotary, replayed on new inputs after the handle is
    gone: the launch keeps its own copy."""
    import torch
    T, H = 33, 4
    x, out = make(T, H, 128, 1), torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rot = pf.Rotary(FREQ(64))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pf.rotary_embed(out, x, pos, rot, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pf.rotary_embed(out, x, pos, rot)
    first = out.clone()
    rot._struct.turns[:] = [0] * 128
    del rot
    y = make(T, H, 128, 2)
    x.copy_(y)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    want = torch.empty_like(out)
    pf.rotary_embed(want, y, pos, pf.Rotary(FREQ(64)))
    assert torch.equal(out, want) and not torch.equal(out, first)


def test_a_part_of_a_cache_beyond_two_gigabytes(pf):
    import torch
    H, P, D, pages = 8, 64, 128, 40000   # 2.6 GB
    k = make(3, H, D, 1)
    cache = torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * P - 1, 0, 33000 * P + 5], device="cuda")
    scale = torch.full((1,), 0.01, device="cuda")
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    pf.rotary_append_fp8(None, None, k, None, cache, None, slots, pos, pf.Rotary(FREQ(64)), pf.SCALE_TENSOR, scale)
    small = torch.zeros(1, H, P, D, dtype=torch.uint8, device="cuda")
    pf.rotary_append_fp8(None, None, k, None, small, None, torch.arange(3, device="cuda"), pos, pf.Rotary(FREQ(64)),
                         pf.SCALE_TENSOR, scale)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(cache[s // P, :, s % P], small[0, :, i])
    assert int((cache != 0).sum()) == int((small != 0).sum())


def test_no_tokens(pf):
    import torch
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    cache = torch.full((2, 4, 16, 128), 7, dtype=torch.uint8, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    pf.rotary_embed(e, e, pos, pf.Rotary(FREQ(64)))
    pf.rotary_append_fp8(e, e, e, None, cache, None, torch.empty(0, dtype=torch.int64, device="cuda"), pos, pf.Rotary(FREQ(64)),
                         pf.SCALE_TENSOR, torch.ones(1, device="cuda"))
    assert int((cache != 7).sum()) == 0


def test_rows_that_are_not_contiguous_within_a_token_are_refused(pf):
    import torch
    rot, pos = pf.Rotary(FREQ(64)), torch.zeros(4, dtype=torch.int32, device="cuda")
    for T in (1, 4):
        good = make(T, 4, 128, 1)
        for bad in (make(T, 128, 4, 1).transpose(1, 2), make(T, 8, 128, 1)[:, ::2], make(T, 4, 256, 1)[..., :128]):
            assert bad.shape == good.shape
            for args in ((bad, good), (good, bad)):
                with pytest.raises(ValueError):
                    pf.rotary_embed(*args, pos[:T], rot)
    wide = make(1, 4, 128, 1, 512)   # one token of wider rows
    out = torch.empty_like(wide)
    pf.rotary_embed(out, wide, pos[:1], rot)
    assert torch.equal(out, wide)


def test_on_another_device_or_its_stream(pf):
    """Every tensor of a call on one device, the current one or not."""
    import torch
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    with torch.cuda.device(0):
        x = make(3, 4, 128, 1).to("cuda:1")
        out, pos = torch.empty_like(x), torch.arange(3, dtype=torch.int32, device="cuda:1")
        pf.rotary_embed(out, x, pos, pf.Rotary(FREQ(64)))
        assert torch.cuda.current_device() == 0
        want = torch.empty_like(x, device="cuda:0")
        pf.rotary_embed(want, x.cuda(0), pos.cuda(0), pf.Rotary(FREQ(64)))
        assert torch.equal(out.cpu(), want.cpu())
