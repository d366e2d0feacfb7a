"""Rotary calls on parts of one buffer: projections whose queries, keys and
values stand in one row, turned into other parts of the same rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

FREQ = 10000.0 ** (-np.arange(64) / 64)


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


def rows(T, wide, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, wide, device="cuda", generator=g).bfloat16()


def part(buf, at, heads, D=128):
    return buf[:, at:at + heads * D].unflatten(1, (heads, D))


@pytest.mark.parametrize("T", [1, 2, 77, 1300])
@pytest.mark.parametrize("near", [False, True])
def test_from_one_part_into_another(pf, T, near):
    import torch
    H, D = 3, 128
    buf = rows(T, 2 * H * D + 40, T)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    rot = pf.Rotary(FREQ, neighbours=near)
    want = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    pf.rotary_embed(want, part(buf, 8, H).contiguous(), pos, rot)
    for source, target in ((8, 16 + H * D), (16 + H * D, 8)):
        now = buf.clone()
        part(now, source, H).copy_(part(buf, 8, H))
        all_ = now.clone()
        pf.rotary_embed(part(now, target, H), part(now, source, H), pos, rot)
        part(all_, target, H).copy_(want)
        assert torch.equal(now, all_)


@pytest.mark.parametrize("T", [1, 64, 700])
@pytest.mark.parametrize("gran", ["tensor", "token"])
def test_append_of_one_buffer(pf, T, gran):
    """Queries turned in place, and into a part behind the values."""
    import torch
    Hq, H, D, P, pages = 6, 2, 128, 16, 50
    width = (2 * Hq + 2 * H) * D
    buf = rows(T, width, T)
    at = {"q": 0, "k": Hq * D, "v": (Hq + H) * D, "out": (Hq + 2 * H) * D}
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 5
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T))[:T].cuda()
    kind, shape = (pf.SCALE_TENSOR, (1,)) if gran == "tensor" else (pf.SCALE_TOKEN, (pages, H, P))
    rot = pf.Rotary(FREQ)

    def call(q_out, q, k, v):
        caches = [torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.full(shape, 0.02, device="cuda") for _ in range(2)]
        pf.rotary_append_fp8(q_out, q, k, v, *caches, slots, pos, rot, kind, *scales)
        return caches + scales

    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    want = call(q_out, *(part(buf, at[x], H if x != "q" else Hq).contiguous() for x in "qkv"))
    for target in ("q", "out"):
        now = buf.clone()
        got = call(part(now, at[target], Hq), part(now, at["q"], Hq), part(now, at["k"], H), part(now, at["v"], H))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        all_ = buf.clone()
        part(all_, at[target], Hq).copy_(q_out)
        assert torch.equal(now, all_)


@pytest.mark.parametrize("T,H,wide", [(5, 12, 16), (64, 64, 2048), (1300, 4, 8), (3, 7, 0)])
def test_what_stands_around_the_input_stays(pf, T, H, wide):
    """Out of place, the input's rows and what lies between them are only read."""
    import torch
    buf = rows(T, H * 128 + wide, T)
    x, before = part(buf, wide // 16 * 8, H), buf.clone()
    out = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    pf.rotary_embed(out, x, torch.arange(T, dtype=torch.int32, device="cuda") + 1, pf.Rotary(FREQ))
    assert torch.equal(buf, before) and not torch.equal(out, x)
