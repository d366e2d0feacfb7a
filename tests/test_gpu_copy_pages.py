"""copy_pages against indexing, byte for byte."""
import numpy as np
import pytest

from guard_helpers import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


def random_bytes(shape, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def some_pairs(pages, n, seed):
    """n destinations, each once, from pages that are none."""
    rng = np.random.default_rng(seed)
    ids = rng.permutation(pages)
    return np.stack([rng.choice(ids[n:], n), ids[:n]], 1).astype(np.int32)


def copied(x, pairs):
    y = x.clone()
    for s, d in pairs.tolist():
        if s >= 0 and d >= 0 and s < x.shape[0] and d < x.shape[0]:
            y[d] = x[s]
    return y


# bytes of a page in each array
SIZES = [[1], [3, 16, 4096], [32, 65536, 2, 12], [4096 * 3 + 5, 8, 4, 100, 4112], [131072, 131072, 32, 32], [262144 + 16]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("pages,n", [(2, 1), (37, 12), (200, 99)])
def test_pages(pf, sizes, pages, n):
    import torch
    arrays = [Guarded((pages, s), torch.uint8, "cuda") for s in sizes]
    for i, a in enumerate(arrays):
        a.t.copy_(random_bytes((pages, sizes[i]), i))
    pairs = some_pairs(pages, n, pages + n)
    want = [copied(a.t, pairs) for a in arrays]
    pf.copy_pages(pf.PagedArrays([a.t for a in arrays]), torch.from_numpy(pairs).cuda())
    for a, w in zip(arrays, want):
        a.check()
        assert torch.equal(a.t, w)


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("page,stride", [(64, 64), (64, 96), (48, 50), (4096, 8192), (5000, 5001)])
def test_strides_and_alignment(pf, offset, page, stride):
    import torch
    pages = 21
    base = random_bytes((offset + pages * stride + 64,), 3)
    view = base[offset:offset + pages * stride].view(pages, stride)[:, :page]
    pairs = some_pairs(pages, 7, offset + page)
    want = base.clone()
    want[offset:offset + pages * stride].view(pages, stride)[:, :page] = copied(view, pairs)
    pf.copy_pages(pf.PagedArrays([view]), torch.from_numpy(pairs).cuda())
    assert torch.equal(base, want)


@pytest.mark.parametrize("layers", [1, 31, 64, 70])
def test_layers(pf, layers):
    """K, V, scales and bounds of every layer: up to 280 arrays, more than one launch takes."""
    import torch
    pages, H, P = 9, 2, 16
    kv = random_bytes((layers, 2, pages, H, P, 128), 1)
    scales = torch.rand(layers, pages, H, P, device="cuda")
    bounds = random_bytes((layers, pages, H, 2, 128), 2).view(torch.int8)
    pairs = some_pairs(pages, 3, layers)
    want = [copied(x.movedim(d, 0), pairs).movedim(0, d) for x, d in ((kv, 2), (scales, 1), (bounds, 1))]
    tensors = [kv[i, j] for i in range(layers) for j in (0, 1)] + list(scales) + list(bounds)
    pf.copy_pages(pf.PagedArrays(tensors), torch.from_numpy(pairs).cuda())
    assert all(torch.equal(x, w) for x, w in zip((kv, scales, bounds), want))


def test_a_cache_with_keys_and_values_side_by_side(pf):
    import torch
    cache = random_bytes((12, 2, 4, 16, 128), 1)
    pairs = some_pairs(12, 5, 1)
    keys = cache.clone()
    keys[:, 0] = copied(cache[:, 0], pairs)
    pf.copy_pages(pf.PagedArrays([cache[:, 0]]), torch.from_numpy(pairs).cuda())
    assert torch.equal(cache, keys)


def test_padding_bad_pages_and_status(pf):
    import torch
    x = random_bytes((8, 300), 4)
    big = 2 ** 31 - 1
    pairs = np.array([[0, 1], [-1, 2], [2, -1], [8, 3], [3, 8], [5, 5], [big, 4], [6, big], [7, 2], [-5, 99]], np.int32)
    want = copied(x, pairs)
    status = Guarded((10,), torch.int32, "cuda")
    pf.copy_pages(pf.PagedArrays([x]), torch.from_numpy(pairs).cuda(), pair_status=status.t)
    status.check()
    bad = pf.DEVERR["BAD_PAGE"]
    assert status.t.tolist() == [0, 0, 0, bad, bad, 0, bad, bad, 0, 0]
    assert torch.equal(x, want)
    pf.copy_pages(pf.PagedArrays([x]), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert torch.equal(x, want)


def test_one_page_to_many(pf):
    import torch
    x = random_bytes((500, 8192), 5)
    pairs = np.stack([np.full(499, 17), np.delete(np.arange(500), 17)], 1).astype(np.int32)
    pf.copy_pages(pf.PagedArrays([x]), torch.from_numpy(pairs).cuda())
    assert bool((x == x[17]).all())


def test_pages_beyond_four_gigabytes(pf):
    import torch
    pages, size = 40000, 131072   # 5.2 GB
    x = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    ids = [0, 16383, 16384, 32767, 32768, 39999]
    for i in ids:
        x[i] = random_bytes((size,), i)
    pairs = torch.tensor([[39999, 1], [0, 39998], [16384, 32769], [32768, 16385]], dtype=torch.int32, device="cuda")
    want = {d: x[s].clone() for s, d in pairs.tolist()}
    total = int(sum(x[i].long().sum() for i in ids) + sum(w.long().sum() for w in want.values()))
    pf.copy_pages(pf.PagedArrays([x]), pairs)
    assert all(torch.equal(x[d], w) for d, w in want.items())
    assert sum(int(part.sum(dtype=torch.int64)) for part in x.split(1000)) == total


def test_replayed_with_other_pairs(pf):
    import torch
    x = random_bytes((30, 2, 16, 128), 6)
    arrays = pf.PagedArrays([x])
    pairs = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pf.copy_pages(arrays, pairs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pf.copy_pages(arrays, pairs)
    for seed in range(3):
        now = some_pairs(30, 3, seed)
        want = copied(x, now)
        pairs[:3] = torch.from_numpy(now).cuda()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)


def test_arrays_that_are_refused(pf):
    import torch
    x = torch.zeros(6, 4, 8, device="cuda")
    for bad in ([], [x, x[:5]], [x.transpose(1, 2)], [x[:, ::2]], [x[:0]], [x, x.cpu()], [x[0, 0, 0]], [x, torch.zeros(6, 0, device="cuda")],
                [x[:1].transpose(1, 2)]):
        with pytest.raises(ValueError):
            pf.PagedArrays(bad)
    for good in ([x], [x[:, 1:3]], [x[..., :]], [x[:, 0], x[:, :, 0][:, :1]], [x[::2]]):
        pf.PagedArrays(good)
    with pytest.raises(pf.PfkvError):   # pages on top of each other
        pf.copy_pages(pf.PagedArrays([x[:1].expand(6, 4, 8)]), torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    pairs = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for bad in (pairs.long(), pairs[0], pairs.cpu(), torch.zeros(2, 1, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            pf.copy_pages(pf.PagedArrays([x]), bad)
