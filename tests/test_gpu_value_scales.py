"""Decode over pages whose V scales lie many binades apart: a page's part in the
output goes by its probability times its values, however large the values of
pages with less of it."""
import numpy as np
import pytest

import block_reference as ref
from attend_reference import Pool, check_unit
from gpu_helpers import pf
from test_gpu_block_scales import bf16, dev

pytestmark = pytest.mark.gpu


def run(rng, pool, lens, G, width, split, favoured, lead, spread_of_heads=False):
    """Per request, the keys of page favoured[b] score `lead` above the others;
    dense decode and the list call over all pages, in random order."""
    import torch
    p, P, H = pf(), pool.P, pool.H
    B = len(lens)
    n = [-(-m // P) for m in lens]
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :n[b]] = at + np.arange(n[b])
        at += n[b]
    assert at <= pool.pages
    # queries along one direction per head group; its sign is the favoured page's keys
    q = rng.standard_normal((B, H * G, 128)) * 0.05
    way = rng.choice([-1.0, 1.0], (B, H, 1, 128))
    q = (q.reshape(B, H, G, 128) + way).reshape(B, H * G, 128)
    if spread_of_heads:  # half the heads look away from the page
        q[:, ::2] = rng.standard_normal(q[:, ::2].shape)
    for b in range(B):
        for h in range(H):
            page = table[b, favoured[b]]
            pool.codes["k"][page, h] = ref.encode(np.broadcast_to(way[b, h, 0], (P, 128)))
            pool.scales["k"][page, h] = 2.0 ** np.ceil(np.log2(lead / 128 / 0.088))
    q, qv = bf16(q)
    ld, bt = dev(np.array(lens, np.int32)), dev(table)
    cache = [dev(pool.codes["k"]), dev(pool.codes["v"]), p.SCALE_BLOCK, dev(pool.scales["k"]), dev(pool.scales["v"])]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    K = max(n)
    sel = np.full((B, H, K), -1, np.int32)
    for b in range(B):
        for h in range(H):
            sel[b, h, :n[b]] = rng.permutation(n[b])
    for call in ("dense", "list"):
        out.fill_(7)
        if call == "dense":
            ws = p.paged_decode_attn_scaled(out, q, *cache, bt, ld, 0.088, lse_out=lse, kv_split_tokens=split,
                                            max_total_chunks=sum(-(-m // split) for m in lens) if split else 0)
            torch.cuda.synchronize()
            assert p.workspace_status(ws) == 0
        else:
            p.paged_sparse_decode_attn(out, q, *cache, dev(sel), bt, ld, 0.088, lse_out=lse)
            torch.cuda.synchronize()
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, L in enumerate(lens):
            for h in range(H):
                heads = slice(h * G, (h + 1) * G)
                k, v, vs = pool.unit(table[b], h, np.arange(n[b]), L)
                check_unit(o[b, heads], l[b, heads], qv[b, heads], k, v, vs, 0.088, (call, b, h))


# 408 lists, so that a warp meets many pages of one list; tables for the one-launch
# kernel, for the kernel with a plan and a merge, and in chunks
B, H = 51, 8
FORMS = pytest.mark.parametrize("width,split", [(64, 0), (4096, 0), (4096, 128)])


def lengths(rng):
    return [16 * 40, 16] + [int(n) for n in rng.integers(16 * 20, 16 * 48, B - 2)]


@FORMS
@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("binades", [15, 26, 110])
def test_a_page_of_small_values_with_most_of_the_probability(width, split, G, binades):
    rng = np.random.default_rng(binades + G)
    lens = lengths(rng)
    pool = Pool(rng, sum(-(-m // 16) for m in lens), H, 16, kbin=(-9, -8), vbin=(-4, -2))
    favoured, first = [], 0
    for m in lens:
        n = -(-m // 16)
        favoured.append(int(rng.integers(0, n)))
        pool.scales["v"][first + favoured[-1]] *= 2.0 ** -binades
        first += n
    run(rng, pool, lens, G, width, split, favoured, lead=binades + 12.0)


@FORMS
@pytest.mark.parametrize("spread", [8, 30, 100])
def test_value_scales_over_many_binades(width, split, spread):
    """Every page its own power; heads that look at one page beside heads that
    look at all of them."""
    rng = np.random.default_rng(spread)
    lens = lengths(rng)
    pool = Pool(rng, sum(-(-m // 16) for m in lens), H, 16, kbin=(-9, -7), vbin=(-spread, 4))
    run(rng, pool, lens, 4, width, split, [int(rng.integers(0, -(-m // 16))) for m in lens], lead=30.0, spread_of_heads=True)


@pytest.mark.parametrize("width", [64, 4096])
def test_pages_with_value_scale_zero(width):
    """They count in the denominator and add nothing; first, last and between."""
    rng = np.random.default_rng(5)
    lens = [16 * 20, 16 * 9, 16]
    pool = Pool(rng, 40, 2, 16, kbin=(-9, -8))
    pool.scales["v"][[0, 1, 7, 19, 20, 28]] = 0
    pool.scales["v"][29] = 0
    run(rng, pool, lens, 4, width, 0, [5, 3, 0], lead=2.0)
