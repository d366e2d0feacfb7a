"""Block-sparse and short dense decode where a warp takes more than the 32 pages
that it looks up at a time: full lists, lists with gaps in them (padding, pages
outside the context or the pool), and lists longer than the context has pages."""
import numpy as np
import pytest

from attend_reference import Pool, check_unit
from gpu_helpers import pf
from guard_helpers import Guarded
from test_gpu_block_scales import bf16, dev

pytestmark = pytest.mark.gpu


def run_lists(rng, pool, lens, G, table, sel, gran, bad=None):
    """One call over lists sel [B][H][K]; bad: the table as the call sees it."""
    import torch
    p, P, H = pf(), pool.P, pool.H
    B = len(lens)
    if gran != p.SCALE_BLOCK:
        for x in "kv":
            s = (rng.random(H if gran == p.SCALE_HEAD else 1) * 0.004 + 0.002).astype(np.float32)
            pool.scales[x + "dev"] = s
            pool.scales[x] = np.broadcast_to(s, (pool.pages, H))
    q, qv = bf16(rng.standard_normal((B, H * G, 128)))
    out, lse = Guarded(q.shape, torch.bfloat16, "cuda"), Guarded(q.shape[:2], torch.float32, "cuda")
    st = Guarded((B, H), torch.int32, "cuda")
    seen = table if bad is None else bad
    p.paged_sparse_decode_attn(out.t, q, dev(pool.codes["k"]), dev(pool.codes["v"]), gran,
                               dev(pool.scales.get("kdev", pool.scales["k"])),
                               dev(pool.scales.get("vdev", pool.scales["v"])), dev(sel), dev(seen),
                               dev(np.array(lens, np.int32)), 0.088, lse_out=lse.t, unit_status=st.t)
    torch.cuda.synchronize()
    for x in (out, lse, st):
        x.check()
    o, l, status = out.t.double().cpu().numpy(), lse.t.double().cpu().numpy(), st.t.cpu().numpy()
    for b, L in enumerate(lens):
        npages = -(-L // P)
        for h in range(H):
            entries = sel[b, h][sel[b, h] >= 0]
            inside = entries[entries < npages]
            good = inside[(seen[b, inside] >= 0) & (seen[b, inside] < pool.pages)]
            want = (p.DEVERR["BAD_TOPK"] if len(inside) < len(entries) else 0) | \
                   (p.DEVERR["BAD_PAGE"] if len(good) < len(inside) else 0)
            assert status[b, h] == want, (b, h)
            heads = slice(h * G, (h + 1) * G)
            k, v, vs = pool.unit(table[b], h, good, L)
            check_unit(o[b, heads], l[b, heads], qv[b, heads], k, v, vs, 0.088, (b, h))


def gappy(rng, B, H, K, npages, share):
    """Lists in which `share` of the entries are pages, in random places."""
    sel = np.full((B, H, K), -1, np.int32)
    for b in range(B):
        for h in range(H):
            at = rng.random(K) < share
            sel[b, h, at] = rng.choice(npages[b], int(at.sum()), replace=False)
    return sel


# 51 requests of 8 heads: one CTA of four warps a list, 64 entries a warp; 2 lists:
# clusters of eight CTAs of eight warps; 64 lists: some CTAs each
@pytest.mark.parametrize("B,H,G,K", [(51, 8, 4, 256), (26, 8, 12, 256), (2, 1, 8, 2600), (8, 8, 2, 1100)])
@pytest.mark.parametrize("share", [0.05, 0.1, 1.0])
@pytest.mark.parametrize("gran", [0, 1, 3])
def test_lists_of_many_entries_a_warp(B, H, G, K, share, gran):
    rng = np.random.default_rng(K + B + gran)
    pool = Pool(rng, 40, H, 16)
    lens = [16 * (K + 3 * b) - b % 16 for b in range(B)]
    npages = [-(-m // 16) for m in lens]
    table = rng.integers(0, pool.pages, (B, max(npages))).astype(np.int32)
    if share == 1.0 and B > 8:  # a few full lists are enough
        lens = [m if b % 5 == 0 else 0 for b, m in enumerate(lens)]
        sel = np.full((B, H, K), -1, np.int32)
        sel[::5] = gappy(rng, len(lens[::5]), H, K, npages[::5], 1.0)
    else:
        sel = gappy(rng, B, H, K, npages, share)
    run_lists(rng, pool, lens, G, table, sel, gran)


@pytest.mark.parametrize("P,G", [(16, 4), (32, 12), (48, 1)])
def test_batches_of_few_entries(P, G):
    """Runs of 32 entries with 0, 1, 2, 3 or 32 pages among padding, pages
    beyond the context and pages outside the pool."""
    B, H, K = 51, 8, 512
    rng = np.random.default_rng(P)
    pool = Pool(rng, 40, H, P)
    lens = [P * (K + 40) - int(rng.integers(0, P)) for _ in range(B)]
    table = rng.integers(0, pool.pages, (B, K + 40)).astype(np.int32)
    bad = table.copy()
    outside = rng.random(table.shape) < 0.2
    bad[outside] = rng.choice([-1, -7, pool.pages, 2 ** 31 - 1], int(outside.sum()))
    sel = np.full((B, H, K), -1, np.int32)
    for b in range(B):
        for h in range(H):
            pages, at = rng.permutation(K + 40), 0
            if (b + h) % 4 == 1:  # wrong entries among the padding as well
                sel[b, h, rng.random(K) < 0.3] = K + 40 + int(rng.integers(0, 1000))
            for i in range(0, K, 32):
                n = int(rng.choice([0, 1, 1, 2, 3, 32]))
                sel[b, h, i + rng.choice(32, n, replace=False)] = pages[at:at + n]
                at += n
    run_lists(rng, pool, lens, G, table, sel, 3, bad if G != 1 else None)


@pytest.mark.parametrize("H,G,P,lens", [(8, 1, 16, [16384] * 8), (8, 9, 16, [16384 - 100 * b for b in range(8)]),
                                        (2, 4, 32, [32768, 30001, 5])])
def test_short_dense_decode_of_many_pages_a_warp(H, G, P, lens):
    """Tables that the one-launch kernel takes with contexts as long as they
    are: about 43 pages a warp for 64 lists of 1024."""
    import torch
    p, rng = pf(), np.random.default_rng(P + G)
    pool, B = Pool(rng, 48, H, P), len(lens)
    table = rng.integers(0, pool.pages, (B, -(-max(lens) // P))).astype(np.int32)
    q, qv = bf16(rng.standard_normal((B, H * G, 128)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = p.paged_decode_attn_scaled(out, q, dev(pool.codes["k"]), dev(pool.codes["v"]), p.SCALE_BLOCK,
                                    dev(pool.scales["k"]), dev(pool.scales["v"]), dev(table),
                                    dev(np.array(lens, np.int32)), 0.088, lse_out=lse)
    torch.cuda.synchronize()
    assert p.workspace_status(ws) == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, L in enumerate(lens):
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            k, v, vs = pool.unit(table[b], h, np.arange(-(-L // P)), L)
            check_unit(o[b, heads], l[b, heads], qv[b, heads], k, v, vs, 0.088, (b, h))


def test_pages_after_padding_are_attended():
    """A list may be longer than the context has pages, with its pages in any
    places: behind the padding too."""
    rng = np.random.default_rng(71)
    pool = Pool(rng, 12, 1, 16)
    table = rng.integers(0, 12, (4, 9)).astype(np.int32)
    sel = np.full((4, 1, 8), -1, np.int32)
    sel[0, 0, :4] = [-1, -1, 0, 1]
    sel[1, 0] = [-1, 1, -1, -1, -1, -1, -1, 0]
    sel[2, 0, 7] = 0
    sel[3, 0] = [2, -3, 0, -1, 9, -1, 1, 400]  # 9 and 400: beyond the context
    run_lists(rng, pool, [32, 20, 5, 48], 4, table, sel, 3)


# clusters of one CTA, of some and of eight; contexts of no page to as many as the list
@pytest.mark.parametrize("B,H,G,K,P", [(51, 8, 4, 300, 16), (2, 1, 8, 2600, 16), (8, 8, 12, 500, 48), (3, 2, 1, 7, 128)])
@pytest.mark.parametrize("gran", [0, 3])
def test_lists_longer_than_the_context(B, H, G, K, P, gran):
    rng = np.random.default_rng(K + gran)
    pool = Pool(rng, 40, H, P)
    npages = rng.integers(0, K + 1, B)
    npages[:3] = [0, 1, K][:B]
    lens = [max(0, int(n) * P - int(rng.integers(0, P))) for n in npages]
    table = rng.integers(0, pool.pages, (B, K + 5)).astype(np.int32)
    bad = table.copy()
    outside = rng.random(table.shape) < 0.05
    bad[outside] = rng.choice([-1, pool.pages], int(outside.sum()))
    sel = np.full((B, H, K), -1, np.int32)
    for b in range(B):
        n = -(-lens[b] // P)
        for h in range(H):
            k = int(rng.integers(0, n + 1)) if rng.random() < 0.7 else n
            # in random places, at the end of the list, or after a run of padding
            at = (rng.choice(K, k, replace=False), K - 1 - np.arange(k), np.arange(k) + (K - k) // 2)[int(rng.integers(3))]
            sel[b, h, at] = rng.choice(n, k, replace=False) if n else []
            if rng.random() < 0.2:
                free = np.flatnonzero(sel[b, h] < 0)
                if len(free):
                    sel[b, h, rng.choice(free)] = K + 1000
    run_lists(rng, pool, lens, G, table, sel, gran, bad)
