"""Page scores beyond fp32's range: pages that are listed by rule stay listed,
pages outside the pool stay last, and scores in range keep their order."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import pf
from test_gpu_block_scales import bf16, dev, tables
from test_gpu_block_sparse import random_bounds

pytestmark = pytest.mark.gpu

LARGEST = float(np.finfo(np.float32).max)


def expected(qv, bnd, bs, ks, bt_row, h, n, pool, top, sink, recent, G):
    """One list from scores clamped to fp32's range."""
    Q = ref.group_query(qv[h * G:(h + 1) * G])
    score = np.full(n, -np.inf)
    for i in range(n):
        page = int(bt_row[i])
        if 0 <= page < pool:
            x = float((bnd[page, h].astype(np.int64) * Q).sum()) * float(bs[page, h]) * float(ks[page, h])
            score[i] = min(max(x, -LARGEST), LARGEST)
    score[:sink] = np.inf
    score[n - recent:] = np.inf
    return np.sort(np.argsort(-score, kind="stable")[:top])


# one launch with clusters, and two kernels
@pytest.mark.parametrize("lens", [(1600, 1500, 333), (16 * 9000, 16 * 8500, 700)])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 1.0])
@pytest.mark.parametrize("exponent", [100, 118, 120, 127])
def test_scores_beyond_the_largest_number(lens, share, exponent):
    import torch
    p, rng, P, H, G, top, sink, recent = pf(), np.random.default_rng(exponent), 16, 2, 4, 20, 2, 3
    bt, pages = tables(rng, lens, P)
    bnd, bs = random_bounds(rng, pages, H)
    bnd[rng.random((pages, H)) < 0.05] = 0  # a score of zero under any scale
    ks = np.exp2(rng.integers(-9, -5, (pages, H))).astype(np.float32)
    large = rng.random((pages, H)) < share
    ks[large] = 2.0 ** exponent
    bad = bt.copy()
    for b, m in enumerate(lens):
        for i in rng.choice(np.arange(sink, -(-m // P) - recent), 3, replace=False):
            bad[b, i] = rng.choice([-1, pages])
    q, qv = bf16(rng.standard_normal((3, H * G, 128)))
    sel = torch.empty((3, H, top), dtype=torch.int32, device="cuda")
    p.select_pages(sel, q, dev(bnd), dev(bs), dev(bad), dev(np.array(lens, np.int32)), P, sink, recent, k_scales=dev(ks))
    got = sel.cpu().numpy()
    for b, m in enumerate(lens):
        for h in range(H):
            want = expected(qv[b], bnd, bs, ks, bad[b], h, -(-m // P), pages, top, sink, recent, G)
            assert np.array_equal(got[b, h], want), (b, h)
