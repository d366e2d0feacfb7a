"""Seeded random configurations of the block-scale and block-sparse calls against
64-bit numpy: head groups, page sizes, ragged and empty requests, tables wider
than needed, spare pages, several appends per request."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import pf
from guard_helpers import Guarded
from test_gpu_block_scales import State, bf16, check_rows, context, dev
from test_gpu_block_sparse import lists, subset

pytestmark = pytest.mark.gpu

HEADS = [(8, 2), (16, 1), (4, 4), (20, 4), (64, 8), (7, 1), (12, 6), (9, 3)]


@pytest.mark.parametrize("seed", range(24))
def test_random_configuration(seed):
    import torch
    p, rng = pf(), np.random.default_rng(1000 + seed)
    Hq, H = HEADS[rng.integers(len(HEADS))]
    P = int(rng.choice([16, 32, 48, 64, 96, 128]))
    B = int(rng.integers(1, 7))
    lens = [int(x) for x in np.round(np.exp(rng.uniform(0, np.log(2500), B)))]
    lens[rng.integers(B)] *= int(rng.random() < 0.8)  # at times an empty request
    width = max(-(-max(lens) // P), 1) + int(rng.choice([0, 1, 3000]))
    st = State(seed, lens, H, 128, P, width=width)
    # two or three appends per request, in calls that take all requests
    cuts = np.sort(rng.integers(0, np.array(lens)[:, None] + 1, (B, int(rng.integers(1, 3)))), 1)
    done = np.zeros(B, int)
    for k in range(cuts.shape[1] + 1):
        upto = cuts[:, k] if k < cuts.shape[1] else np.array(lens)
        new = [int(x) for x in upto - done]
        if sum(new):
            st.append(new, upto)
            st.check(f"append {k}")
        done = upto
    full = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ctx, bt = dev(np.array(lens, np.int32)), dev(st.bt)
    # bounds
    bnd, bs = Guarded((st.pages, H, 2, 128), torch.int8, "cuda"), Guarded((st.pages, H), torch.float32, "cuda")
    rb, rs = bnd.t.cpu().numpy().copy(), bs.t.cpu().numpy().copy()
    p.page_key_bounds(bnd.t, bs.t, st.g["k"].t, bt, ctx, dev(full), max(max(lens), 1))
    ref.bounds(st.ref["k"], rb, rs, st.bt, lens, full, max(max(lens), 1))
    torch.cuda.synchronize()
    bnd.check()
    bs.check()
    assert np.array_equal(bnd.t.cpu().numpy(), rb)
    assert np.array_equal(bs.t.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    # selection
    q, qv = bf16(rng.standard_normal((B, Hq, 128)) * 2.0 ** rng.integers(-4, 4))
    top = int(rng.integers(1, max(2, -(-max(lens) // P) + 2)))
    recent = int(rng.integers(0, min(3, top + 1)))
    sink = int(rng.integers(0, min(3, top - recent + 1)))
    sel = Guarded((B, H, top), torch.int32, "cuda")
    status = Guarded((2, B, H), torch.int32, "cuda")
    ks = st.s["k"].t if rng.random() < 0.7 else None
    p.select_pages(sel.t, q, bnd.t, bs.t, bt, ctx, P, sink, recent, k_scales=ks, unit_status=status.t[0])
    torch.cuda.synchronize()
    sel.check()
    want = ref.select(qv, rb, rs, None if ks is None else st.ref["ks"], st.bt, lens, P, top, sink, recent)
    assert np.array_equal(sel.t.cpu().numpy(), want)
    # attention over those lists or others, and over everything
    if rng.random() < 0.5:
        want = lists(rng, lens, H, P, top, shuffled=True)
        sel.t.copy_(dev(want))
    c = {"k": st.ref["k"], "v": st.ref["v"], "ks": st.ref["ks"], "vs": st.ref["vs"]}
    scale = 2.0 ** -10
    out, lse = Guarded(q.shape, torch.bfloat16, "cuda"), Guarded(q.shape[:2], torch.float32, "cuda")
    cache = (st.g["k"].t, st.g["v"].t, p.SCALE_BLOCK, st.s["k"].t, st.s["v"].t)
    p.paged_sparse_decode_attn(out.t, q, *cache, sel.t, bt, ctx, scale, lse_out=lse.t, unit_status=status.t[1])
    torch.cuda.synchronize()
    for x in (out, lse, status):
        x.check()
    assert int(status.t.abs().sum()) == 0
    sets = [[subset(c, st.bt[b], h, m, P, want[b, h][want[b, h] >= 0]) for h in range(H)] for b, m in enumerate(lens)]
    check_rows(out.t.double().cpu().numpy(), lse.t.cpu().numpy(), qv, sets, scale, f"sparse, seed {seed}")
    split = int(rng.choice([0, 32, 256]))
    ws = p.paged_decode_attn_scaled(out.t, q, *cache, bt, ctx, scale, kv_split_tokens=split, lse_out=lse.t,
                                    max_total_chunks=sum(-(-m // split) for m in lens) if split else 0)
    torch.cuda.synchronize()
    assert p.workspace_status(ws) == 0
    out.check()
    lse.check()
    sets = [[context(c, st.bt[b], h, m, P) for h in range(H)] for b, m in enumerate(lens)]
    check_rows(out.t.double().cpu().numpy(), lse.t.cpu().numpy(), qv, sets, scale, f"dense, seed {seed}")
