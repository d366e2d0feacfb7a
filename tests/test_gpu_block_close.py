"""Seeded random configurations of decode over block scales and over lists, with
logits that keep many tokens in play, within the bound of the f16 products the
kernels use (attend_reference)."""
import numpy as np
import pytest

from attend_reference import check_unit
from gpu_helpers import pf
from guard_helpers import Guarded
from test_gpu_block_random import HEADS
from test_gpu_block_scales import State, bf16, context, dev
from test_gpu_block_sparse import lists, subset

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(24))
def test_random_configuration_closely(seed):
    import torch
    p, rng = pf(), np.random.default_rng(4000 + seed)
    Hq, H = HEADS[rng.integers(len(HEADS))]
    G = Hq // H
    P = int(rng.choice([16, 32, 48, 64, 96, 128]))
    B = int(rng.integers(1, 7))
    lens = [int(x) for x in np.round(np.exp(rng.uniform(0, np.log(2500), B)))]
    lens[rng.integers(B)] *= int(rng.random() < 0.8)  # at times an empty request
    width = max(-(-max(lens) // P), 1) + int(rng.choice([0, 1, 3000]))
    st = State(seed, lens, H, 128, P, width=width)
    if sum(lens):
        st.append(lens, lens)
        st.check("append")
    c = {"k": st.ref["k"], "v": st.ref["v"], "ks": st.ref["ks"], "vs": st.ref["vs"]}
    q, qv = bf16(rng.standard_normal((B, Hq, 128)) * np.exp2(rng.integers(-6, 7, (B, Hq, 1))))
    # softmax_scale by the largest product of any head: logits within +-8 at most
    full = [[context(c, st.bt[b], h, m, P) for h in range(H)] for b, m in enumerate(lens)]
    largest = max([float(np.abs(qv[b, h * G:(h + 1) * G] @ full[b][h][0].T).max())
                   for b, m in enumerate(lens) if m for h in range(H)] + [1e-30])
    scale = float(np.float32(8.0 / largest))
    top = int(rng.integers(1, max(2, -(-max(lens) // P) + 2)))
    sel = lists(rng, lens, H, P, top, shuffled=True)
    bt, ctx = dev(st.bt), dev(np.array(lens, np.int32))
    cache = (st.g["k"].t, st.g["v"].t, p.SCALE_BLOCK, st.s["k"].t, st.s["v"].t)
    out, lse = Guarded(q.shape, torch.bfloat16, "cuda"), Guarded(q.shape[:2], torch.float32, "cuda")

    def check(sets, what):
        torch.cuda.synchronize()
        out.check(what)
        lse.check(what)
        o, l = out.t.double().cpu().numpy(), lse.t.double().cpu().numpy()
        for b in range(B):
            for h in range(H):
                heads = slice(h * G, (h + 1) * G)
                check_unit(o[b, heads], l[b, heads], qv[b, heads], *sets[b][h], scale, (what, seed, b, h))

    p.paged_sparse_decode_attn(out.t, q, *cache, dev(sel), bt, ctx, scale, lse_out=lse.t)
    check([[subset(c, st.bt[b], h, m, P, sel[b, h][sel[b, h] >= 0]) for h in range(H)] for b, m in enumerate(lens)], "lists")
    for split in (0, 64):
        ws = p.paged_decode_attn_scaled(out.t, q, *cache, bt, ctx, scale, kv_split_tokens=split, lse_out=lse.t,
                                        max_total_chunks=sum(-(-m // split) for m in lens) if split else 0)
        check(full, f"dense {split}")
        assert p.workspace_status(ws) == 0
