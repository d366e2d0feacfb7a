"""Block-sparse decode on the GPU: key bounds and page lists equal to 64-bit
numpy, attention over lists within the bound derived in
block_reference.tolerance, and the calls of a decode step in a row."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import pf
from guard_helpers import Guarded
from test_gpu_block_scales import State, bf16, check_rows, context, dev, filled, tables

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bounds
@pytest.mark.parametrize("H,P", [(2, 16), (1, 1), (3, 7), (48, 32), (1, 128)])
def test_bounds_of_contexts_and_of_last_pages(H, P):
    import torch
    p, rng = pf(), np.random.default_rng(P)
    lens = np.array([1, P, P + 1, 5 * P - 1, 0, 77], np.int32)
    bt, pages = tables(rng, lens, P)
    k = rng.integers(0, 256, (pages, H, P, 128)).astype(np.uint8)
    k[(k & 127) == 127] = 0x22
    k[rng.random((pages, H, P)) < 0.1] = 0
    k[bt[2, 0]] = 0x80  # a page of -0
    k[bt[3, 0], :, P // 2:] = 0x81  # rows of the smallest negative value
    for b, m in enumerate(lens):
        if m % P:
            k[bt[b, m // P], :, m % P:] = 0x7E  # 448 past the context
    got, sc = Guarded((pages, H, 2, 128), torch.int8, "cuda"), Guarded((pages, H), torch.float32, "cuda")
    want, want_s = got.t.cpu().numpy().copy(), sc.t.cpu().numpy().copy()
    for new in (lens, np.minimum(lens, 1), np.minimum(lens, P + 1)):
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        got.t.fill_(-91)
        want[:] = -91
        p.page_key_bounds(got.t, sc.t, dev(k), dev(bt), dev(lens), dev(start), int(new.max()))
        torch.cuda.synchronize()
        ref.bounds(k, want, want_s, bt, lens, start, int(new.max()))
        got.check()
        sc.check()
        assert np.array_equal(got.t.cpu().numpy(), want)
        assert np.array_equal(sc.t.cpu().numpy().view(np.uint32), want_s.view(np.uint32))


def test_bounds_pass_over_nan_codes_and_what_does_not_fit():
    import torch
    p, rng, P = pf(), np.random.default_rng(4), 16
    lens = np.array([40, 40, 40, 40], np.int32)
    bt, pages = tables(rng, lens, P)
    k = rng.integers(0, 0x70, (pages, 2, P, 128)).astype(np.uint8)
    k[bt[0, 0], 0, 3, 7] = 0x7F
    k[bt[0, 1], 1, 5:9, :] = 0xFF
    bad = bt.copy()
    bad[1, 1], bad[2, 0] = -1, pages
    got = torch.full((pages, 2, 2, 128), -91, dtype=torch.int8, device="cuda")
    sc = torch.full((pages, 2), -1.0, device="cuda")
    want, want_s = got.cpu().numpy().copy(), sc.cpu().numpy().copy()
    arg = np.array([40, 40, 40, 49], np.int32)  # the last is longer than its table
    start = np.array([0, 40, 80, 120, 160], np.int32)
    p.page_key_bounds(got, sc, dev(k), dev(bad), dev(arg), dev(start), 40)
    torch.cuda.synchronize()
    ref.bounds(k, want, want_s, bad, arg, start, 40)
    assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(sc.cpu().numpy(), want_s)


def test_bounds_of_channels_with_only_nan_codes():
    import torch
    p, rng, P = pf(), np.random.default_rng(5), 16
    lens = np.array([16, 17, 33], np.int32)  # the last pages hold one token
    bt, pages = tables(rng, lens, P)
    k = rng.integers(0, 0x70, (pages, 2, P, 128)).astype(np.uint8)
    zeros = k.copy()  # such a channel counts as 0, and the others as if it were not there
    for b, i, h, d in ((0, 0, 1, slice(3, 9)), (1, 1, 0, 127), (2, 2, 0, slice(0, 128)), (2, 1, 1, slice(16, 40, 8))):
        k[bt[b, i], h, :, d] = 0xFF if h else 0x7F
        zeros[bt[b, i], h, :, d] = 0
    got, sc = torch.zeros((pages, 2, 2, 128), dtype=torch.int8, device="cuda"), torch.zeros((pages, 2), device="cuda")
    want, want_s = got.cpu().numpy().copy(), sc.cpu().numpy().copy()
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    p.page_key_bounds(got, sc, dev(k), dev(bt), dev(lens), dev(start), 33)
    torch.cuda.synchronize()
    ref.bounds(zeros, want, want_s, bt, lens, start, 33)
    assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(sc.cpu().numpy(), want_s)


# ------------------------------------------------------------------ select
def random_bounds(rng, pages, H, flat=False):
    lo = rng.integers(-127, 100, (pages, H, 1, 128))
    hi = np.minimum(lo + rng.integers(0, 90, lo.shape), 127)
    b = np.concatenate([lo, hi], 2).astype(np.int8)
    if flat:
        b[:] = b[:1, :1]
    return b, np.exp2(rng.integers(-1, 1 if flat else 3, (pages, H)) * (0 if flat else 1)).astype(np.float32)


def run_select(lens, Hq, Hkv, P, top, sink, recent, seed=0, flat=False, ks=False, width=None, qscale=1.0, qbits=None):
    import torch
    p, rng = pf(), np.random.default_rng(seed)
    bt, pages = tables(rng, lens, P, width=width)
    bnd, bs = random_bounds(rng, pages, Hkv, flat)
    kscales = np.exp2(rng.integers(-9, -5, (pages, Hkv))).astype(np.float32) if ks else None
    q, qv = bf16(rng.standard_normal((len(lens), Hq, 128)) * qscale)
    if qbits is not None:
        q, qv = bf16(np.broadcast_to(qbits, qv.shape))
    sel = Guarded((len(lens), Hkv, top), torch.int32, "cuda")
    st = Guarded((len(lens), Hkv), torch.int32, "cuda")
    p.select_pages(sel.t, q, dev(bnd), dev(bs), dev(bt), dev(np.array(lens, np.int32)), P, sink, recent,
                   k_scales=None if kscales is None else dev(kscales), unit_status=st.t)
    torch.cuda.synchronize()
    sel.check()
    st.check()
    assert int(st.t.abs().sum()) == 0
    want = ref.select(qv, bnd, bs, kscales, bt, lens, P, top, sink, recent)
    assert np.array_equal(sel.t.cpu().numpy(), want), (lens, top)


@pytest.mark.parametrize("Hq,Hkv,P", [(8, 2, 16), (16, 1, 64), (4, 4, 48), (20, 4, 1), (7, 1, 128)])
@pytest.mark.parametrize("top,sink,recent", [(1, 0, 0), (1, 0, 1), (5, 1, 2), (64, 64, 0), (33, 0, 3)])
def test_select_equals_reference(Hq, Hkv, P, top, sink, recent):
    lens = [0, 1, P * top, P * top + 1, 40 * P - P // 2, 700 * P]
    run_select(lens, Hq, Hkv, P, top, sink, recent, seed=top, ks=top % 2 == 1)


def test_select_ties_go_to_the_lower_page():
    run_select([3000, 5001], 8, 2, 16, 100, 0, 0, flat=True)
    run_select([32000], 8, 1, 16, 1000, 2, 3, flat=True)   # a cluster a list
    run_select([9000, 8999], 8, 1, 1, 1500, 2, 3, flat=True)  # two kernels
    run_select([9000], 8, 1, 1, 8999, 0, 0, flat=True)
    run_select([3000], 8, 2, 16, 17, 0, 1, qbits=np.zeros(128))  # every score is zero


@pytest.mark.parametrize("top", [3, 255, 4097])
def test_select_large_tables(top):
    """Clusters of up to eight CTAs, shares of all sizes."""
    run_select([16 * 5000, 16 * 4097, 17], 8, 1, 16, top, 1, 2, seed=1, ks=True)
    run_select([8 * 30001], 3, 1, 8, top, 0, 0, seed=2)
    run_select([4096 * 7] * 20, 8, 8, 16, min(top, 1700), 1, 1, seed=3)
    run_select([8192, 8191], 8, 2, 1, top, 1, 1, seed=4)
    run_select([8193, 8191], 8, 2, 1, top, 1, 1, seed=5)
    run_select([2048, 2047, 300], 8, 2, 1, min(top, 2040), 1, 1, seed=6)
    run_select([2049, 2047, 300], 8, 2, 1, min(top, 2040), 1, 1, seed=7)


def test_select_table_much_wider_than_the_contexts():
    run_select([16 * 100, 5, 16 * 77], 8, 2, 16, 20, 1, 1, width=393216)


@pytest.mark.parametrize("qscale", [2.0 ** -133, 2.0 ** -100, 2.0 ** 120])
def test_select_queries_of_any_size(qscale):
    run_select([4000], 8, 1, 16, 40, 0, 0, qscale=qscale)


@pytest.mark.parametrize("batch", [9, 10, 13, 19, 20, 38, 39, 76])
@pytest.mark.parametrize("width", [2, 64, 512, 1024, 2048])
def test_select_for_every_cluster(batch, width):
    # 4 lists a request; the cluster of a list and one launch or two follow from both sizes
    rng = np.random.default_rng(width + batch)
    lens = [8 * width, 8 * width - 7, 0, 1] + [int(n) for n in rng.integers(0, 8 * width + 1, batch - 4)]
    run_select(lens, 8, 4, 8, max(1, width // 3), 1, 1 if width > 2 else 0, seed=batch, ks=batch % 2 == 0, width=width)


def test_select_by_two_kernels_in_a_graph_and_on_two_streams():
    """The path with a workspace: replayed from a graph with new queries, and
    two calls at once with a workspace each."""
    import torch
    p, rng, P, top = pf(), np.random.default_rng(17), 1, 100
    lens = [9000, 8500, 50]
    bt, pages = tables(rng, lens, P)
    bnd, bs = random_bounds(rng, pages, 2)
    q = [bf16(rng.standard_normal((3, 8, 128))) for _ in range(3)]
    d = [dev(bnd), dev(bs), dev(bt), dev(np.array(lens, np.int32))]
    assert p.select_pages_workspace_size(3, 2, bt.shape[1]) > 0
    sel = [torch.empty((3, 2, top), dtype=torch.int32, device="cuda") for _ in range(2)]
    ws = [torch.empty(p.select_pages_workspace_size(3, 2, bt.shape[1]), dtype=torch.uint8, device="cuda") for _ in range(2)]
    qin = q[0][0].clone()
    call = lambda i, x: p.select_pages(sel[i], x, *d, P, 1, 2, workspace=ws[i])
    call(0, qin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, qin)
    for x, xv in q:
        qin.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(sel[0].cpu().numpy(), ref.select(xv, bnd, bs, None, bt, lens, P, top, 1, 2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i, q[i][0])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(sel[i].cpu().numpy(), ref.select(q[i][1], bnd, bs, None, bt, lens, P, top, 1, 2))
    # a stream argument, the workspace left to the call
    sel[0].fill_(-5)
    torch.cuda.synchronize()
    for _ in range(3):
        p.select_pages(sel[0], q[1][0], *d, P, 1, 2, stream=streams[0])
    streams[0].synchronize()
    assert np.array_equal(sel[0].cpu().numpy(), ref.select(q[1][1], bnd, bs, None, bt, lens, P, top, 1, 2))


def test_select_bad_pages_and_lengths():
    import torch
    p, rng, P, top = pf(), np.random.default_rng(9), 16, 4
    lens = np.array([160, 160, 160], np.int32)
    bt, pages = tables(rng, lens, P)
    bnd, bs = random_bounds(rng, pages, 1)
    q, qv = bf16(rng.standard_normal((3, 4, 128)))
    bad = bt.copy()
    bad[0, 3], bad[0, 6] = -2, pages
    arg = np.array([160, -7, 161], np.int32)
    sel = torch.empty((3, 1, top), dtype=torch.int32, device="cuda")
    st = torch.empty((3, 1), dtype=torch.int32, device="cuda")
    p.select_pages(sel, q, dev(bnd), dev(bs), dev(bad), dev(arg), P, 1, 1, unit_status=st)
    torch.cuda.synchronize()
    assert st.cpu().numpy().ravel().tolist() == [p.DEVERR["BAD_PAGE"], p.DEVERR["BAD_CONTEXT"], p.DEVERR["BAD_CONTEXT"]]
    got = sel.cpu().numpy()
    want = ref.select(qv, bnd, bs, None, bt, np.array([160, 0, 160]), P, top, 1, 1)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    keep = [i for i in range(10) if i not in (3, 6)]
    Q = ref.group_query(qv[0])
    score = (bnd[bt[0], 0].astype(np.int64) * Q).sum((1, 2)) * bs[bt[0], 0].astype(np.float64)
    score[[0, 9]] = np.inf
    assert got[0, 0].tolist() == sorted(sorted(keep, key=lambda i: (-score[i], i))[:top])


# ------------------------------------------------------------------ sparse
def lists(rng, lens, Hkv, P, top, shuffled=False):
    """Random distinct pages; some entries of padding, in front as well."""
    sel = np.full((len(lens), Hkv, top), -1, np.int32)
    for b, m in enumerate(lens):
        n = -(-m // P)
        for h in range(Hkv):
            k = min(n, top) if (b + h) % 3 else int(rng.integers(0, min(n, top) + 1))
            got = rng.choice(n, k, replace=False) if n else np.zeros(0, int)
            if k and n - 1 not in got and h % 2:
                got[0] = n - 1  # the last, partial page
            width = min(n, top)
            at = np.sort(rng.choice(width, k, replace=False)) if shuffled else np.arange(k)
            sel[b, h, at] = got if shuffled else np.sort(got)
    return sel


def subset(c, bt_row, h, L, P, pages):
    k, v, vs = context(c, bt_row, h, L, P)
    t = np.concatenate([np.arange(i * P, min((i + 1) * P, L)) for i in pages] + [np.zeros(0, int)]).astype(int)
    return k[t], v[t], vs[t]


@pytest.mark.parametrize("Hq,Hkv,P,top,lens", [
    (8, 2, 16, 4, (1, 16, 17, 300, 0)), (16, 1, 64, 40, (5000, 64, 63)), (4, 4, 48, 1, (33, 96, 500)),
    (20, 4, 128, 9, (1000, 3, 129)), (64, 8, 16, 128, (2049, 257, 1, 31, 512, 6000)), (7, 1, 96, 33, (5000, 9000)),
    (48, 48, 16, 20, (700,)), (8, 1, 16, 1000, (16000, 15999, 40)),
    (32, 2, 16, 30, tuple(range(1, 1200, 57))),   # 42 lists of 16 heads
    (18, 6, 32, 25, tuple(range(3, 2000, 117))),  # 108 lists: clusters of 3 or 4
    (30, 15, 16, 12, tuple(range(1, 900, 45)))])  # 300 lists: clusters of 1 or 2
@pytest.mark.parametrize("gran", [0, 1, 3])
def test_sparse_decode_matches_reference(Hq, Hkv, P, top, lens, gran):
    import torch
    p, rng = pf(), np.random.default_rng(top + gran)
    bt, c = filled(rng, list(lens), Hkv, P)
    if gran != 3:
        for x in "kv":
            s = (rng.random(Hkv if gran else 1) * 0.01 + 0.002).astype(np.float32)
            c[x + "dev"] = s
            c[x + "s"] = np.broadcast_to(s, (c[x].shape[0], Hkv))
    sel = lists(rng, lens, Hkv, P, top, shuffled=gran == 1)
    q, qv = bf16(rng.standard_normal((len(lens), Hq, 128)))
    out, lse = Guarded(q.shape, torch.bfloat16, "cuda"), Guarded(q.shape[:2], torch.float32, "cuda")
    st = Guarded((len(lens), Hkv), torch.int32, "cuda")
    p.paged_sparse_decode_attn(out.t, q, dev(c["k"]), dev(c["v"]), gran, dev(c.get("kdev", c["ks"])),
                               dev(c.get("vdev", c["vs"])), dev(sel), dev(bt), dev(np.array(lens, np.int32)), 0.088,
                               lse_out=lse.t, unit_status=st.t)
    torch.cuda.synchronize()
    for x in (out, lse, st):
        x.check()
    assert int(st.t.abs().sum()) == 0
    sets = [[subset(c, bt[b], h, m, P, sel[b, h][sel[b, h] >= 0]) for h in range(Hkv)] for b, m in enumerate(lens)]
    check_rows(out.t.float().cpu().numpy().astype(np.float64), lse.t.cpu().numpy(), qv, sets, 0.088, f"{lens} {top}")


def test_sparse_over_all_pages_is_dense_decode():
    import torch
    p, rng, P = pf(), np.random.default_rng(6), 16
    lens = [777, 1, 4096]
    bt, c = filled(rng, lens, 2, P)
    top = 256
    sel = np.full((3, 2, top), -1, np.int32)
    for b, m in enumerate(lens):
        sel[b, :, :-(-m // P)] = np.arange(-(-m // P))
    q, qv = bf16(rng.standard_normal((3, 8, 128)))
    args = [dev(c["k"]), dev(c["v"]), p.SCALE_BLOCK, dev(c["ks"]), dev(c["vs"])]
    ld = dev(np.array(lens, np.int32))
    for sparse in (False, True):
        out, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")
        if sparse:
            p.paged_sparse_decode_attn(out, q, *args, dev(sel), dev(bt), ld, 0.088, lse_out=lse)
        else:
            p.paged_decode_attn_scaled(out, q, *args, dev(bt), ld, 0.088, lse_out=lse)
        sets = [[context(c, bt[b], h, m, P) for h in range(2)] for b, m in enumerate(lens)]
        check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, 0.088, f"sparse {sparse}")


def test_sparse_bad_entries_are_passed_over():
    import torch
    p, rng, P = pf(), np.random.default_rng(8), 16
    lens = [100, 100, 100, 100]
    bt, c = filled(rng, lens, 1, P)
    bad = bt.copy()
    bad[1, 2], bad[1, 3] = -1, 2 ** 31 - 1
    sel = np.array([[0, 7, 2 ** 31 - 1, 3], [1, 2, 3, -1], [-5, -1, -1, -1], [6, 0, 1, 2]], np.int32)[:, None]
    arg = np.array([100, 100, 100, 113], np.int32)  # the last is longer than its table: clamped to 112
    q, qv = bf16(rng.standard_normal((4, 8, 128)))
    out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    st = torch.empty((4, 1), dtype=torch.int32, device="cuda")
    c["v"][bt[3, 6]] = c["v"][bt[0, 1]]  # no NaN codes in the rows that the clamped length reaches
    c["k"][bt[3, 6]] = c["k"][bt[0, 1]]
    p.paged_sparse_decode_attn(out, q, dev(c["k"]), dev(c["v"]), p.SCALE_BLOCK, dev(c["ks"]), dev(c["vs"]), dev(sel),
                               dev(bad), dev(arg), 0.088, lse_out=lse, unit_status=st)
    torch.cuda.synchronize()
    E = p.DEVERR
    assert st.cpu().numpy().ravel().tolist() == [E["BAD_TOPK"], E["BAD_PAGE"], 0, E["BAD_CONTEXT"]]
    sets = [[subset(c, bt[0], 0, 100, P, [0, 3])], [subset(c, bt[1], 0, 100, P, [1])], [(np.zeros((0, 128)),) * 3],
            [subset(c, bt[3], 0, 112, P, [6, 0, 1, 2])]]
    check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, 0.088)


@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** 100])
def test_sparse_queries_of_any_size(size):
    import torch
    p, rng, P = pf(), np.random.default_rng(12), 16
    bt, c = filled(rng, [500], 2, P)
    sel = np.broadcast_to(np.arange(0, 32, 2, dtype=np.int32), (1, 2, 16)).copy()
    q, qv = bf16(rng.standard_normal((1, 8, 128)) * size)
    scale = float(np.float32(0.088 / size)) if size > 1 else 0.088
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    p.paged_sparse_decode_attn(out, q, dev(c["k"]), dev(c["v"]), p.SCALE_BLOCK, dev(c["ks"]), dev(c["vs"]), dev(sel),
                               dev(bt), dev(np.array([500], np.int32)), scale, lse_out=lse)
    sets = [[subset(c, bt[0], h, 500, P, sel[0, h]) for h in range(2)]]
    check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, scale)


# --------------------------------------------------------------- a decode step
def test_steps_of_append_bounds_select_attend():
    """Prompts, then decode steps with all the calls on one stream without a
    wait between them, eager and replayed from a graph on another stream."""
    import torch
    p, P, H, Hq, top = pf(), 16, 2, 8, 6
    lens = [150, 47, 300]
    full = [m + 8 for m in lens]
    st = State(31, full, H, 128, P)
    bnd = torch.zeros((st.pages, H, 2, 128), dtype=torch.int8, device="cuda")
    bs = torch.zeros((st.pages, H), device="cuda")
    rb, rs = bnd.cpu().numpy().copy(), bs.cpu().numpy().copy()
    bt = dev(st.bt)
    ctx, start = dev(np.array(lens, np.int32)), dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    sel = torch.empty((3, H, top), dtype=torch.int32, device="cuda")
    q, qv = bf16(st.rng.standard_normal((3, Hq, 128)))
    out, lse = torch.empty_like(q), torch.empty((3, Hq), device="cuda")
    stat = torch.full((2, 3, H), -1, dtype=torch.int32, device="cuda")
    scale = 2.0 ** -12
    kn = {x: torch.zeros((3, H, 128), dtype=torch.bfloat16, device="cuda") for x in "kv"}

    st.append(lens, lens)
    p.page_key_bounds(bnd, bs, st.g["k"].t, bt, ctx, start, max(lens))
    ref.bounds(st.ref["k"], rb, rs, st.bt, lens, start.cpu().numpy(), max(lens))
    start.copy_(dev(np.arange(4, dtype=np.int32)))

    def step():
        p.kv_append_fp8_block(kn["k"], kn["v"], st.g["k"].t, st.g["v"].t, st.s["k"].t, st.s["v"].t, bt, ctx, start, 1)
        p.page_key_bounds(bnd, bs, st.g["k"].t, bt, ctx, start, 1)
        p.select_pages(sel, q, bnd, bs, bt, ctx, P, 1, 1, k_scales=st.s["k"].t, unit_status=stat[0])
        p.paged_sparse_decode_attn(out, q, st.g["k"].t, st.g["v"].t, p.SCALE_BLOCK, st.s["k"].t, st.s["v"].t, sel, bt,
                                   ctx, scale, lse_out=lse, unit_status=stat[1])

    side = torch.cuda.Stream()
    graph = None
    for t in range(8):
        now = [m + t + 1 for m in lens]
        new = {}
        for x in "kv":
            r, rv = bf16(st.rng.standard_normal((3, H, 128)) * 2.0 ** (t - 3))
            kn[x].copy_(r)
            new[x] = rv
        qt, qv = bf16(st.rng.standard_normal((3, Hq, 128)))
        q.copy_(qt)
        ctx.copy_(dev(np.array(now, np.int32)))
        torch.cuda.synchronize()
        if t < 3:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for x in "kv":
            ref.append(new[x], st.ref[x], st.ref[x + "s"], st.bt, now, [0, 1, 2, 3], 1)
        st.check(f"step {t}")
        ref.bounds(st.ref["k"], rb, rs, st.bt, now, [0, 1, 2, 3], 1)
        assert np.array_equal(bnd.cpu().numpy(), rb) and np.array_equal(bs.cpu().numpy(), rs)
        want = ref.select(qv, rb, rs, st.ref["ks"], st.bt, now, P, top, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want)
        assert int(stat.abs().sum()) == 0
        c = {"k": st.ref["k"], "v": st.ref["v"], "ks": st.ref["ks"], "vs": st.ref["vs"]}
        sets = [[subset(c, st.bt[b], h, m, P, want[b, h][want[b, h] >= 0]) for h in range(H)] for b, m in enumerate(now)]
        check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, scale, f"step {t}")


def test_refusals_of_tensors_that_do_not_match():
    import torch
    p = pf()
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    q, bnd, bs = z(2, 8, 128, dt=torch.bfloat16), z(9, 2, 2, 128, dt=torch.int8), z(9, 2)
    bt, ctx, sel = z(2, 4, dt=torch.int32), z(2, dt=torch.int32), z(2, 2, 3, dt=torch.int32)
    k, start = z(9, 2, 16, 128, dt=torch.uint8), z(3, dt=torch.int32)
    good = dict(selected=sel, q=q, bounds=bnd, bound_scales=bs, block_tables=bt, context_lens=ctx, page_size=16)
    p.select_pages(**good)
    for name, t in (("selected", sel.long()), ("selected", sel[:, :1]), ("q", q.float()), ("bounds", bnd[:8]),
                    ("bounds", bnd.view(torch.uint8)), ("context_lens", ctx[:1]), ("block_tables", bt[:1]),
                    ("q", q.cpu()), ("k_scales", z(9)), ("unit_status", z(2, 3, dt=torch.int32)),
                    ("q", z(2, 128, 8, dt=torch.bfloat16).transpose(1, 2))):
        with pytest.raises(ValueError):
            p.select_pages(**{**good, name: t})
    with pytest.raises(p.PfkvError):
        p.select_pages(**good, sink_pages=2, recent_pages=2)
    good = dict(out=q.clone(), q=q, k_cache=k, v_cache=k, granularity=p.SCALE_BLOCK, k_scales=bs, v_scales=bs,
                selected=sel, block_tables=bt, context_lens=ctx, softmax_scale=0.1)
    p.paged_sparse_decode_attn(**good)
    for name, t in (("granularity", p.SCALE_HEAD), ("granularity", p.SCALE_TENSOR), ("k_scales", bs.double()),
                    ("v_cache", k[:8]), ("selected", sel[:, :1]), ("out", q.half()), ("lse_out", z(2, 7))):
        with pytest.raises(ValueError):
            p.paged_sparse_decode_attn(**{**good, name: t})
    for name, t in (("granularity", p.SCALE_TOKEN), ("granularity", 9), ("softmax_scale", 0.0)):
        with pytest.raises(p.PfkvError):
            p.paged_sparse_decode_attn(**{**good, name: t})
    x = z(5, 2, 128, dt=torch.bfloat16)
    good = dict(k_new=x, v_new=x, k_cache=k, v_cache=k.clone(), k_scales=bs, v_scales=bs.clone(), block_tables=bt,
                context_lens=ctx, new_start=start, max_new_len=1)
    p.kv_append_fp8_block(**good)
    for name, t in (("v_new", x[:4]), ("v_cache", None), ("k_cache", k.float()), ("new_start", start[:2]),
                    ("k_scales", z(9, 1)), ("k_new", x.float())):
        with pytest.raises(ValueError):
            p.kv_append_fp8_block(**{**good, name: t})
    good = dict(bounds=bnd, bound_scales=bs, k_cache=k, block_tables=bt, context_lens=ctx, new_start=start, max_new_len=1)
    p.page_key_bounds(**good)
    for name, t in (("bounds", z(9, 2, 128, dt=torch.int8)), ("bound_scales", z(9)), ("k_cache", k.float())):
        with pytest.raises(ValueError):
            p.page_key_bounds(**{**good, name: t})
    torch.cuda.synchronize()


def test_offsets_beyond_31_bits():
    """Pages at the far end of caches of 2.9 GB each: the same results as the
    same rows in a small pool."""
    import torch
    p, rng, H, P, pages = pf(), np.random.default_rng(23), 8, 64, 45000
    lens = [700, 65]
    n = [-(-m // P) for m in lens]
    small = {x: np.zeros((sum(n), H, P, 128), np.uint8) for x in "kv"}
    scales = {x: np.zeros((sum(n), H), np.float32) for x in "kv"}
    sbt = np.full((2, max(n)), -1, np.int32)
    sbt[0, :n[0]], sbt[1, :n[1]] = np.arange(n[0]), n[0] + np.arange(n[1])
    bt = np.where(sbt >= 0, pages - 1 - sbt, -1).astype(np.int32)
    start = np.array([0, 700, 765], np.int32)
    big = {x: torch.empty((pages, H, P, 128), dtype=torch.uint8, device="cuda") for x in "kv"}
    bsc = {x: torch.empty((pages, H), device="cuda") for x in "kv"}
    new = {x: bf16(rng.standard_normal((765, H, 128))) for x in "kv"}
    ctx = dev(np.array(lens, np.int32))
    p.kv_append_fp8_block(new["k"][0], new["v"][0], big["k"], big["v"], bsc["k"], bsc["v"], dev(bt), ctx, dev(start), 700)
    torch.cuda.synchronize()
    for x in "kv":
        ref.append(new[x][1], small[x], scales[x], sbt, lens, start, 700)
        for b in range(2):
            for i in range(n[b]):
                hi = min(P, lens[b] - i * P)
                got = big[x][int(bt[b, i])].cpu().numpy()
                assert np.array_equal(got[:, :hi], small[x][sbt[b, i], :, :hi])
                assert np.array_equal(bsc[x][int(bt[b, i])].cpu().numpy(), scales[x][sbt[b, i]])
    bnd, bs = torch.empty((pages, H, 2, 128), dtype=torch.int8, device="cuda"), torch.empty((pages, H), device="cuda")
    rb, rs = np.zeros((sum(n), H, 2, 128), np.int8), np.zeros((sum(n), H), np.float32)
    p.page_key_bounds(bnd, bs, big["k"], dev(bt), ctx, dev(start), 700)
    ref.bounds(small["k"], rb, rs, sbt, lens, start, 700)
    q, qv = bf16(rng.standard_normal((2, 64, 128)))
    sel = torch.empty((2, H, 4), dtype=torch.int32, device="cuda")
    p.select_pages(sel, q, bnd, bs, dev(bt), ctx, P, 1, 1, k_scales=bsc["k"])
    want = ref.select(qv, rb, rs, scales["k"], sbt, lens, P, 4, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)
    out, lse = torch.empty_like(q), torch.empty((2, 64), device="cuda")
    c = {"k": small["k"], "v": small["v"], "ks": scales["k"], "vs": scales["v"]}
    cache = (big["k"], big["v"], p.SCALE_BLOCK, bsc["k"], bsc["v"])
    p.paged_sparse_decode_attn(out, q, *cache, sel, dev(bt), ctx, 0.088, lse_out=lse)
    sets = [[subset(c, sbt[b], h, m, P, want[b, h][want[b, h] >= 0]) for h in range(H)] for b, m in enumerate(lens)]
    check_rows(out.double().cpu().numpy(), lse.cpu().numpy(), qv, sets, 0.088)
    for split in (0, 64):
        p.paged_decode_attn_scaled(out, q, *cache, dev(bt), ctx, 0.088, kv_split_tokens=split, lse_out=lse,
                                   max_total_chunks=13)
        sets = [[context(c, sbt[b], h, m, P) for h in range(H)] for b, m in enumerate(lens)]
        check_rows(out.double().cpu().numpy(), lse.cpu().numpy(), qv, sets, 0.088)
