"""Scales per (page, KV head) on the GPU: kv_append_fp8_block bit for bit
against 64-bit numpy, and paged_decode_attn_scaled with SCALE_BLOCK within the
bound derived in block_reference.tolerance."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import pf
from guard_helpers import Guarded

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(x):
    """numpy float64 -> (device bf16 tensor, its values in float64)."""
    import torch
    t = torch.from_numpy(np.array(x, np.float32, order="C")).cuda().bfloat16()
    return t, t.float().cpu().numpy().astype(np.float64)


def tables(rng, lens, P, spare=2, width=None):
    n = [-(-int(m) // P) for m in lens]
    ids = rng.permutation(sum(n) + spare).astype(np.int32)
    bt = np.full((len(lens), width or max(max(n), 1)), -1, np.int32)
    at = 0
    for b, k in enumerate(n):
        bt[b, :k] = ids[at:at + k]
        at += k
    return bt, sum(n) + spare


def rows(rng, T, H, D):
    """Rows over 24 binades, some of zeros, some with -0."""
    x = rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-12, 12, (T, H, 1)))
    x[rng.random((T, H)) < 0.1] = 0.0
    x[rng.random((T, H, D)) < 0.02] = -0.0
    return x


class State:
    """Caches, scales and their numpy copies, filled by append calls."""

    def __init__(self, seed, lens, H, D, P, width=None):
        import torch
        self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        self.H, self.D, self.P = H, D, P
        self.bt, self.pages = tables(self.rng, lens, P, width=width)
        shape = (self.pages, H, P, D)
        self.ref, self.g, self.s = {}, {}, {}
        for x in "kv":
            self.ref[x] = self.rng.integers(0, 256, shape).astype(np.uint8)
            self.ref[x + "s"] = np.full((self.pages, H), np.nan, np.float32)
            self.g[x] = Guarded(shape, torch.uint8, "cuda")
            self.s[x] = Guarded((self.pages, H), torch.float32, "cuda")
            self.g[x].t.copy_(dev(self.ref[x]))
            self.s[x].t.copy_(dev(self.ref[x + "s"]))

    def append(self, new, upto, max_new=None, lens_arg=None, start=None, bt=None, v=True):
        """The last new[b] tokens of contexts of upto[b]."""
        p = pf()
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) if start is None else np.asarray(start, np.int32)
        upto = np.asarray(upto if lens_arg is None else lens_arg, np.int32)
        bt = self.bt if bt is None else bt
        max_new = max(new) if max_new is None else max_new
        T = int(np.sum(new))
        x = {c: bf16(rows(self.rng, T, self.H, self.D)) for c in ("kv" if v else "k")}
        args = [x["k"][0], x["v"][0] if v else None, self.g["k"].t, self.g["v"].t if v else None, self.s["k"].t,
                self.s["v"].t if v else None, dev(bt), dev(upto), dev(start), max_new]
        p.kv_append_fp8_block(*args)
        for c in x:
            ref.append(x[c][1], self.ref[c], self.ref[c + "s"], bt, upto, start, max_new)
        return args

    def check(self, what=""):
        for x in "kv":
            self.g[x].check(what)
            self.s[x].check(what)
            assert np.array_equal(self.g[x].t.cpu().numpy(), self.ref[x]), what
            assert np.array_equal(self.s[x].t.cpu().numpy().view(np.uint32), self.ref[x + "s"].view(np.uint32)), what


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("H,D,P", [(2, 128, 16), (1, 16, 16), (3, 64, 5), (2, 512, 48), (1, 128, 128), (48, 128, 1)])
def test_append_prompts_and_steps_bit_exact(H, D, P):
    lens = [1, P, P + 1, 3 * P - 1, 40]
    st = State(7 * P + D, [m + 7 for m in lens], H, D, P)
    st.append(lens, lens)
    st.check("prompts")
    for k in (1, 2, 4):  # steps of one, one, two tokens: pages begin, end and grow their scales
        st.append([max(1, k // 2)] * 5, [m + k for m in lens])
        st.check(f"step {k}")


def test_append_growth_is_exact_and_repeatable():
    """Rows of growing size into one page: every growth moves the earlier codes
    by powers of two; the same call again changes nothing."""
    import torch
    st = State(3, [16], 1, 128, 16)
    for t in range(16):
        x = st.rng.standard_normal((1, 1, 128)) * 4.0 ** (t - 8)
        k, kv = bf16(x)
        args = (k, k, st.g["k"].t, st.g["v"].t, st.s["k"].t, st.s["v"].t, dev(st.bt),
                dev(np.array([t + 1], np.int32)), dev(np.array([0, 1], np.int32)), 1)
        for _ in range(2):
            pf().kv_append_fp8_block(*args)
        for c in "kv":
            ref.append(kv, st.ref[c], st.ref[c + "s"], st.bt, [t + 1], [0, 1], 1)
        torch.cuda.synchronize()
        st.check(f"token {t}")


@pytest.mark.parametrize("amax", [0.0, 2.0 ** -133, 2.0 ** -118, 1.75, 1.7578125, 448.0, 450.0, 3.3895313892515355e38])
def test_append_scale_at_its_borders(amax):
    """Amaxes at and next to 448 times a power of two, subnormal ones and the
    largest bf16."""
    import torch
    st = State(5, [3], 1, 32, 16)
    x = np.zeros((3, 1, 32))
    x[1, 0, 5] = -amax
    k, kv = bf16(x)
    pf().kv_append_fp8_block(k, None, st.g["k"].t, None, st.s["k"].t, None, dev(st.bt), dev(st.lens),
                             dev(np.array([0, 3], np.int32)), 3)
    ref.append(kv, st.ref["k"], st.ref["ks"], st.bt, st.lens, [0, 3], 3)
    torch.cuda.synchronize()
    st.check(f"amax {amax}")


@pytest.mark.parametrize("bad", [np.nan, -1.0, 0.0])
def test_append_over_a_scale_that_is_none(bad):
    """Earlier rows whose scale was never written become zeros; the new rows
    and their scale are as on a fresh page."""
    import torch
    st = State(9, [20], 2, 128, 16)
    st.s["k"].t.fill_(bad)
    k, kv = bf16(st.rng.standard_normal((3, 2, 128)))
    pf().kv_append_fp8_block(k, None, st.g["k"].t, None, st.s["k"].t, None, dev(st.bt), dev(np.array([11], np.int32)),
                             dev(np.array([0, 3], np.int32)), 3)
    torch.cuda.synchronize()
    got, sc = st.g["k"].t.cpu().numpy(), st.s["k"].t.cpu().numpy()
    page = int(st.bt[0, 0])
    for h in range(2):
        s = ref.block_scale(float(np.abs(kv[:, h]).max()))
        assert sc[page, h] == s
        assert np.array_equal(got[page, h, 8:11], ref.encode(kv[:, h] / s))
        codes = st.ref["k"][page, h, :8]
        fine = (codes & 0x7F) != 0x7F
        assert np.all((got[page, h, :8] & 0x7F)[fine] == 0)


def test_append_leaves_out_what_does_not_fit():
    """Requests with impossible numbers and pages outside the pool are skipped,
    the others written; nothing else changes."""
    lens = [20, 33, 50, 17, 64, 5]
    st = State(11, lens, 2, 128, 16)
    st.append(lens, lens)
    st.check("prompts")
    new = [2, 3, 4, 5, 6, 5]
    st.append(new, lens, max_new=5)  # request 4 brings more than max_new_len
    st.check("too many")
    bad = list(lens)
    bad[0], bad[1], bad[3] = 1, st.bt.shape[1] * 16 + 1, -3  # shorter than its new part, beyond the table, negative
    st.append(new, lens, lens_arg=bad)
    st.check("lengths")
    bt = st.bt.copy()
    bt[2, 3], bt[1, 2], bt[5, 0] = -1, st.pages, 2 ** 31 - 1
    st.append(new, lens, bt=bt)
    st.check("pages")
    st.append(new, lens, start=[-4, 2, 5, 9, 9, 24, 30])  # starts before the rows, an empty part, ends past them
    st.check("starts")
    st.append([1, 1, 1, 1, 1, 1], lens, max_new=0)
    st.check("max_new_len 0")


def test_append_keys_alone_on_another_stream_and_in_a_graph():
    import torch
    st = State(13, [30, 47], 2, 128, 16)
    side = torch.cuda.Stream()
    st.append([30, 47], [30, 47])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        st.append([2, 1], [30, 47], v=False)
    side.synchronize()
    st.check("stream")
    args = st.append([1, 3], [30, 47])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pf().kv_append_fp8_block(*args)
    k, kv = bf16(rows(st.rng, 4, 2, 128) * 64)
    args[0].copy_(k)
    args[1].copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    for c in "kv":
        ref.append(kv, st.ref[c], st.ref[c + "s"], st.bt, [30, 47], [0, 1, 4], 3)
    st.check("graph")


# ------------------------------------------------------------------ decode
def filled(rng, lens, H, P, spread=4):
    """Caches of random codes (no NaN in attended rows, NaN codes past them)
    and power-of-two scales -> numpy arrays."""
    bt, pages = tables(rng, lens, P)
    out = {}
    for x in "kv":
        c = rng.integers(0, 256, (pages, H, P, 128)).astype(np.uint8)
        c[(c & 127) == 127] = 0x30
        c[(c & 127) > 0x70] -= 0x18  # a normal quantiser's codes are not all near the top
        out[x] = c
        out[x + "s"] = np.exp2(rng.integers(-8 - spread, -8, (pages, H))).astype(np.float32)
    for b, m in enumerate(lens):
        if m % P:
            for x in "kv":
                out[x][bt[b, m // P], :, m % P:] = 0x7F
    return bt, out


def context(c, bt_row, h, L, P):
    """Dequantised K, V rows of one head in float64, and each row's V scale."""
    n = -(-L // P)
    ids = bt_row[:n]
    return [(ref.VALUES[c[x][ids, h]] * c[x + "s"][ids, h].astype(np.float64)[:, None, None]).reshape(n * P, 128)[:L]
            for x in "kv"] + [np.repeat(c["vs"][ids, h].astype(np.float64), P)[:L]]


def check_rows(out, lse, q, sets, softmax_scale, what=""):
    """Rows (b, h) of a call against attend() over sets[b][h] = (keys, values,
    V scales)."""
    B, Hq, _ = q.shape
    Hkv = len(sets[0])
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            k, v, vs = sets[b][h]
            heads = slice(h * G, (h + 1) * G)
            if not len(k):
                assert np.all(out[b, heads] == 0) and np.all(np.isneginf(lse[b, heads])), (what, b, h)
                continue
            o, l, w, floor, ds = ref.attend(q[b, heads], k, v, softmax_scale, vs)
            excess = float((np.abs(out[b, heads] - o) / ref.tolerance(o, w, floor, ds)).max())
            assert excess <= 1, (what, b, h, excess)
            excess = float((np.abs(lse[b, heads] - l) / ref.lse_tolerance(l, ds)).max())
            assert excess <= 1, (what, "lse", b, h, excess)


def run_decode(p, rng, lens, Hq, Hkv, P, split=0, spread=4, width=0):
    import torch
    bt, c = filled(rng, lens, Hkv, P, spread)
    bt = np.pad(bt, ((0, 0), (0, max(0, width - bt.shape[1]))), constant_values=-1)
    q, qv = bf16(rng.standard_normal((len(lens), Hq, 128)) * np.exp2(rng.integers(-3, 2, (len(lens), Hq, 1))))
    out = Guarded(q.shape, torch.bfloat16, "cuda")
    lse = Guarded(q.shape[:2], torch.float32, "cuda")
    chunks = int(sum(-(-m // split) for m in lens)) if split else 0
    ws = p.paged_decode_attn_scaled(out.t, q, dev(c["k"]), dev(c["v"]), p.SCALE_BLOCK, dev(c["ks"]), dev(c["vs"]),
                                    dev(bt), dev(np.array(lens, np.int32)), 0.088, kv_split_tokens=split,
                                    lse_out=lse.t, max_total_chunks=chunks)
    torch.cuda.synchronize()
    assert p.workspace_status(ws) == 0
    out.check("out")
    lse.check("lse")
    sets = [[context(c, bt[b], h, m, P) for h in range(Hkv)] for b, m in enumerate(lens)]
    check_rows(out.t.float().cpu().numpy().astype(np.float64), lse.t.cpu().numpy(), qv, sets, 0.088, f"{lens} P {P}")


@pytest.mark.parametrize("Hq,Hkv,P,lens", [
    (8, 2, 16, (1, 16, 17, 300)), (16, 1, 64, (0, 130, 64, 5)), (4, 4, 48, (33, 96, 47, 100)), (20, 4, 128, (1000, 3)),
    (64, 8, 16, (2049, 257, 1, 31, 512)), (7, 1, 96, (5000,)), (32, 2, 16, tuple(range(0, 1200, 57))),
    (30, 15, 16, tuple(range(0, 900, 45)))])
@pytest.mark.parametrize("split", [0, 64])
def test_block_decode_matches_reference(Hq, Hkv, P, lens, split):
    run_decode(pf(), np.random.default_rng(Hq + P), list(lens), Hq, Hkv, P, split)


@pytest.mark.parametrize("width", [0, 4096])
def test_block_decode_scales_over_many_binades(width):
    run_decode(pf(), np.random.default_rng(1), [700, 1300], 16, 2, 16, 0, spread=20, width=width)


@pytest.mark.parametrize("Hq,Hkv,P,lens", [(8, 2, 16, (1, 0, 17, 3000)), (16, 1, 64, (1300, 64)), (48, 48, 16, (200,))])
def test_block_decode_by_table_width(Hq, Hkv, P, lens):
    """Narrow tables take one kernel, wide ones another: both at their borders."""
    for tokens in (0, 32768, 32784, (1 << 20) // (len(lens) * Hkv), (1 << 20) // (len(lens) * Hkv) + P):
        run_decode(pf(), np.random.default_rng(tokens), list(lens), Hq, Hkv, P, width=tokens // P)


@pytest.mark.parametrize("width", [3, 4096])
def test_block_decode_bad_page_reads_zeros(width):
    import torch
    p, rng, P = pf(), np.random.default_rng(2), 16
    bt, c = filled(rng, [40, 40], 1, P)
    bad = np.pad(bt, ((0, 0), (0, width - 3)), constant_values=-1)
    bad[0, 0], bad[1, 1] = -5, c["k"].shape[0] + 7
    q, qv = bf16(rng.standard_normal((2, 4, 128)))
    out = torch.empty_like(q)
    lse = torch.empty((2, 4), dtype=torch.float32, device="cuda")
    lens = dev(np.array([40, 40], np.int32))
    ws = p.paged_decode_attn_scaled(out, q, dev(c["k"]), dev(c["v"]), p.SCALE_BLOCK, dev(c["ks"]), dev(c["vs"]),
                                    dev(bad), lens, 0.088, lse_out=lse)
    torch.cuda.synchronize()
    assert p.workspace_status(ws) == p.DEVERR["BAD_PAGE"]
    sets = []
    for b, gap in ((0, slice(0, 16)), (1, slice(16, 32))):
        k, v, vs = context(c, bt[b], 0, 40, P)
        k[gap] = 0
        v[gap] = 0
        sets.append([(k, v, vs)])
    check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, 0.088, "bad page")


def test_block_decode_after_append_and_refusals():
    """Rows appended by the product, decoded by it; wrong scale shapes refused."""
    import torch
    p, P = pf(), 16
    lens = [33, 64, 100]
    st = State(21, lens, 2, 128, P)
    half = [m // 2 for m in lens]
    st.append(half, half)
    st.append([m - n for m, n in zip(lens, half)], lens)
    st.check()
    c = {"k": st.ref["k"], "v": st.ref["v"], "ks": st.ref["ks"], "vs": st.ref["vs"]}
    q, qv = bf16(st.rng.standard_normal((3, 8, 128)))
    out = torch.empty_like(q)
    lse = torch.empty((3, 8), dtype=torch.float32, device="cuda")
    scale = 2.0 ** -12  # the rows go up to 2^13: logits stay ordinary
    args = [out, q, st.g["k"].t, st.g["v"].t, p.SCALE_BLOCK, st.s["k"].t, st.s["v"].t, dev(st.bt), dev(st.lens), scale]
    p.paged_decode_attn_scaled(*args, lse_out=lse)
    sets = [[context(c, st.bt[b], h, m, P) for h in range(2)] for b, m in enumerate(lens)]
    check_rows(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), qv, sets, scale, "after append")
    for bad in (st.s["k"].t[:-1], st.s["k"].t.double(), torch.ones(2, device="cuda")):
        with pytest.raises(ValueError):
            p.paged_decode_attn_scaled(*args[:5], bad, *args[6:])
