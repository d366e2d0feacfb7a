"""The calls around the attention as a serving loop uses them: requests mapped
and forked in the page pool, pages copied before a fork writes, queries and keys
turned on their way into the cache, drafted tokens attended in one pass and
verified, lengths and pages cut to what stays, the pool compacted."""
import numpy as np
import pytest

import around_reference as ref
from gpu_helpers import assert_within_tolerance

pytestmark = pytest.mark.gpu

HQ, HKV, D, P, V, PAGES, ROW = 8, 2, 128, 16, 1000, 40, 8
FREQ = 10000.0 ** (-np.arange(64) / 64)
KS, VS, SM = 0.011, 0.013, D ** -0.5


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


class Model:
    """Rows of q, k, v per token from tables, and logits from the attention's
    output: enough of a model to have something to draft and verify."""

    def __init__(self, pf):
        import torch
        g = torch.Generator(device="cuda").manual_seed(1)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.q, self.k, self.v = (rand(V, n, D).bfloat16() for n in (HQ, HKV, HKV))
        self.w = rand(HQ * D, V) * 0.4
        self.rotary = pf.Rotary(FREQ)
        self.scales = [torch.tensor([s], dtype=torch.float32, device="cuda") for s in (KS, VS)]

    def probs(self, out):
        import torch
        return torch.softmax(out.flatten(1).float() @ self.w, 1)


class Loop:
    def __init__(self, pf):
        import torch
        self.pf, self.model = pf, Model(pf)
        self.pool = pf.PagePool(PAGES, P)
        self.cache = [torch.zeros(PAGES, HKV, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.arrays = pf.PagedArrays(self.cache)
        self.requests = []   # [tokens, row, tags]; the last token's rows are not in the cache yet
        self.rng = np.random.default_rng(2)

    def append(self, tokens, positions, slots, cache=None, q_out=None):
        import torch
        t = torch.as_tensor(np.asarray(tokens)).cuda()
        m, c = self.model, cache or self.cache
        q = None if q_out is None else m.q[t]
        self.pf.rotary_append_fp8(q_out, q, m.k[t], m.v[t], c[0], c[1], torch.as_tensor(np.asarray(slots, np.int64)).cuda(),
                                  torch.as_tensor(np.asarray(positions, np.int32)).cuda(), m.rotary, self.pf.SCALE_TENSOR, *m.scales)
        return q

    def admit(self, tokens):
        row, tags, cached = self.pool.map_request(np.array(tokens[:-1], np.int32), ROW)
        n = len(tokens) - 1 - cached
        if n:
            self.append(tokens[cached:-1], range(cached, cached + n), self.pf.slots_from_table(row, P, cached, n))
        self.requests.append([list(tokens), row, tags])

    def fork(self, i):
        tokens, row, tags = self.requests[i]
        self.pool.fork(row, int((row >= 0).sum()))
        self.requests.append([list(tokens), row.copy(), tags.copy()])

    def release(self, i):
        _, row, _ = self.requests.pop(i)
        self.pool.release(row, int((row >= 0).sum()))

    def copy(self, pairs):
        import torch
        if len(pairs):
            self.pf.copy_pages(self.arrays, torch.as_tensor(np.ascontiguousarray(pairs)).cuda())

    def compact(self):
        pairs, remap = self.pool.compact()
        self.copy(pairs)
        now = self.pool.page_tags()
        for _, row, tags in self.requests:
            held = row >= 0
            row[held] = remap[row[held]]
            tags[held] = now[row[held]]
        return len(pairs)

    def rows_are_right(self):
        """Every request's cached rows, through its table, against a cache of
        its own that holds its tokens in order."""
        import torch
        for tokens, row, _ in self.requests:
            n = len(tokens) - 1
            if n == 0:
                continue
            own = [torch.zeros(-(-n // P), HKV, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.append(tokens[:-1], range(n), range(n), own)
            pages = torch.as_tensor(row[:-(-n // P)].astype(np.int64)).cuda()
            for a, b in zip(self.cache, own):
                got, want = (x.transpose(1, 2).reshape(-1, HKV, D)[:n] for x in (a[pages], b))
                assert torch.equal(got, want)

    def step(self, drafts):
        """One verification pass with drafts[i] drafted tokens of request i."""
        import torch
        pf, B = self.pf, len(self.requests)
        new, pairs = [], []
        for (tokens, row, tags), n in zip(self.requests, drafts):
            guess = self.rng.integers(0, V, n).tolist()
            first = len(tokens) - 1
            self.pool.resize(row, tags, first + 1 + n)
            pairs.append(self.pool.make_writable(row, tags, first))
            new.append([tokens[-1]] + guess)
        self.copy(np.concatenate(pairs))
        for (tokens, row, _) in self.requests:   # written pages are the request's own
            assert all(self.pool.refcount(int(p)) == 1 for p in row[(len(tokens) - 1) // P:] if p >= 0)
        status = torch.empty(B, dtype=torch.int32, device="cuda")
        tables = torch.as_tensor(np.stack([r[1] for r in self.requests])).cuda()
        pf.verify_page_tags(tables, torch.as_tensor(np.stack([r[2] for r in self.requests]).view(np.int32)).cuda(),
                            torch.as_tensor(np.array([len(r[0]) + n for r, n in zip(self.requests, drafts)], np.int32)).cuda(), P,
                            torch.as_tensor(self.pool.page_tags().view(np.int32)).cuda(), status)
        assert status.tolist() == [0] * B
        flat = np.concatenate(new)
        start = np.concatenate([[0], np.cumsum([len(x) for x in new])]).astype(np.int32)
        pos = np.concatenate([np.arange(len(r[0]) - 1, len(r[0]) + n) for r, n in zip(self.requests, drafts)])
        slots = np.concatenate([pf.slots_from_table(r[1], P, len(r[0]) - 1, 1 + n) for r, n in zip(self.requests, drafts)])
        lens = torch.as_tensor(np.array([len(r[0]) + n for r, n in zip(self.requests, drafts)], np.int32)).cuda()
        T = len(flat)
        q_start = torch.as_tensor(start).cuda()
        before = [c.clone() for c in self.cache]
        q, q_out, out = self.model.q[torch.as_tensor(flat).cuda()], *(torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k, v = self.model.k[torch.as_tensor(flat).cuda()], self.model.v[torch.as_tensor(flat).cuda()]
        tokens = torch.as_tensor(flat.astype(np.int32)).cuda()
        d_slots, d_pos = torch.as_tensor(slots).cuda(), torch.as_tensor(pos.astype(np.int32)).cuda()
        g = torch.Generator(device="cuda").manual_seed(int(start[-1]))
        guess = torch.softmax(torch.randn(T, V, device="cuda", generator=g), 1)
        u = torch.rand(T, device="cuda", generator=g)
        u[::3] *= 0.001   # some drafts stay
        nxt, acc = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(256, pf.paged_prefill_workspace_size(B, HQ, HKV, 8, ROW * P)), dtype=torch.uint8, device="cuda")

        def run(cache, lens):
            pf.rotary_append_fp8(q_out, q, k, v, cache[0], cache[1], d_slots, d_pos, self.model.rotary, pf.SCALE_TENSOR,
                                 *self.model.scales)
            pf.paged_prefill_attn(out, q_out, cache[0], cache[1], tables, lens, q_start, 8, ROW * P, KS, VS, SM, workspace=ws)
            probs = self.model.probs(out)
            pf.verify_drafts(nxt, acc, probs, guess, tokens, u, q_start, context_lens=lens, request_status=status)
            return probs

        lens_in = lens.clone()
        probs = run(self.cache, lens)
        got = [x.clone() for x in (q_out, out, nxt, acc, lens, status)]
        # the same from a graph, on the cache as it was
        graph, graph_lens = torch.cuda.CUDAGraph(), lens_in.clone()
        with torch.cuda.graph(graph):
            run(before, graph_lens)
        for _ in range(2):
            graph_lens.copy_(lens_in)
            for x in (q_out, out, nxt, acc):
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (q_out, out, nxt, acc, graph_lens, status)))
            assert all(torch.equal(a, b) for a, b in zip(before, self.cache))
        # attention against 64 bits over the cached codes
        value = ref.e4m3_values()
        codes = [c.cpu().numpy() for c in self.cache]
        qf, of = q_out.float().cpu().numpy().astype(np.float64), out.float().cpu().numpy().astype(np.float64)
        want = np.zeros_like(of)
        for b, (toks, row, _) in enumerate(self.requests):
            L = len(toks) + drafts[b]
            at = row[np.arange(L) // P], np.arange(L) % P
            kf, vf = (value[c[at[0], :, at[1]]] * s for c, s in zip(codes, (KS, VS)))
            for i in range(start[b], start[b + 1]):
                seen = len(toks) + i - start[b]
                for h in range(HQ):
                    s = kf[:seen, h // (HQ // HKV)] @ qf[i, h] * SM
                    p = np.exp(s - s.max())
                    want[i, h] = p @ vf[:seen, h // (HQ // HKV)] / p.sum()
        assert_within_tolerance(of, want, "verification pass")
        # verification against whole-number arithmetic
        f = lambda t: t.float().cpu().numpy()
        w_next, w_acc, w_status, w_lens = ref.verify(f(probs), f(guess), flat, f(u), start, lens_in.cpu().numpy())
        assert np.array_equal(got[2].cpu().numpy(), w_next) and np.array_equal(got[3].cpu().numpy(), w_acc)
        assert np.array_equal(got[4].cpu().numpy(), w_lens) and not w_status.any() and status.tolist() == [0] * B
        for b, r in enumerate(self.requests):
            kept = int(w_acc[b])
            r[0] += [int(x) for x in w_next[start[b]:start[b] + kept + 1]]
            assert len(r[0]) - 1 == w_lens[b]
            self.pool.resize(r[1], r[2], len(r[0]) - 1)
        return w_acc


def test_fork_draft_verify_cut_compact(pf):
    loop = Loop(pf)
    shared = list(range(100, 140))
    loop.admit(shared + [5, 6, 7])
    loop.admit(shared + [8])
    loop.admit([9])
    loop.admit(list(range(300, 333)))
    loop.rows_are_right()
    loop.fork(0)
    loop.fork(0)
    loop.fork(3)
    accepted = []
    for drafts in ([3, 0, 7, 1, 3, 2, 4], [0, 5, 2, 7, 1, 1, 3], [7] * 7):
        accepted += loop.step(drafts).tolist()
        loop.rows_are_right()
    assert len(set(accepted)) > 2   # drafts stay and go
    loop.release(1)
    loop.release(0)
    loop.fork(1)
    assert loop.compact() > 0
    loop.rows_are_right()
    held = {int(p) for _, row, _ in loop.requests for p in row if p >= 0}
    assert held == set(range(len(held))) and loop.pool.num_free() == PAGES - len(held)
    loop.step([2, 3, 1, 0, 4, 6])
    loop.rows_are_right()
    while loop.requests:
        loop.release(0)
    assert loop.pool.num_free() == PAGES


def test_turned_keys_go_to_the_other_caches(pf):
    """rotary_embed before kv_append_fp8_block and kv_append_bf16: the turned
    keys are those rows, and the block append's codes come back to them."""
    import torch
    T, pages = 50, 5
    m = Model(pf)
    tok = torch.arange(T, device="cuda")
    turned = torch.empty(T, HKV, D, dtype=torch.bfloat16, device="cuda")
    pf.rotary_embed(turned, m.k[tok], tok.int(), m.rotary)
    cache = torch.zeros(pages, HKV, P, D, dtype=torch.bfloat16, device="cuda")
    pf.kv_append_bf16(turned, None, cache, None, tok)
    assert torch.equal(cache.transpose(1, 2).reshape(-1, HKV, D)[:T], turned)
    codes = torch.zeros(pages, HKV, P, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, HKV, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pf.kv_append_fp8_block(turned, None, codes, None, scales, None, i32(*range(pages))[None], i32(T), i32(0, T), T)
    want, _, _ = ref.turned(m.k[tok].double().cpu().numpy(), np.arange(T)[None], FREQ, np.zeros(64, int), 0, False)
    s = scales.double().cpu().numpy()[np.arange(T) // P][..., None]
    got = ref.e4m3_values()[codes.cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, HKV, D)[:T] * s
    # bf16's rounding, then e4m3's half step of the value over its scale; fp32's turn beside them
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 * 1.1 + ref.e4m3_half_step(want / s * (1 + 2.0 ** -7)) * s + 1e-6)
