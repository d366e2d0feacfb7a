"""verify_drafts against whole-number arithmetic on the host: every output equal."""
import numpy as np
import pytest

import around_reference as ref
from guard_helpers import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


class Case:
    def __init__(self, counts, V, dtype="float32", draft=True, pad=0, seed=0, near=0.5):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        T = int(sum(counts))
        self.V, self.T = V, T
        self.q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        logits = torch.randn(T, V, device="cuda", generator=g) * 2
        dt = getattr(torch, dtype)
        self.p = torch.zeros(T, V + pad, dtype=dt, device="cuda")[:, :V]
        self.p.copy_(torch.softmax(logits, 1))
        self.q = None
        guess = torch.softmax(logits + torch.randn(T, V, device="cuda", generator=g) * near, 1)
        if draft:
            self.q = torch.zeros(T, V + 2 * pad, dtype=dt, device="cuda")[:, :V]
            self.q.copy_(guess)
        wait = torch.empty_like(guess).exponential_(generator=g)
        self.tokens = torch.roll((guess / wait).argmax(1), 1).int()
        self.u = torch.rand(T, device="cuda", generator=g)
        self.lens = torch.arange(50, 50 + len(counts), dtype=torch.int32, device="cuda") * 3

    def run(self, pf, stream=None, lens=True):
        import torch
        B = len(self.q_start) - 1
        nxt, acc = Guarded((max(self.T, 1),), torch.int32, "cuda"), Guarded((B,), torch.int32, "cuda")
        nxt.t.fill_(-7)
        status, new_lens = Guarded((B,), torch.int32, "cuda"), Guarded((B,), torch.int32, "cuda")
        new_lens.t.copy_(self.lens)
        pf.verify_drafts(nxt.t[:self.T], acc.t, self.p, self.q, self.tokens, self.u, torch.from_numpy(self.q_start).cuda(),
                         context_lens=new_lens.t if lens else None, request_status=status.t, stream=stream)
        torch.cuda.synchronize()
        for x in (nxt, acc, status, new_lens):
            x.check()
        return nxt.t[:self.T].cpu().numpy(), acc.t.cpu().numpy(), status.t.cpu().numpy(), new_lens.t.cpu().numpy()

    def want(self):
        h = lambda t: None if t is None else t.float().cpu().numpy()
        return ref.verify(h(self.p), h(self.q), self.tokens.cpu().numpy(), h(self.u), self.q_start, self.lens.cpu().numpy())

    def check(self, pf):
        got, want = self.run(pf), self.want()
        for name, a, b in zip(("next", "accepted", "status", "lens"), got, want):
            assert np.array_equal(a, b), (name, a, b)
        return got


COUNTS = {"one": [1], "two": [2], "eight": [8] * 5, "ragged": [1, 4, 0, 2, 9, 1, 3, 0], "long": [70, 33, 34, 1],
          "many": [1 + i % 4 for i in range(200)], "crowd": [1 + i % 2 for i in range(700)]}


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("V,pad", [(1, 0), (2, 1), (31, 0), (1000, 24), (1003, 0), (32003, 5)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("draft", [True, False])
def test_equal(pf, counts, V, pad, dtype, draft):
    Case(COUNTS[counts], V, dtype, draft, pad, seed=V + len(counts)).check(pf)


@pytest.mark.parametrize("V", [131072, 151937, 262144, 1 << 20])
@pytest.mark.parametrize("batch", [1, 3, 20])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_vocabularies(pf, V, batch, dtype):
    if V == 1 << 20 and batch > 3:
        batch = 5
    Case([1 + i % 3 for i in range(batch)], V, dtype, seed=V + batch).check(pf)


@pytest.mark.parametrize("dtype,pad,draft", [("float32", 0, True), ("float32", 1, True), ("float16", 3, False)])
def test_many_requests_of_the_largest_vocabulary(pf, dtype, pad, draft):
    """A CTA per request and as many blocks per warp as there can be.  The rows
    are two, over and over, so that the reference is two rows."""
    import torch
    B, V = 640, 1 << 20
    c = Case([1, 2], V, dtype, draft, seed=5)
    dt, row = c.p.dtype, V + pad
    p = torch.empty(B * row + 8, dtype=dt, device="cuda")[pad:pad + B * row].view(B, row)[:, :V]
    p[0::2], p[1::2] = c.p[0], c.p[1]
    q = None
    if draft:   # elsewhere in its 16 bytes than the target's rows
        q = torch.empty(B * (row + pad), dtype=dt, device="cuda").view(B, row + pad)[:, :V]
        q[0::2], q[1::2] = c.q[0], c.q[1]
    u = torch.rand(B, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    u[:6] = torch.tensor([0, 0, 2.0 ** -24, 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24])
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    for n in (1, 2):   # no drafts; one draft each, outside the vocabulary: always drawn from the first row less the draft's
        start = torch.arange(0, B + 1, n, dtype=torch.int32, device="cuda")
        nxt, acc, status = i32(B), i32(B // n), i32(B // n)
        pf.verify_drafts(nxt, acc, p, q, torch.full_like(nxt, V), u, start, request_status=status)
        f = lambda t: t.float().cpu().numpy()
        other = [np.zeros(V, np.float32)] * 2 if n == 1 or not draft else [f(c.q[0])] * 2
        sums = [np.cumsum(ref.weights(f(c.p[k]), other[k])) for k in (0, 1)]
        got, chance = nxt.cpu().numpy(), f(u)
        for b in range(B // n):
            total = sums[b * n % 2]
            bar = int(total[-1]) * int(chance[b * n + n - 1] * 2 ** 24) >> 24
            assert got[b * n] == np.searchsorted(total, bar, side="right"), (n, b)
        assert (got[1::2] == -1).all() or n == 1
        assert status.tolist() == [0 if n == 1 else pf.REQ_BAD_TOKEN] * (B // n) and not acc.any()


def test_the_accepted_vary(pf):
    """The cases above are no lot of all-or-nothing ones."""
    accepted = Case([8] * 200, 1000, seed=4, near=0.7).check(pf)[1]
    assert len(set(accepted.tolist())) == 8


def one(pf, p, q, tokens, u, **kw):
    import torch
    c = Case([len(tokens)], len(p[0]), draft=q is not None)
    c.p = torch.tensor(p, dtype=torch.float32, device="cuda")
    c.q = None if q is None else torch.tensor(q, dtype=torch.float32, device="cuda")
    c.tokens = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    c.u = torch.tensor(u, dtype=torch.float32, device="cuda")
    c.lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    nxt, acc, status, lens = c.check(pf)
    return nxt.tolist(), int(acc[0]), int(status[0]), int(lens[0])


def test_by_hand(pf):
    nan, inf = float("nan"), float("inf")
    p = [[0.5, 0.25, 0.25, 0.0], [0.0, 0.0, 0.0, 1.0]]
    q = [[0.25, 0.5, 0.25, 0.0], [0.25] * 4]
    # x = 1: u 0.5 < 0.25 fails at equality and above
    assert one(pf, p, q, [9, 1], [0.5, 0.0]) == ([0, -1], 0, 0, 99)
    assert one(pf, p, q, [9, 1], [0.499, 0.3]) == ([1, 3], 1, 0, 100)
    # only token 0 has residual mass
    assert one(pf, p, q, [9, 1], [0.9, 0.999]) == ([0, -1], 0, 0, 99)
    # p and q both 0 at the drafted token: it does not stay, and u = 0 draws the first word with mass
    assert one(pf, p, q, [9, 3], [0.0, 0.0]) == ([0, -1], 0, 0, 99)
    # a draft without a distribution: stays with probability p, else is left out of the draw
    assert one(pf, p, None, [9, 0], [0.49, 0.0]) == ([0, 3], 1, 0, 100)
    assert one(pf, p, None, [9, 0], [0.5, 0.0]) == ([1, -1], 0, 0, 99)
    assert one(pf, p, None, [9, 0], [0.5, 0.51]) == ([2, -1], 0, 0, 99)
    # equal rows: nothing is left, so the target's weights are taken
    assert one(pf, [[0.5, 0.5], [1, 0]], [[0.5, 1.0], [0, 1]], [0, 1], [0.9, 0.75]) == ([1, -1], 0, 0, 99)
    # no mass at all
    assert one(pf, [[0.0, 0.0], [0, 0]], [[0.5, 0.5], [0, 1]], [0, 1], [0.9, 0.75]) == ([-1, -1], 0, 8, 99)
    assert one(pf, [[nan, -1.0]], None, [0], [0.2]) == ([-1], 0, 8, 100)
    # NaN never accepts and has no weight; infinity counts as 1
    assert one(pf, [[nan, 0.5, 0.5], [1, 0, 0]], [[0.1, 0.4, 0.5], [0, 1, 0]], [0, 0], [0.0, 0.999]) == ([1, -1], 0, 0, 99)
    assert one(pf, [[0.5, 0.5, 0.0], [1, 0, 0]], [[0.1, nan, 0.1], [0, 1, 0]], [0, 1], [0.0, 0.999]) == ([0, -1], 0, 0, 99)
    assert one(pf, [[inf, 1.0]], None, [0], [0.49]) == ([0], 0, 0, 100)
    assert one(pf, [[inf, 1.0]], None, [0], [0.5]) == ([1], 0, 0, 100)
    # tokens outside the vocabulary
    assert one(pf, p, q, [0, 4], [0.0, 0.0])[1:3] == (0, 4)
    assert one(pf, p, None, [0, -1], [0.0, 0.6]) == ([1, -1], 0, 4, 99)
    assert one(pf, p, q, [0, 2 ** 31 - 1], [0.0, 0.0])[1:3] == (0, 4)


def test_borders_of_the_draw(pf):
    """Each word gets the uniforms of its own part: eight equal words."""
    p = [[0.125] * 8]
    for k in range(8):
        for u in (k / 8, np.nextafter(np.float32((k + 1) / 8), np.float32(0))):
            assert one(pf, p, None, [0], [float(u)])[0] == [k]
    # one word, far out, among 200,000
    import torch
    for at in (0, 1, 31, 32, 99999, 199999):
        c = Case([1], 200000, draft=False)
        c.p.zero_()
        c.p[0, at] = 2.0 ** -40
        for u in (0.0, 0.5, 1 - 2.0 ** -24):
            c.u.fill_(u)
            assert c.check(pf)[0].tolist() == [at]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pads", [(0, 0), (3, 3), (0, 1)])   # rows alike within 16 bytes, shifted alike, and not alike
@pytest.mark.parametrize("draft", [True, False])
def test_values_that_are_no_probabilities(pf, dtype, pads, draft):
    """NaN, infinities and negative numbers anywhere in the rows."""
    import torch
    for seed in range(4):
        c = Case([3] * 40, 5003, dtype, draft, seed=seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        for name, pad in zip("pq", pads):
            x = getattr(c, name)
            if x is None:
                continue
            y = torch.zeros(c.T, c.V + pad, dtype=x.dtype, device="cuda")[:, :c.V]
            y.copy_(x)
            odd = torch.tensor([float("nan"), float("inf"), -float("inf"), -1.0, 2.0, 1e-40, 1.0], device="cuda").to(x.dtype)
            at = torch.rand(c.T, c.V, device="cuda", generator=g) < (0.001, 0.2, 0.9, 0.0)[seed]
            which = torch.randint(0, len(odd), (c.T, c.V), device="cuda", generator=g)
            setattr(c, name, y)
            y.copy_(torch.where(at, odd[which], x))
        c.check(pf)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("pads", [(0, 0), (0, 1), (1, 0), (3, 3), (2, 5), (8, 1)])
@pytest.mark.parametrize("V", [7, 5003, 70001])
def test_nothing_left_but_the_target(pf, dtype, pads, V):
    """A draft twice the target everywhere: every draft goes, no weight is
    left, and the second reading is of the target's row alone, which may stand
    otherwise within its 16 bytes than both rows together."""
    import torch
    c = Case([1 + i % 4 for i in range(30)], V, dtype, seed=V)
    for name, pad in zip("pq", pads):
        y = torch.zeros(c.T, V + pad, dtype=c.p.dtype, device="cuda")[:, :V]
        y.copy_(c.p * (1 if name == "p" else 2))
        if name == "q":
            c.q = y
        else:
            p = y
    c.p = p
    c.u = c.u * 0.4 + 0.55
    _, accepted, status, _ = c.check(pf)
    assert not accepted.any() and not status.any()


def test_the_largest_sums(pf):
    """Every weight 1: the sums come to 2^62."""
    c = Case([1, 1, 1], 1 << 20, draft=False)
    c.p.fill_(1)
    c.p[1, ::2] = float("inf")
    c.u = c.u * 0 + c.u.new_tensor([0.0, 0.5, 1 - 2.0 ** -24])
    assert c.check(pf)[0].tolist() == [0, 1 << 19, (1 << 20) - 1]


def test_draws_follow_the_target(pf):
    """What comes out first is distributed as the target, whatever the draft:
    a chi-squared bound of 20,000 requests over 8 words (7 degrees of freedom;
    40 is passed with probability 1e-6)."""
    import torch
    B, V = 20000, 8
    c = Case([2] * B, V, seed=11)
    p = torch.softmax(torch.linspace(0, 2, V, device="cuda"), 0)
    q = torch.softmax(torch.linspace(1.5, 0, V, device="cuda"), 0)
    c.p.copy_(p.expand_as(c.p))
    c.q.copy_(q.expand_as(c.q))
    c.tokens = torch.multinomial(q, 2 * B, replacement=True, generator=torch.Generator(device="cuda").manual_seed(3)).int()
    nxt = c.run(pf)[0][0::2]
    count, expect = np.bincount(nxt, minlength=V), p.cpu().numpy().astype(np.float64) * B
    assert ((count - expect) ** 2 / expect).sum() < 40


def test_bad_q_start_leaves_rows_alone(pf):
    import torch
    c = Case([2, 3, 2, 2], 500, seed=6)
    # (starts whose good requests claim each row once)
    for change in ([4, 2, 5, 7, 9], [0, 2, 5, 7, 10], [-1, 2, 5, 7, 9], [0, 2, 5, 2 ** 31 - 1, 9], [9, 2, 5, 7, 9]):
        c.q_start = np.array(change, np.int32)
        c.check(pf)


def test_rows_behind_the_last_request_stay(pf):
    """A padded batch: rows and requests that are not there."""
    c = Case([2, 3, 2, 2], 500, seed=8)
    c.q_start = np.array([0, 2, 5, 5, 5], np.int32)
    nxt, acc, _, _ = c.check(pf)
    assert (nxt[5:] == -7).all() and (acc[2:] == 0).all()


def test_graph_replay_and_two_streams(pf):
    import torch
    c, d = Case([3] * 9, 5003, seed=1), Case([4, 1, 2], 40000, "bfloat16", seed=2)
    want = c.want()
    nxt, acc = torch.empty(c.T, dtype=torch.int32, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda")
    start = torch.from_numpy(c.q_start).cuda()
    lens = c.lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pf.verify_drafts(nxt, acc, c.p, c.q, c.tokens, c.u, start, context_lens=lens)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        lens.copy_(c.lens)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(nxt.cpu().numpy(), want[0]) and np.array_equal(lens.cpu().numpy(), want[3])
    for _ in range(10):
        a, b = c.run(pf, stream=s1), d.run(pf, stream=s2)
        assert all(np.array_equal(x, y) for x, y in zip(a, want))
        assert all(np.array_equal(x, y) for x, y in zip(b, d.want()))


def test_no_requests(pf):
    import torch
    z = lambda *s, dt=torch.int32: torch.empty(*s, dtype=dt, device="cuda")
    pf.verify_drafts(z(0), z(0), z(0, 10, dt=torch.float32), None, z(0), z(0, dt=torch.float32), z(1).zero_())
    acc = z(2).fill_(9)
    pf.verify_drafts(z(0), acc, z(0, 10, dt=torch.float32), None, z(0), z(0, dt=torch.float32), z(3).zero_())
    assert acc.tolist() == [0, 0]
