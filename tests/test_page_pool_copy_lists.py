"""Which pairs of the pool may stand in one list of copies, whose copies run at
the same time: pairs of one compact, or of make_writable calls without a fork, a
cut, a release or a compact between them (CPU only; pages are rows of numpy)."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as pf
    from paged_fp8_kv_02_gb300 import _build
    _build.build_pfkv()
    return pf


def conflicts(pairs):
    """A destination named twice, or one that is a source too."""
    src, dst = [p[0] for p in pairs], [p[1] for p in pairs]
    return len(set(dst)) < len(dst) or bool(set(src) & set(dst))


class Memory:
    """Pages of numbers, and requests that hold some through the pool."""

    def __init__(self, pf, pages, P, row, seed):
        self.pool, self.P, self.row = pf.PagePool(pages, P), P, row
        self.pages = np.full((pages, P), -1, np.int64)
        self.rng = np.random.default_rng(seed)
        self.requests = []   # [row, tags, contents]

    def copy(self, pairs):
        """One list: its copies in any order, each of two halves of a page."""
        pairs = [tuple(p) for p in np.asarray(pairs).reshape(-1, 2).tolist()]
        parts = [(s, d, h) for s, d in pairs for h in (slice(0, self.P // 2), slice(self.P // 2, None))]
        for i in self.rng.permutation(len(parts)):
            s, d, h = parts[i]
            self.pages[d, h] = self.pages[s, h]
        return pairs

    def write(self, r, first, new):
        for t, x in enumerate(new, first):
            self.pages[r[0][t // self.P], t % self.P] = x
        r[2][first:] = new

    def map(self, n):
        row, tags, _ = self.pool.map_request(self.rng.integers(0, 2 ** 30, n).astype(np.int32), self.row)
        self.requests.append([row, tags, []])
        self.write(self.requests[-1], 0, self.rng.integers(0, 1000, n).tolist())
        return self.requests[-1]

    def held(self, r):
        return -(-len(r[2]) // self.P)

    def fork(self, r):
        self.pool.fork(r[0], self.held(r))
        self.requests.append([r[0].copy(), r[1].copy(), list(r[2])])
        return self.requests[-1]

    def release(self, r):
        self.pool.release(r[0], self.held(r))
        self.requests = [x for x in self.requests if x is not r]

    def compact(self, moves=None):
        """-> its pairs; the copies are the caller's."""
        pairs, remap = self.pool.compact(moves)
        now = self.pool.page_tags()
        for row, tags, _ in self.requests:
            held = row >= 0
            row[held] = remap[row[held]]
            tags[held] = now[row[held]]
        return pairs

    def right(self):
        for row, _, contents in self.requests:
            got = [self.pages[row[t // self.P], t % self.P] for t in range(len(contents))]
            assert got == contents


@pytest.mark.parametrize("seed,P,pages", [(0, 4, 60), (1, 16, 40), (2, 2, 200), (3, 8, 90)])
def test_lists_of_a_loop(pf, seed, P, pages):
    """Many requests made writable, copied with one list, then written."""
    m = Memory(pf, pages, P, 10, seed)
    lists = 0
    for step in range(300):
        for _ in range(int(m.rng.integers(0, 6))):
            what = m.rng.choice(["map", "fork", "fork", "fork", "cut", "release", "compact"])
            if len(m.requests) > 8:
                what = "release"
            r = m.requests[int(m.rng.integers(len(m.requests)))] if m.requests else None
            try:
                if what == "map" or r is None:
                    m.map(int(m.rng.integers(1, 5 * P)))
                elif what == "fork":
                    m.fork(r)
                elif what == "cut":
                    n = int(m.rng.integers(1, len(r[2]) + 1))
                    m.pool.resize(r[0], r[1], n)
                    del r[2][n:]
                elif what == "release":
                    m.release(r)
                else:
                    pairs = m.copy(m.compact(int(m.rng.integers(0, pages))))
                    assert not conflicts(pairs)
            except pf.PfkvError as e:
                assert e.code == -6
            m.right()
        pairs, writes = [], []
        for i in m.rng.permutation(len(m.requests)):
            r = m.requests[i]
            first = int(m.rng.integers(0, len(r[2]) + 1))
            more = min(10 * P, len(r[2]) + int(m.rng.integers(0, 2 * P)))
            grown = len(r[2])
            try:   # grown before or after, as here and there
                if m.rng.random() < 0.5:
                    m.pool.resize(r[0], r[1], more)
                    grown = more
                pairs.append(m.pool.make_writable(r[0], r[1], first))
            except pf.PfkvError as e:
                assert e.code == -6
                m.pool.resize(r[0], r[1], len(r[2]))   # a cut: the list ends
                break
            try:
                m.pool.resize(r[0], r[1], more)
                grown = more
            except pf.PfkvError as e:
                assert e.code == -6
            more = grown
            writes.append((r, first, m.rng.integers(0, 1000, more - first).tolist()))
        pairs = m.copy(np.concatenate(pairs)) if pairs else []
        assert not conflicts(pairs)
        lists += len(pairs) > 1
        for r, first, new in writes:
            m.write(r, first, new)
        m.right()
    assert lists > 20


def test_a_compaction_and_a_fork_after_it_take_a_list_each(pf):
    """compact gives pages it has emptied back, lowest first, so that the next
    call may hand them out."""
    m = Memory(pf, 10, 4, 4, 0)
    first = m.map(4)
    m.fork(m.map(6))
    m.release(first)
    a = m.copy(m.compact())
    r = m.requests[-1]
    b = m.pool.make_writable(r[0], r[1], 6).tolist()
    assert conflicts(a + [tuple(p) for p in b])
    m.copy(b)
    m.write(r, 6, [5000])
    m.right()


def test_a_fork_of_a_fork_takes_a_list_of_its_own(pf):
    """The copy that the first list makes is the second's source."""
    m = Memory(pf, 10, 4, 4, 0)
    r = m.fork(m.map(6))
    a = m.pool.make_writable(r[0], r[1], 6).tolist()
    m.copy(a)
    s = m.fork(r)
    b = m.pool.make_writable(s[0], s[1], 6).tolist()
    assert conflicts([tuple(p) for p in a + b])
    m.copy(b)
    m.write(s, 6, [5000, 5001])
    m.right()
