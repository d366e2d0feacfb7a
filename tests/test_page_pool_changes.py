"""Requests that fork, grow, shrink and move in the host page pool: the library
against the oracle on seeded random sequences, and what the sequences must keep
(CPU only; no CUDA call)."""
import ctypes

import numpy as np
import pytest

from oracle import page_pool as op


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as pf
    from paged_fp8_kv_02_gb300 import _build
    _build.build_pfkv()
    return pf


def same(lib, ref):
    assert lib.num_free() == len(ref.free)
    assert [lib.refcount(p) for p in range(lib.num_pages)] == ref.ref
    assert lib.page_tags().tolist() == ref.tag


@pytest.mark.parametrize("seed,P,num_pages", [(0, 16, 60), (1, 4, 200), (2, 1, 90), (3, 64, 40)])
def test_random_sequences_match_the_oracle(pf, seed, P, num_pages):
    rng = np.random.default_rng(seed)
    max_pages = 12
    lib, ref = pf.PagePool(num_pages, P), op.PagePool(num_pages, P)
    prefixes = [rng.integers(0, 50, int(rng.integers(0, 5 * P))).tolist() for _ in range(3)]
    live = []   # [row, tags, length, oracle row, oracle tags]

    def both(f, g):
        """The library's and the oracle's answer, or an error of both."""
        try:
            want = g()
        except (op.NoPages, ValueError):
            with pytest.raises(pf.PfkvError):
                f()
            return None
        return f(), want

    for step in range(400):
        what = rng.choice(["map", "release", "fork", "grow", "cut", "write", "compact"], p=[.2, .15, .15, .2, .1, .15, .05])
        if what == "map" or not live:
            toks = (prefixes[int(rng.integers(3))] + rng.integers(0, 50, int(rng.integers(0, 3 * P))).tolist())[:max_pages * P]
            got = both(lambda: lib.map_request(np.array(toks, np.int32), max_pages), lambda: ref.map_request(toks, max_pages))
            if got:
                (row, tags, _), (rrow, rtags, _) = got
                live.append([row, tags, len(toks), rrow, rtags])
        elif what == "compact":
            moves = int(rng.integers(0, num_pages + 5))
            pairs, remap = lib.compact(moves)
            rpairs, rremap = ref.compact(moves)
            assert [tuple(p) for p in pairs.tolist()] == rpairs and remap.tolist() == rremap
            assert not set(pairs[:, 0].tolist()) & set(pairs[:, 1].tolist()) and len(set(pairs.ravel().tolist())) == 2 * len(pairs)
            now = lib.page_tags()
            for r in live:
                held = r[0] >= 0
                moved = held & (remap[np.where(held, r[0], 0)] != r[0])
                r[0][held] = remap[r[0][held]]
                r[1][moved] = now[r[0][moved]]
                r[3] = [rremap[p] if p >= 0 else p for p in r[3]]
                r[4] = [ref.tag[p] if m else t for p, t, m in zip(r[3], r[4], moved)]
        else:
            k = int(rng.integers(len(live)))
            row, tags, n, rrow, rtags = live[k]
            if what == "release":
                lib.release(row, -(-n // P))
                ref.release(rrow, -(-n // P))
                live.pop(k)
            elif what == "fork":
                lib.fork(row, -(-n // P))
                ref.fork(rrow, -(-n // P))
                live.append([row.copy(), tags.copy(), n, list(rrow), list(rtags)])
            elif what == "write":
                first = int(rng.integers(0, n + 1))
                got = both(lambda: lib.make_writable(row, tags, first), lambda: ref.make_writable(rrow, rtags, first))
                if got:
                    assert [tuple(p) for p in got[0].tolist()] == got[1]
                    assert all(lib.refcount(int(p)) == 1 for p in row[first // P:-(-n // P)])
                    if got[1]:
                        assert got[1][0][1] == row[first // P] and first % P
            else:
                m = int(rng.integers(n, max_pages * P + 4)) if what == "grow" else int(rng.integers(0, n + 1))
                if both(lambda: lib.resize(row, tags, m), lambda: ref.resize(rrow, rtags, m)) is not None:
                    live[k][2] = m
        same(lib, ref)
        for row, tags, n, rrow, rtags in live:
            assert row.tolist() == rrow and tags.tolist() == rtags, (step, what)
            held = -(-n // P)
            assert (row[:held] >= 0).all() and (row[held:] == -1).all()
            assert np.array_equal(tags[:held], lib.page_tags()[row[:held]])   # every entry verifies
    for row, _, n, _, _ in live:
        lib.release(row, -(-n // P))
    assert lib.num_free() == num_pages


def test_a_fork_writes_only_its_own_page(pf):
    """Two forks of a 10-token request with pages of 4: the pages of tokens 0-7
    stay shared, each fork but the last holder gets a copy of the third page."""
    pool = pf.PagePool(20, 4)
    row, tags, _ = pool.map_request(np.arange(10, dtype=np.int32), 6)
    a, at, b, bt = row.copy(), tags.copy(), row.copy(), tags.copy()
    pool.fork(row, 3)
    pool.fork(row, 3)
    assert [pool.refcount(int(p)) for p in row[:3]] == [3, 3, 3]
    pa, pb, p0 = pool.make_writable(a, at, 10), pool.make_writable(b, bt, 10), pool.make_writable(row, tags, 10)
    assert pa.tolist() == [[row[2], a[2]]] and pb.tolist() == [[row[2], b[2]]] and p0.shape == (0, 2)
    assert len({int(row[2]), int(a[2]), int(b[2])}) == 3
    assert np.array_equal(a[:2], row[:2]) and [pool.refcount(int(p)) for p in row[:3]] == [3, 3, 1]
    # a fork at a page's border shares everything and copies nothing
    pool.resize(a, at, 13)
    assert (a[3] >= 0) and pool.make_writable(a, at, 12).shape == (0, 2)


def test_a_cut_page_leaves_the_prefix_table(pf):
    pool = pf.PagePool(20, 4)
    toks = np.arange(8, dtype=np.int32)
    row, tags, _ = pool.map_request(toks, 4)
    pool.resize(row, tags, 6)
    pool.make_writable(row, tags, 6)   # other tokens come behind the sixth
    _, _, cached = pool.map_request(toks, 4)
    assert cached == 4


def test_a_moved_page_is_still_found_by_its_hash(pf):
    pool = pf.PagePool(20, 4)
    first, _, _ = pool.map_request(np.arange(100, 112, dtype=np.int32), 4)
    toks = np.arange(8, dtype=np.int32)
    row, _, _ = pool.map_request(toks, 4)
    pool.release(first, 3)
    pairs, remap = pool.compact()
    assert sorted(remap[row[:2]].tolist()) == [0, 1] and len(pairs) == 2
    again, _, cached = pool.map_request(toks, 4)
    assert cached == 8 and np.array_equal(again[:2], remap[row[:2]])
    assert pool.compact()[0].shape == (0, 2)
    assert pool.compact(0)[0].shape == (0, 2)


def test_refusals_change_nothing(pf):
    pool = pf.PagePool(6, 4)
    row, tags, _ = pool.map_request(np.arange(10, dtype=np.int32), 8)
    shared, stags = row.copy(), tags.copy()
    pool.fork(row, 3)
    before = ([pool.refcount(p) for p in range(6)], pool.page_tags().tolist(), row.tolist(), tags.tolist())
    bad = row.copy()
    bad[1] = 5   # not held
    twice = np.array([row[0], row[0], row[0], -1], np.int32)   # held by two
    far = np.array([99, -1], np.int32)
    for call in (lambda: pool.fork(bad, 2), lambda: pool.fork(row, 4), lambda: pool.resize(row, tags, 40),
                 lambda: pool.resize(row, tags, 28), lambda: pool.resize(bad, tags, 20), lambda: pool.resize(row, tags, -1),
                 lambda: pool.resize(twice, np.zeros(4, np.uint32), 4), lambda: pool.resize(far, np.zeros(2, np.uint32), 0),
                 lambda: pool.make_writable(bad, tags, 0), lambda: pool.make_writable(row, tags, -1), lambda: pool.compact(-1)):
        with pytest.raises(pf.PfkvError):
            call()
    pool.resize(shared, stags, 24)   # the last three pages
    with pytest.raises(pf.PfkvError) as e:
        pool.make_writable(row, tags, 0)
    assert e.value.code == -6
    pool.resize(shared, stags, 10)
    assert before == ([pool.refcount(p) for p in range(6)], [t for t in before[1]], row.tolist(), tags.tolist())
    for r, t in ((row.tolist(), tags), (row.astype(np.int64), tags), (row, tags[:3]), (row[::2], tags[::2]), (row, tags.astype(np.int32))):
        with pytest.raises(ValueError):
            pool.resize(r, t, 4)
        with pytest.raises(ValueError):
            pool.make_writable(r, t, 4)
    for n in (-1, 9):
        with pytest.raises(ValueError):
            pool.fork(row, n)
    with pytest.raises(ValueError):
        pool.resize(row, tags, 2 ** 32 + 4)


def test_null_pointers(pf):
    lib = pf.load()
    h = lib.pfkv_pool_create(4, 4)
    one = (ctypes.c_int32 * 8)()
    for rc in (lib.pfkv_pool_fork(None, one, 1), lib.pfkv_pool_fork(h, None, 1), lib.pfkv_pool_fork(h, one, -1),
               lib.pfkv_pool_resize(None, one, one, 4, 1), lib.pfkv_pool_resize(h, None, one, 4, 1),
               lib.pfkv_pool_resize(h, one, None, 4, 1), lib.pfkv_pool_resize(h, one, one, 0, 1),
               lib.pfkv_pool_make_writable(h, one, one, 4, 0, None, one), lib.pfkv_pool_make_writable(h, one, one, 4, 0, one, None),
               lib.pfkv_pool_make_writable(None, one, one, 4, 0, one, one),
               lib.pfkv_pool_compact(h, 1, None, one, one), lib.pfkv_pool_compact(h, 1, one, None, one),
               lib.pfkv_pool_compact(h, 1, one, one, None), lib.pfkv_pool_compact(None, 1, one, one, one)):
        assert rc == -1
    lib.pfkv_pool_destroy(h)
