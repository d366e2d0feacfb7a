"""verify_drafts refuses arrays that it would write over one another or over
what it reads, on the host, before anything is enqueued."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


def test_arrays_that_are_written_stand_alone(pf):
    import torch
    counts = [3, 1, 4, 2]
    B, T, V = len(counts), sum(counts), 500
    g = torch.Generator(device="cuda").manual_seed(1)
    p, q = (torch.softmax(torch.randn(T, V, device="cuda", generator=g) * 3, 1) for _ in "pq")
    size = {"next": T, "accepted": B, "lens": B, "status": B, "tokens": T, "uniforms": T, "start": B + 1}
    names, gap = list(size), 64
    at = {n: gap + 64 * i for i, n in enumerate(names)}
    buf = torch.zeros(64 * 9, dtype=torch.int32, device="cuda")
    fill = {"tokens": torch.randint(0, V, (T,), device="cuda", generator=g).int(), "uniforms": torch.rand(T, device="cuda", generator=g).view(torch.int32),
            "start": torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda(),
            "lens": torch.full((B,), 50, dtype=torch.int32, device="cuda")}

    def call(at):
        buf.fill_(7)
        for n, x in fill.items():
            buf[at[n]:at[n] + size[n]] = x
        a = {n: buf[at[n]:at[n] + size[n]] for n in names}
        before = buf.clone()
        try:
            pf.verify_drafts(a["next"], a["accepted"], p, q, a["tokens"], a["uniforms"].view(torch.float32), a["start"],
                             context_lens=a["lens"], request_status=a["status"])
        except pf.PfkvError as e:
            assert e.code == -1 and "overlaps" in str(e)
            assert torch.equal(buf, before)
            return None
        return {n: a[n].clone() for n in names}

    good = call(at)
    assert good is not None
    for x, y in itertools.permutations(names, 2):
        if {"next", "accepted", "lens", "status"} & {x, y}:
            for off in (0, 1, size[y] - 1, 1 - size[x]):   # x from some place of y on, or with its end on y's first
                assert call(dict(at, **{x: at[y] + off})) is None, (x, y, off)
        # beside each other, all is as it was
        for off in (size[y], -size[x]):
            got = call(dict(at, **{x: at[y] + off}))
            assert got is not None and all(torch.equal(got[n], good[n]) for n in names), (x, y, off)
