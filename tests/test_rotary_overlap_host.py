"""Which rows the rotary calls take for overlapping, on the host: rows of one
stride by where each of them lies, others by their whole extents (CPU only: the
calls that are in order fail for want of a device, with -3)."""

from test_around_host import refuses


def test_parts_of_one_buffer():
    """Rows beside each other in wider rows, against byte sets: 2 or 3 tokens of
    2 heads of 16 channels (64 bytes) in rows of 64 to 256 bytes."""
    refuses("""
    import itertools
    small = pf.Rotary([1.0] * 8)
    def bytes_of(at, stride, T):
        return {at + t * 2 * stride + i for t in range(T) for i in range(64)}
    seen = {NO: 0, BAD: 0}
    for T, stride in itertools.product((1, 2, 3), (32, 40, 64, 72, 128)):
        for off in range(-4 * 2 * stride, 4 * 2 * stride + 1, 16):
            out, x = 0x10000 + off, 0x10000
            same = off == 0
            want = NO if same or not bytes_of(out, stride, T) & bytes_of(x, stride, T) else BAD
            expect(embed, want, out=out, x=x, os=stride, xs=stride, T=T, H=2, D=16, r=small._ptr)
            seen[want] += 1
    assert min(seen.values()) > 50, seen
    # one token: the strides say nothing
    expect(embed, NO, out=0x10040, x=0x10000, os=4096, xs=32, T=1, H=2, D=16, r=small._ptr)
    # strides that differ: by extents
    expect(embed, BAD, out=0x10040, x=0x10000, os=72, xs=64, T=3, H=2, D=16, r=small._ptr)
    expect(embed, NO, out=0x10000 + 2 * 2 * 64 + 64, x=0x10000, os=72, xs=64, T=3, H=2, D=16, r=small._ptr)
    # queries of projections that stand in one row with keys and values, turned into a part behind them
    expect(append, NO, q=0x10000, qs=3200, qo=0x10000 + 2 * 1536, qos=3200, k=0x10000 + 2 * 1024, ks=3200, v=0x10000 + 2 * 1280, vs=3200)
    """)


def test_queries_over_keys_or_values_are_refused():
    """q_out is written while k_new and v_new are read."""
    refuses("""
    far, row = 0x900000, 3 * 2048
    for kv, step in (("k", "ks"), ("v", "vs")):
        expect(append, BAD, **{kv: 0x100000})
        expect(append, BAD, **{kv: 0x100000 + row - 16})
        expect(append, BAD, **{kv: 0x100000 - 3 * 512 + 16})
        expect(append, NO, **{kv: 0x100000 + row})
        expect(append, NO, **{kv: 0x100000 - 3 * 512})
        # one row of queries, keys and values: in place, and with the queries' output a head too far
        wide = dict(q=far, qs=1536, qo=far, qos=1536, k=far + 2048, ks=1536, v=far + 2560, vs=1536)
        expect(append, NO, **wide)
        expect(append, BAD, **dict(wide, **{kv: far + 2048 - 256}))
        expect(append, BAD, **dict(wide, **{kv: far + 2 * 1536 - 256}))     # the next token's first head
        expect(append, NO, **dict(wide, T=1, **{kv: far + 2 * 1536 - 256}))
        expect(append, BAD, **dict(wide, T=1, **{kv: far + 2048 - 256}))
        expect(append, BAD, **dict(wide, **{step: 1544}))   # another stride: by extents
        expect(append, NO, **dict(wide, T=1, **{step: 1544}))
    # no queries, nothing that is written over
    expect(append, NO, qo=None, q=None, k=0x100000)
    expect(append, NO, v=None, vc=None, sv=None, vs=0)
    """)
