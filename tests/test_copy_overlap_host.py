"""copy_pages: its pairs are read while the status of pairs is written (CPU
only)."""
from test_around_host import refuses


def test_a_status_over_the_pairs_is_refused():
    refuses("""
    copy.__name__ = "copy_pages"
    far = ((0x900000, 4096, 4096),)
    for st in (0x10000, 0x10004, 0x10010 - 4, 0x10000 - 4):   # two pairs: 16 bytes, their status 8
        expect(copy, BAD, arrays=far, st=st)
    for st in (0x10010, 0x10000 - 8):
        expect(copy, NO, arrays=far, st=st)
    expect(copy, 0, arrays=far, np=0, st=0x10000)
    """)
