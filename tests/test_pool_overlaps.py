"""Sizes and memory that the page operators refuse on the host, before any launch: outputs that overlap an input, the ring
or each other, and tables too wide to be counted."""
import pytest

from test_pool_host import FAKE, compact, fork, lib  # noqa: F401

# of test_pool_host's calls, 4096 bytes apart: 4 old and 4 new rows of 4 columns, 64 pages, a ring of 64
FORK_BYTES = dict(parents=16, past=16, held=16, table=64, ring=256, state=8, pinned=64, past_out=16, held_out=16, table_out=64,
                  copies=32, state_out=8, error=4)
FORK_OUT = ["ring", "past_out", "held_out", "table_out", "copies", "state_out", "error"]
COMPACT_BYTES = dict(held=16, table=64, ring=256, pinned=64, table_out=64, copies=64, state_out=8, end=4, error=4)
COMPACT_OUT = ["ring", "table_out", "copies", "state_out", "end", "error"]


def pairs(sizes, outs):
    return [(a, b) for a in outs for b in sizes if a != b]


def check(call, lib, sizes, a, b, short):  # noqa: F811
    at = FAKE + 4096 * 200  # where b is, past the workspace
    step = 8 if a == "copies" else 4
    last = (sizes[b] - 1) // step * step
    for offset in (0, last, step - sizes[a] if sizes[a] > step else 0):
        assert call(lib, ws_bytes=short, **{b: at, a: at + offset}) == 1, (a, b, offset)
    up = -(-sizes[b] // step) * step
    down = -(-sizes[a] // step) * step
    for offset in (up, -down):  # side by side: the workspace is what is refused
        assert call(lib, ws_bytes=short, **{b: at, a: at + offset}) == 3, (a, b, offset)


@pytest.mark.parametrize("a,b", pairs(FORK_BYTES, FORK_OUT))
def test_fork(lib, a, b):  # noqa: F811
    if b == "copies" and a != "copies":
        a, b = b, a
    check(fork, lib, FORK_BYTES, a, b, 16)


@pytest.mark.parametrize("a,b", pairs(COMPACT_BYTES, COMPACT_OUT))
def test_compact(lib, a, b):  # noqa: F811
    if b == "copies" and a != "copies":
        a, b = b, a
    if {a, b} == {"table", "table_out"}:
        return
    check(compact, lib, COMPACT_BYTES, a, b, 16)


def test_a_table_renamed_in_place_is_one(lib):  # noqa: F811
    at = FAKE + 4096 * 200
    assert compact(lib, ws_bytes=16, table=at, table_out=at) == 3
    for offset in (4, -4, 60, -60):
        assert compact(lib, ws_bytes=16, table=at, table_out=at + offset) == 1
    for offset in (64, -64):
        assert compact(lib, ws_bytes=16, table=at, table_out=at + offset) == 3


def test_the_workspace_is_the_calls_alone(lib):  # noqa: F811
    need = lib.pa_pool_workspace_size(64)
    for call, outs in ((fork, FORK_BYTES), (compact, COMPACT_BYTES)):
        for name in outs:
            assert call(lib, ws_bytes=16, **{"ws": FAKE + 4096 * 40, name: FAKE + 4096 * 40 + 64}) == 1, name
    assert fork(lib, ws_bytes=16, ws=FAKE + 4096 * 40, error=FAKE + 4096 * 40 + need) == 3


@pytest.mark.parametrize("columns", [(1 << 31) - 1, (1 << 31) - 256, (1 << 31) - 1024])
def test_rows_whose_columns_do_not_fit_32_bits_with_a_part_behind_them(lib, columns):  # noqa: F811
    """Columns are counted in parts of up to 256: those behind the last must have numbers too."""
    assert fork(lib, B=1, n=1, cols=columns, bs=1, ws_bytes=16) == 2
    assert fork(lib, B=0, n=1, cols=columns, bs=1, ws_bytes=16) == 2
    assert compact(lib, B=1, cols=columns, ws_bytes=16) == 2
    most = (1 << 31) - 1025
    assert fork(lib, B=0, n=0, cols=most, bs=1, ws_bytes=16) == 3
    assert compact(lib, B=0, cols=most, ws_bytes=16) == 3
