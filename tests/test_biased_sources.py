"""What the biased attention's kernels promise and no run can show: waits that give up cannot be brought about on
a healthy GPU, nor can rows of so many keys that computing them again takes as long as a wait may."""
import os
import re

import pytest

from test_step_sources import CSRC, kernel_body

KERNELS = [("biased.cu", "biased_rows_kernel"), ("biased_tile.cuh", "biased_tile_kernel")]


def body_of(file, name):
    with open(os.path.join(CSRC, file), encoding="utf-8") as f:
        return kernel_body(f.read(), name)


@pytest.mark.parametrize("file,name", KERNELS)
def test_time_outs_are_reported_after_every_wait(file, name):
    body = body_of(file, name)
    report = [m.start() for m in re.finditer(r"atomicOr\(a\.error, \*err\)", body)]
    last_wait = max(m.start() for m in re.finditer(r"mbar_wait\(", body))
    assert len(report) == 1 and report[0] > last_wait
    depth = body[:last_wait].count("{") - body[:last_wait].count("}")
    barrier = False
    for m in re.finditer(r"[{}]|__syncthreads\(\)", body[last_wait: report[0]]):
        depth += {"{": 1, "}": -1}.get(m.group(), 0)
        barrier = barrier or (m.group() == "__syncthreads()" and depth == 1)
    assert barrier


@pytest.mark.parametrize("file,name", KERNELS)
def test_rows_are_computed_again_when_no_warp_waits_any_more(file, name):
    """A row of many keys may take longer than the limit of a wait, so a warp that waits meanwhile would give up."""
    body = body_of(file, name)
    again = [m.start() for m in re.finditer(r"redo_row<", body)]
    assert again and min(again) > max(m.start() for m in re.finditer(r"mbar_wait\(|named_bar_sync\(", body))
