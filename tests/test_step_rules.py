"""The operators' launch rules, compiled by themselves and run on the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "varlen_paged_kv_gb300", "csrc")
WRAP = """
#include "rules.h"
extern "C" int64_t items(int64_t N, int64_t B, int64_t rows, int64_t full, int64_t one) {
  return pa::items_of_batch(N, B, rows, full, one);
}
extern "C" int cluster(int64_t items, int64_t slots, int64_t pieces, int least, int most) {
  return pa::cluster_size(items, slots, pieces, least, most);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(WRAP)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(d / "rules.cpp"), "-o", str(d / "rules.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "rules.so"))
    lib.items.restype = ctypes.c_int64
    lib.items.argtypes = [ctypes.c_int64] * 5
    lib.cluster.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    return lib


def test_batches_of_short_sequences_have_a_block_for_each(rules):
    """The blocks that a batch has, rows of different sequences in different ones, and those the rule counts."""
    r = np.random.default_rng(0)
    for _ in range(300):
        R = int(r.integers(1, 65))
        q = r.integers(1, int(r.integers(1, 200)) + 1, int(r.integers(1, 100)))
        real, counted = int((-(-q // R)).sum()), rules.items(int(q.sum()), len(q), R, 1, 1)
        assert real / 2 <= counted <= real  # (each sequence has less than one block more than its share of the rows)
    assert rules.items(64, 64, 16, 1, 1) == 64 and rules.items(8192, 4, 32, 1, 1) == 256 and rules.items(1, 64, 4, 1, 1) == 1
    assert rules.items(2 ** 31 - 1, 2 ** 29, 1, 64, 64) == 64 * (2 ** 31 - 1)


def test_clusters_are_no_more_than_run_at_once(rules):
    """64 one-row sequences of 8 KV heads called in blocks of 16 fill the 304 places by themselves."""
    assert rules.cluster(rules.items(64, 64, 16, 1, 1) * 8, 304, 32, 4, 8) == 1
    assert rules.cluster(8, 304, 32, 4, 8) == 8 and rules.cluster(64, 304, 32, 4, 8) == 4
    assert rules.cluster(8, 304, 31, 4, 8) == 4 and rules.cluster(1, 304, 7, 4, 8) == 1


def test_more_tiles_than_can_be_numbered_are_refused():
    """2^28 sequences of blocks of 15 tiles each: the grid would be taken for its low 32 bits."""
    import varlen_paged_kv_gb300 as pa
    from varlen_paged_kv_gb300 import build, step
    build.build()
    d = pa.PaSparseDims(16, 1 << 28, 68, 1, 64, 64, 64, 16, 0, 4, 15, 0, 1, 0, 68 * 64)
    p = 1 << 20  # aligned and never dereferenced: the call is refused before any launch
    assert step._library().pa_sparse_paged_attention(p, p, p, p, p, p, p, 0.0, p, None, d, None, None) == 2
