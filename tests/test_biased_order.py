"""The rows kernel of the biased attention beside the tile kernel: what it reads before it has waited for any kernel.
That a load is served from a cache that nothing has made coherent cannot be brought about at will, so the order of the
statements is read from the source (test_biased_calls_gpu rewrites a call's inputs right before it)."""
import re

from test_biased_sources import body_of


def test_the_rows_kernel_reads_nothing_before_its_fence_or_wait_and_nothing_past_the_coherent_caches():
    body = body_of("biased.cu", "biased_rows_kernel")
    order = re.search(r"if \(a\.after_tiles\) acquire_earlier_kernels\(\);\s*else pdl_wait\(\);", body)
    assert order
    first_use = re.search(r"check_biased_batch\(|walk\.load\(|seq_at\(|a\.(cum|past|table|query|slopes|first|prefix)\s*\[", body)
    assert first_use.start() > order.end()
    depth = body[:order.start()].count("{") - body[:order.start()].count("}")
    assert depth == 1  # every thread comes by
    assert "__ldg" not in body and "ld.global.nc" not in body
    walk = body_of_struct("biased.cu", "BiWalk")
    assert "__ldg" not in walk


def body_of_struct(file, name):
    import os

    from test_step_sources import CSRC
    with open(os.path.join(CSRC, file), encoding="utf-8") as f:
        text = f.read()
    at = text.index("struct " + name)
    return text[at: text.index("\n};", at)]
