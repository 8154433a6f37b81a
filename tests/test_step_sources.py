"""What the operators' kernels promise and no run can show: a pipeline wait that gives up cannot be brought
about on a healthy GPU, so the order of the statements that report it is read from the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "varlen_paged_kv_gb300", "csrc")


def kernel_body(text, name):
    """The body of a kernel, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    at = re.search(r"__global__[^;{]*\b" + name + r"\s*\(", text).end()
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at: i + 1]
    raise AssertionError(name)


def test_time_outs_are_reported_after_every_wait():
    """The word that a wait of any warp sets when it gives up is read by one thread, after a barrier of the whole
    block that follows every such wait of every warp."""
    text = open(os.path.join(CSRC, "sparse.cu"), encoding="utf-8").read()
    for name in ("sparse_rows_kernel", "sparse_tile_kernel"):
        body = kernel_body(text, name)
        report = [m.start() for m in re.finditer(r"atomicOr\(a\.error, \*err\)", body)]
        assert len(report) == 1, name
        last_wait = max(m.start() for m in re.finditer(r"mbar_wait\(", body))
        between = body[last_wait: report[0]]
        assert report[0] > last_wait
        # an unconditional barrier of the block: at the kernel's own depth of braces
        depth = body[:last_wait].count("{") - body[:last_wait].count("}")
        ok = False
        for m in re.finditer(r"[{}]|__syncthreads\(\)", between):
            if m.group() == "{":
                depth += 1
            elif m.group() == "}":
                depth -= 1
            else:
                ok = ok or depth == 1
        assert ok, name
