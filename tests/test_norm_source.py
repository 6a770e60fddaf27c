"""Rules that the norms' kernels keep in their source, where no result would show a breach (CPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "equivariant_gnn_message_gb300", "csrc")


def _kernels(text):
    """name -> body of each __global__ function."""
    out = {}
    for m in re.finditer(r"__global__ void(?: __launch_bounds__\([^)]*\))? (\w+)\([^{]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out[m.group(1)] = text[m.end():i]
    return out


def test_kernels_wait_for_their_asynchronous_copies():
    """A kernel that feeds its rows by asynchronous copies drains them before it returns: the copies of the rows behind
    the last one write zeros into shared memory."""
    kernels = _kernels(open(os.path.join(CSRC, "norm_rows.cuh")).read())
    fed = {k: v for k, v in kernels.items() if "load_row()" in v}
    assert set(fed) == {"k_norm_rows", "k_norm_bwd_rows"}
    for name, body in fed.items():
        last = body.rindex("load_row();")
        assert "feed.drain();" in body[last:], name
        assert not re.search(r"\breturn\b", body[last:body.index("feed.drain();", last)]), name
