"""Kernels whose CTAs write into each other's shared memory, read as source (no GPU needed): a wait that
gives up in one CTA must not let it go while another may still send to it.  After the cluster's CTAs
have met first, the warps that may meet at its last barrier (all of them, or those of one role: threads
that have left count as arrived) come to it on every path; only a warp that has seen the last of what
can be sent to it may pass it by.
"""
import os
import re

import pytest

import sparse_top_lookup_gb300 as pk

CSRC = os.path.join(os.path.dirname(pk.__file__), "csrc")


def block(text, at):
    """The text of the braces that open at or after `at`, and where they end."""
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i], i + 1
    raise AssertionError("unbalanced braces")


def kernels():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)\s*)?"
                             r"(\w+)\s*\(", text):
            if re.match(r"[^;{]*\{", text[m.end():]):
                yield name, m.group(1), block(text, m.end())[0]


def without_lambdas(body):
    while True:
        m = re.search(r"\[&?\]\s*(\([^()]*(\([^()]*\)[^()]*)*\))?\s*(->\s*\w+\s*)?\{", body)
        if not m:
            return body
        _, end = block(body, m.start())
        body = body[:m.start()] + body[end:]


CLUSTERS = [(f, k, b) for f, k, b in kernels() if "cluster_sync()" in b]


def test_there_are_cluster_kernels():
    assert {"distill_stream_kernel", "ffn_gemm_kernel", "ffn_few_kernel"} <= {k for _, k, _ in CLUSTERS}


@pytest.mark.parametrize("body", [b for _, _, b in CLUSTERS], ids=[k for _, k, _ in CLUSTERS])
def test_every_path_of_those_that_stay_ends_at_the_clusters_last_barrier(body):
    body = without_lambdas(body)
    assert body.count("cluster_sync()") >= 2
    last = body.rindex("cluster_sync()")
    depth, start = 0, last            # the innermost block that holds it
    while start > 0 and depth >= 0:
        start -= 1
        depth += {"}": 1, "{": -1}.get(body[start], 0)
    between = body[max(start, body.index("cluster_sync()")):last]
    assert not re.search(r"\breturn\b", between)


# what each kernel's copies signal: on its way out a warp that gave up waits (with a limit) for these too
COPIES = [("ffn_few.cu", "ffn_few_kernel", ["bar_full", "bar_done"]),  # (bar_done: its MMAs)
          ("ffn.cu", "ffn_gemm_kernel", ["bar_full", "bar_set|bar_done \\+ 8u"]),
          ("distill.cu", "distill_stream_kernel", ["bar_full", "bar_sums"]),
          ("lookup_2sm.cu", "select_2sm_kernel", ["bar_full"]),
          ("qnet.cu", "qnet2_kernel", ["bar_full"])]


@pytest.mark.parametrize("name,kernel,barriers", COPIES, ids=[k for _, k, _ in COPIES])
def test_copies_on_their_way_are_waited_for(name, kernel, barriers):
    body = {(f, k): b for f, k, b in kernels()}[name, kernel]
    for b in barriers:
        assert re.search(r"wait_phase_drain\([^;]*(%s)" % b, body), b
