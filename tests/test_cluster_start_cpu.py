"""A block may write another block's shared memory only once that block runs,
which a barrier over the cluster guarantees and nothing else. Every kernel
that reaches into another block's shared memory has to pass one first."""

import os
import re

import pytest

from trellis_quantized_linear_rot_gb300 import build as b

REMOTE = r"map_shared_rank\("
BARRIER = r"cluster_wait\(\)|cluster\.sync\(\)|cluster\.barrier_wait\("


def bodies(text):
    """(name, body) of every kernel of a source without its comments."""
    text = re.sub(r"//[^\n]*|__launch_bounds__\([^)]*\)", "", text)
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\([^{};]*\)\s*{", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), text[m.end():end]


def begins_with_a_barrier(body):
    """Whether a barrier stands before the first remote access, in the
    kernel's own sequence of statements (not in a block of braces, which may
    be entered late or not at all)."""
    first = re.search(REMOTE, body)
    for m in re.finditer(BARRIER, body):
        depth = body[:m.start()].count("{") - body[:m.start()].count("}")
        if depth == 0 and m.start() < first.start():
            return True
    return False


def remote_kernels():
    out = []
    for src in sorted(os.listdir(b.CSRC)):
        if src.endswith((".cu", ".cuh")):
            with open(os.path.join(b.CSRC, src)) as f:
                out += [(src, name, body) for name, body in bodies(f.read()) if re.search(REMOTE, body)]
    return out


@pytest.mark.parametrize("src,name,body", remote_kernels(), ids=lambda x: x if len(x) < 60 else "")
def test_no_remote_access_before_the_cluster_runs(src, name, body):
    assert begins_with_a_barrier(body), "%s in %s" % (name, src)


def test_the_reader_finds_the_kernels_and_a_missing_barrier():
    assert "verify_draft_kernel" in [name for _, name, _ in remote_kernels()]
    good = "cluster_wait(); auto f = [&] { c.map_shared_rank(&x, 0)->y = 1; }; f(); cluster.sync(); }"
    assert begins_with_a_barrier(good)
    assert not begins_with_a_barrier(good.replace("cluster_wait(); ", ""))
    assert not begins_with_a_barrier("if (z) { cluster_wait(); } c.map_shared_rank(&x, 0); }")
