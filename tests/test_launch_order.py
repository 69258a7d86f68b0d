"""The programmatic launch protocol of kernels that use TMEM, read from their
sources: a kernel's dependents may start (and take all of an SM's TMEM in their
setup, before they wait for it) once every CTA of it has called
grid_dep_launch(), so a CTA calls that behind its own TMEM allocation."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rag_kv_cache_layer_gb300", "csrc")
ALLOC = re.compile(r"\btmem_alloc(?:_pair)?\s*\(|tcgen05\.alloc\b")


def closing(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    while True:
        depth += (text[at] == pair[0]) - (text[at] == pair[1])
        at += 1
        if depth == 0:
            return at


def functions():
    """(file, name, body without comments) of every kernel and device function."""
    out = []
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith(".cu"):
            continue
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, f)).read(), flags=re.S)
        for m in re.finditer(r"\bvoid\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            at = closing(text, m.end() - 1, "()")
            body = re.match(r"\s*\{", text[at:])
            if body:
                start = at + body.end() - 1
                out.append((f, m.group(1), text[start:closing(text, start, "{}")]))
    return out


USERS = [k for k in functions() if ALLOC.search(k[2])]


def test_the_kernels_that_allocate_are_found():
    assert {n for _, n, _ in USERS} >= {"gemm_body", "gemm_tc_kernel", "attn_tc_kernel", "mass_tc_kernel",
                                        "paged_chunk_kernel"}


@pytest.mark.parametrize("f,name,body", USERS, ids=[u[1] for u in USERS])
def test_dependents_start_after_the_allocation(f, name, body):
    if "grid_dep_launch();" not in body:
        return                                   # then the kernel's end starts them
    first = body.index("grid_dep_launch();")
    allocs = [m.end() for m in ALLOC.finditer(body)]
    assert max(allocs) < first, (f, name)
    # the allocating warp has returned from it: the block met in between
    assert "__syncthreads();" in body[max(allocs):first], (f, name)
