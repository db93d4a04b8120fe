"""Kernels that may start while the launch before them still writes their inputs
(wait_for_launch_before) read by ordinary loads: the read-only path is for data that nothing
writes while the kernel lives, and no ordering of memory holds such a load back."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_57_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_early_kernels_use_no_read_only_loads():
    early = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "wait_for_launch_before()" in _source(n)]
    assert {"cache_rw.cu", "decode_int4.cu"} <= set(early)
    seen, todo = set(), list(early)
    while todo:  # and the headers they take in
        n = todo.pop()
        if n in seen or not os.path.exists(os.path.join(CSRC, n)):
            continue
        seen.add(n)
        todo += re.findall(r'#include "([^"]+)"', _source(n))
    bad = [n for n in sorted(seen) if READ_ONLY.search(_source(n))]
    assert not bad, f"read-only loads in {bad}"
