"""Latent attention and eviction: what can be checked without a GPU beside the
argument checks of test_latent_host."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_kf_gb300", "csrc")


def _kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\(", text):
        at = text.index("{", m.end())
        depth = 0
        for i in range(at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            if depth == 0:
                yield m.group(1), text[at:i]
                break


def test_no_kernel_holds_tmem_while_it_waits_for_its_predecessor():
    """A kernel that may start before the one ahead of it has ended allocates TMEM after
    that wait: taken before, a predecessor that has yet to allocate could not end."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for kernel, body in _kernels(text):
            wait = body.rfind("griddepcontrol.wait")
            alloc = re.search(r"tmem_alloc2?\(", body)
            if wait >= 0 and alloc:
                seen += 1
                # (a wait inside a lambda is placed by its calls)
                calls = [m.start() for m in re.finditer(r"\bexpansion_done\(\)", body)]
                assert alloc.start() > max(calls + [wait]), (name, kernel)
    assert seen >= 2
