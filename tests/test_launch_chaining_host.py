"""Kernels that start beside their predecessor (programmatic dependent launch),
checked in the sources: what such a kernel reads may still be written while it
is resident, so nothing goes through the read-only data path, which allows no
writer during the kernel's life.  A stale read cannot be provoked reliably, so
the rule itself is tested."""
import glob
import os
import re

import pytest

from sparse_long_context_02_b200 import build as dsa_build

CHAINED = sorted(f for f in glob.glob(os.path.join(dsa_build.CSRC, "*.cuh"))
                 if re.search(r"\bpdl_wait\(\);", open(f).read()))


def _code(path):
    """The source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_the_chained_sources_are_found():
    names = {os.path.basename(f) for f in CHAINED}
    assert {"decode.cuh", "kv8.cuh", "rope.cuh", "sparse_attn.cuh"} <= names


@pytest.mark.parametrize("path", CHAINED, ids=os.path.basename)
def test_no_read_only_loads_in_a_chained_kernel(path):
    code = _code(path)
    assert not re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc|const\s[^;()]*\*\s*__restrict__", code)


@pytest.mark.parametrize("path", CHAINED, ids=os.path.basename)
def test_a_chained_kernel_waits_before_it_releases_its_successor(path):
    """A kernel's end has to imply its predecessors', so every kernel of these
    files waits, and one that releases its successor early waits before."""
    for body in _code(path).split("__global__")[1:]:
        body = body[body.index("{"):]
        at = body.find("pdl_wait();")
        if at < 0:
            continue  # not launched by programmatic dependence
        early = body.find("pdl_launch_dependents();")
        assert early < 0 or at < early
        assert "return;" not in body[:at]
