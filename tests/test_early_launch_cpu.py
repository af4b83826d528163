"""Sources of the kernels that may start before the stream's previous kernel has ended: they
must not promise the compiler that what they read stays constant while they run, since the
previous kernel may still be writing it when they start. That rules out the read-only load
path (ld.global.nc: __ldg, and what const __restrict__ pointers allow) and load intrinsics
that the compiler may move across the wait."""
import os
import re

import pytest

from exact_io_aware_27_gb300 import _build


def _sources():
    """Files that launch kernels early, and what they include."""
    text = {f: open(os.path.join(_build.CSRC, f)).read() for f in os.listdir(_build.CSRC)}
    todo = [f for f, t in text.items() if re.search(r"\blaunch_(early|as)\(", t)
            and '#include "fa_launch.h"' in t]
    assert len(todo) >= 5
    seen = set()
    while todo:
        f = todo.pop()
        if f in seen or f not in text:
            continue
        seen.add(f)
        todo += re.findall(r'#include "([^"]+)"', text[f])
    return {f: re.sub(r"//[^\n]*|/\*.*?\*/", "", text[f], flags=re.S) for f in sorted(seen)}


def test_the_sources_are_found():
    assert {"fa_packed_plan.cu", "fa_packed_forward.cu", "fa_packed_backward.cu", "fa_cache.cu",
            "fa_prefix.cu", "fa_forward.cuh", "fa_backward.cuh", "sm103.cuh"} <= set(_sources())


@pytest.mark.parametrize("pattern", [
    r"\b__ldg\s*\(", r"\b__ldc[asgv]\s*\(", r"\b__ldlu\s*\(", r"ld\.global\.nc",
    # a pointer to constant data that is also restricted
    r"\bconst\b[\w\s:]*\*\s*(?:const\s+)?__restrict__"])
def test_no_promise_of_constant_data(pattern):
    for f, text in _sources().items():
        hit = re.search(pattern, text)
        assert hit is None, f"{f}: {hit.group(0)!r}"
