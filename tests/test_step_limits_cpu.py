"""The limits that the header states for the operators around a step are those that the calls enforce (no CUDA device
needed: what is within them gets as far as the check for device memory)."""
import os
import re

import pytest

from beam_search_shared_gb300 import bsp, build
from test_step_cpu import INVALID, ROOT, UNSUPPORTED, Staged, advance, evict, process, select, weigh


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsp.load()


@pytest.fixture(scope="module")
def limit():
    text = open(os.path.join(ROOT, "include", "bsp.h")).read()
    found = dict(re.findall(r"#define (BSP_MAX_\w+) +([^/\n]+)", text))
    return lambda name: eval(found["BSP_MAX_" + name])  # noqa: S307 - a constant of this repository's header


def test_batches(lib, limit):
    for name, call in (("STEP_BATCH", select), ("STEP_BATCH", evict), ("WEIGHTS_BATCH", weigh)):
        n = limit(name)
        for batch, want in ((n, INVALID), (n + 1, UNSUPPORTED)):
            s = Staged(W=1, prefix=(1,) * batch, tail=(0,) * batch)
            assert call(lib, s.plan) == want, (name, call.__name__, batch)


def test_other_limits(lib, limit):
    s = Staged(tail=(0, 0))
    n = limit("VOCAB")
    for v, want in ((n, INVALID), (n + 1, UNSUPPORTED)):
        assert process(lib, s.plan, vocab=v, stride=n + 1, out_stride=n + 1) == want
        assert select(lib, s.plan, vocab=v, stride=n + 1) == want
    n = limit("CANDIDATES")
    assert select(lib, s.plan, num=n) == INVALID and select(lib, s.plan, num=n + 1) == UNSUPPORTED
    n = limit("ADVANCE_BEAMS")
    for w, want in ((n, INVALID), (n + 1, UNSUPPORTED)):
        assert advance(lib, Staged(W=w).plan, stride=n + 1) == want
