"""The sources that stored counters are tied to (no GPU)."""
import os
import re

from conftest import ROOT
from heterogeneous_adapter_batching_amd import profiling

CSRC = os.path.join(ROOT, "heterogeneous_adapter_batching_amd", "csrc")


def test_every_source_of_the_delta_kernels_counts():
    """Counters of the delta's kernels are void once a source of theirs
    changes: the headers that kernels.hip includes are sources too."""
    text = open(os.path.join(CSRC, "kernels.hip")).read()
    own = [f for f in re.findall(r'#include "([^"]+)"', text) if os.path.exists(os.path.join(CSRC, f))]
    assert "device_ops.h" in own and set(own) <= set(profiling._SOURCES)
