"""Global memory is read coherently in every kernel.  A kernel is scheduled while the
one before it in the stream still runs (its first statement allows that and waits),
so any tensor it reads may be written during its life by that kernel: the
non-coherent path (ld.global.nc, __ldg), which holds only for data that nobody
writes meanwhile, reads none of them."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "normalisation_rope_transformers_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def code(path):
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_sources_are_found():
    assert len(SOURCES) >= 10


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_non_coherent_loads(path):
    bad = re.findall(r"__ldg\s*\(|ld\.global[\w.:]*\.nc\b", code(path))
    assert not bad, bad
