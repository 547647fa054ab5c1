"""Instructions that want the whole warp together come behind a point where it does come together.

PTX leaves an `.aligned` instruction undefined unless all threads of the warp execute it together.  The cluster barriers
and the allocation of tensor memory stand behind loops and branches of single lanes, so the functions that hold them
begin with ``__syncwarp()``.  Read from the sources: a violation may hang a GPU and is not run on one.  Runs on CPU.
"""
import glob
import os
import re

import pytest

from submanifold_sparse_convolution_gb300 import build as build_mod

CSRC = os.path.join(os.path.dirname(os.path.abspath(build_mod.__file__)), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
WANTED = re.compile(r"barrier\.cluster\.(arrive|wait)[.\w]*\.aligned|tcgen05\.(alloc|dealloc|relinquish_alloc_permit)[.:\w]*\.aligned")
FUNCTION = re.compile(r"^__device__ __forceinline__ \w+ (\w+)\([^)]*\) \{", re.M)


def bodies(text):
    """(name, body) of each device function that starts a line and ends at a brace that does."""
    for m in FUNCTION.finditer(text):
        line_end = text.index("\n", m.end())
        end = line_end if text[m.end():line_end].rstrip().endswith("}") else text.index("\n}", m.end())
        yield m.group(1), text[m.end():end]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_a_warp_comes_together_first(path):
    text = open(path).read()
    uses = WANTED.findall(text)
    held = 0
    for name, body in bodies(text):
        at = [m.start() for m in WANTED.finditer(body)]
        if not at:
            continue
        held += len(at)
        before = body[:body.index("asm")]
        assert before.strip().startswith("__syncwarp();"), f"{name} in {os.path.basename(path)}"
    assert held == len(uses), f"{os.path.basename(path)}: such an instruction outside of a function of its own"


def test_the_instructions_are_found():
    found = [m.group(0) for p in SOURCES for m in WANTED.finditer(open(p).read())]
    assert len(found) >= 10   # three of tensor memory, alone and for a pair, and the cluster barriers' halves
