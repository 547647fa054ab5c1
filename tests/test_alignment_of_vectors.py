"""Memory that kernels read or write in vectors is declared with their alignment.

Dynamic shared memory begins where its declaration lets the linker put it, behind whatever static shared memory a kernel
has: an array of 2- or 4-byte elements promises no more than their size.  Read from the sources.  Runs on CPU.
"""
import glob
import os
import re

import pytest

from submanifold_sparse_convolution_gb300 import build as build_mod

CSRC = os.path.join(os.path.dirname(os.path.abspath(build_mod.__file__)), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
DYNAMIC = re.compile(r"extern __shared__ (?:__align__\((\d+)\) )?\w+ (\w+)\[\];")


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_dynamic_shared_memory(path):
    text = open(path).read()
    assert len(DYNAMIC.findall(text)) == text.count("extern __shared__")
    for m in DYNAMIC.finditer(text):
        # 16 bytes, or moved up to 1024 by hand (tiles of the tensor cores)
        by_hand = any(form in text for form in (f"1024 - (ptx::smem_u32({m.group(2)}) & 1023)", "(1024 - (raw & 1023)) & 1023",
                                                f"(reinterpret_cast<uintptr_t>({m.group(2)}) + 1023) & ~uintptr_t(1023)"))
        assert int(m.group(1) or 0) >= 16 or by_hand, f"{m.group(0)} in {os.path.basename(path)}"


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_vector_store_to_an_array_of_smaller_elements(path):
    """A local array is aligned for its elements: vector stores go through values, or arrays declared for them."""
    text = open(path).read()
    arrays = set(re.findall(r"^\s+(?:u?int(?:8|16|32)_t|float|__nv_bfloat16) (\w+)\[[\w\s/*+]+\];", text, re.M))
    shared = set(re.findall(r"__shared__.* (\w+)\[", text))
    bad = [n for n in arrays - shared if re.search(rf"store_e4m3<\d>\(reinterpret_cast<uint8_t\*>\({n}\)|reinterpret_cast<(?:u?int|float)[24]\*>\({n}\) = ", text)]
    assert not bad, f"{bad} in {os.path.basename(path)}"
