"""Loads of the serving operators' kernels."""

import os
import re

import pytest

import speculative_decoding_draft_stream_gb300 as ns

CSRC = os.path.join(os.path.dirname(ns.__file__), "csrc")
# the attention and cache kernels, which are launched in the ends of kernels that write what they read
FILES = sorted(f for f in os.listdir(CSRC)
               if re.match(r"ns_(paged|shared|pages|rotate|attn|prompt|umma_attn|umma_ptx|ptx)", f))


@pytest.mark.parametrize("name", FILES)
def test_no_load_that_wants_memory_to_be_read_only(name):
    """A kernel that begins before the writer of its inputs has ended may not read them as constant for its lifetime."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"\b__ldg\b|\bld\.global\.nc\b|\b__restrict__\b", text)


def test_the_kernels_are_there():
    assert {"ns_paged_mode.cuh", "ns_shared_attn.cuh", "ns_pages.cu", "ns_rotate.cu"} <= set(FILES)
