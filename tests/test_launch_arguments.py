"""What the operators' entries hand to their kernels is read there."""

import os
import re

import pytest

import speculative_decoding_draft_stream_gb300 as ns

CSRC = os.path.join(os.path.dirname(ns.__file__), "csrc")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def fields(struct):
    body = re.search(r"struct %s \{(.*?)\n\};" % struct, text("ns_ops.cuh"), re.S).group(1)
    for line in body.split(";"):
        for name in line.split(","):
            found = re.search(r"([A-Za-z_]\w*)\s*(?:\[[^\]]*\]\s*)*$", name.strip())
            if found:
                yield found.group(1)


@pytest.mark.parametrize("struct,seen", [("PagedAttnArgs", {"q", "kep8", "n_groups"}), ("RotateArgs", {"q", "ko_head"}),
                                         ("PromptAttnArgs", {"q", "err"}), ("LogprobArgs", {"logits", "err"})])
def test_every_field_is_read_beyond_the_entries(struct, seen):
    names = set(fields(struct))
    assert seen <= names
    kernels = "".join(text(f) for f in sorted(os.listdir(CSRC))
                      if f.startswith("ns_") and f not in ("ns_ops.cuh", "ns_ops_api.cu", "ns_binding.cpp"))
    assert [n for n in sorted(names) if not re.search(r"\.%s\b" % n, kernels)] == []
