"""Kernels launched with programmatic stream serialisation may start while the kernel before them runs.  What that one
writes is visible behind their wait to plain loads; a load through the read-only path asks for data that nobody writes while
the kernel lives.  So the decode-step operators read tokens' places, lengths, page tables and queries, which other
operators' kernels write, by plain loads; the table of rotary frequencies alone is the host's."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routed_expert_layer_fp32_gb300", "csrc")
FILES = ["pages.cu", "rope.cu", "kv_cache.cu", "kv_rows.cuh", "attn_decode.cuh", "attn_decode.cu", "attn_int4.cu",
         "block_norm.cu", "decoder.cuh"]


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    loads = re.findall(r"__ldg\s*\(\s*([^\n]*)", code) + re.findall(r"ld\.global[.\w]*\.nc[^\n]*", code)
    assert [x for x in loads if not x.startswith("r.turns")] == []
    # (with it the compiler may choose the read-only path for what a kernel only reads)
    assert re.findall(r"const[^,;(){}]*\*\s*__restrict__", code) == []
