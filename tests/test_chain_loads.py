"""Kernels that start before the ones ahead of them end: how they read what those write (source check, no GPU).

The non-coherent load (__ldg) may be served from a cache line, or moved to a place, from before the words were
written, so it is for a call's inputs alone. Words of the workspace that an earlier kernel of the chain writes are
read with __ldcg or a plain load, and behind the wait unless the kernel ahead has passed that wait itself (then only
with __ldcg).
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_split_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def noncoherent(text):
    """The arguments of every __ldg in the text."""
    for m in re.finditer(r"__ldg\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def test_prompt_pass_reads_its_workspace_past_l1():
    with open(os.path.join(CSRC, "gqa_kernels.h")) as f:
        struct = re.search(r"struct MlaPrefillParams \{.*?\n\};", f.read(), re.S).group(0)
    fields = re.findall(r"\*\s*(\w+);", struct.split("// workspace")[1])
    assert {"kv_len", "kv_start", "q_start", "qt_start", "bad", "valid"} <= set(fields)
    fields.remove("err")
    for arg in noncoherent(source("gqa_mla_prefill.cu")):
        assert not any(re.search(rf"\bp\.{f}\b", arg) for f in fields), arg


def test_latent_merge_reads_the_token_count_behind_its_wait():
    """The decode triggers its dependents before its own wait, so the merge may start while the scan still runs."""
    body = source("gqa_mla.cu").split("gqa_mla_merge_kernel(const MlaParams p) {")[1]
    before = body[:body.index("pdl_wait();")]
    assert "p.kv_indptr" not in before and "p.bounds" not in before


def test_latent_decode_reads_the_scan_with_coherent_loads():
    """kv_indptr and the ranges are the scan's words: no non-coherent load of them, by name or through a helper."""
    for name in ("gqa_mla.cu", "gqa_mla_tc.cu"):
        text = source(name)
        for arg in noncoherent(text):
            assert not re.search(r"\b(kv_indptr|indptr|bounds|cuts|cost_ptr|slots)\b", arg), (name, arg)
        assert not re.search(r"\b(warp_find_seq|load_indptr_window|warp_find_window)\(", text)
        assert not re.search(r"const int\* __restrict__ indptr", text)
