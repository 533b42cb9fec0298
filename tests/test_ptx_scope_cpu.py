"""Memory-model rules that the kernels' inline PTX has to keep, checked in the sources: no run can
show that an ordering is guaranteed."""
import glob
import os
import re

import pytest

from int8_w8a8_quantized_smoothed_b200 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu*")))
LITERAL = r'"(?:[^"\\]|\\.)*"'


def _statements(path):
    """The PTX statements of a source file's asm blocks."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = []
    for block in re.findall(r"\basm(?:\s+volatile)?\s*\(((?:\s*%s)+)" % LITERAL, text):
        code = "".join(t[1:-1] for t in re.findall(LITERAL, block))
        found += [t.strip() for t in re.split(r";|\\n|\\t|[{}]", code)]
    return [t for t in found if t]


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_arrivals_on_another_cta_are_at_cluster_scope(path):
    """An mbarrier arrival without a scope releases at CTA scope, which orders nothing for a
    thread of another CTA: one on a cluster address has to name the cluster."""
    for s in _statements(path):
        if s.startswith("mbarrier.arrive") and "shared::cluster" in s:
            assert ".cluster.shared::cluster" in s, s


def test_waits_on_the_pairs_barriers_are_at_cluster_scope():
    """In the gradient GEMM the even CTA's commits arrive on both CTAs' `empty` and `tfull`, and
    both CTAs arrive on the even one's `full` and `tempty`: a wait on any of them observes a thread
    that may be of the other CTA."""
    with open(os.path.join(build.CSRC, "gradgemm.cuh")) as f:
        text = f.read()
    start = text.index("grad_gemm_kernel(const __grid")
    kernel = text[start:text.index("__global__", start)]
    waits = re.findall(r"\b(mbar_wait(?:_cluster)?)\(bar_(full|empty|tfull|tempty)\b", kernel)
    assert {bar for _, bar in waits} == {"full", "empty", "tfull", "tempty"}
    assert all(fn == "mbar_wait_cluster" for fn, _ in waits), waits


def test_the_rule_finds_statements():
    found = [s for p in SOURCES for s in _statements(p) if s.startswith("mbarrier.arrive")]
    assert sum("shared::cluster" in s for s in found) >= 2
    assert any("shared::cta" in s for s in found)
