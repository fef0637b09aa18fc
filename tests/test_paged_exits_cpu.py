"""The join of the paged attention reads a cut of every CTA and stores through it, so no CTA may leave the
products' kernels without one: read from the source, as nothing makes a CTA leave early on purpose."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rank_linear_complexity_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, at):
    """The text in braces that opens first from `at` on."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def enclosing(body, at):
    """The innermost block around `at`."""
    depth = 0
    for i in range(at, -1, -1):
        depth += {"}": 1, "{": -1}.get(body[i], 0)
        if depth < 0:
            return block(body, i)
    raise AssertionError("not in a block")


@pytest.mark.parametrize("name,kernel", [("paged_attn.cu", "paged_attn_kernel("),
                                         ("paged_attn_wide.cu", "paged_wide_kernel(")])
def test_every_early_end_of_a_cta_writes_its_cut(name, kernel):
    text = source(name)
    body = block(text, text.index(")", text.index(kernel)))
    assert "write_cut(p" in body
    ends = [m.start() for m in re.finditer(r"\breturn;", body)]
    assert ends
    for at in ends:
        assert re.search(r"\bleave\(p, \d+\);\s*return;", enclosing(body, at)), body[max(0, at - 200):at]


def test_leaving_waits_before_it_writes_the_cut():
    text = source("paged_attn.cuh")
    body = block(text, text.index("void leave("))
    assert 0 < body.index("wait_prerequisites();") < body.index("p.cuts[blockIdx.x] = make_int4(-1")
