"""Bounded waits of the prompt kernels, read from their sources: what happens
when one gives up is not to be provoked on a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_04_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["prompt_fwd.cu", "prompt_bwd.cu"])
def test_elections_go_by_answers_given_together(name):
    """An election names all lanes of its warp: what guards it has to be the
    same in all of them, also when some lanes' waits give up."""
    text = source(name)
    guarded = re.findall(r"(?:if \(|return )(.*?)umma::elect_one\(\)", text)
    assert guarded
    for condition in guarded:
        assert not re.search(r"\bwait\(", condition), condition
    for kept in re.findall(r"const bool (\w+) = wait\(", text):
        assert kept + " && umma::elect_one()" not in text


@pytest.mark.parametrize("name,rings", [("prompt_fwd.cu", ("full[i]", "q_full")), ("prompt_bwd.cu", ("full1[i]", "full2[i]", "a2_full"))])
def test_a_cta_that_gave_up_ends_after_its_copies_and_products(name, rings):
    """Every barrier that copies land on is waited for behind the roles, in the
    phase of its last copy, and all products before the tensor memory goes
    back; one look at a phase that may be an older one is no wait."""
    text = source(name)
    assert not re.search(r"mbar_try_wait\(&bars", text)
    tail = text[text.index("if (dead && threadIdx.x == 0)"):]
    tail = tail[:tail.index("tmem_dealloc")]
    for ring in rings:
        assert "wait_end(&bars.%s, " % ring in tail, ring
    assert re.search(r"commit\(&bars\.end\);\s*wait_end\(&bars\.end, 0, p\.err\);", text)
