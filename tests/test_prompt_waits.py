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
    assert len(guarded) >= 5
    for condition in guarded:
        assert not re.search(r"\bwait\(", condition), condition
    for kept in re.findall(r"const bool (\w+) = wait\(", text):
        assert kept + " && umma::elect_one()" not in text
