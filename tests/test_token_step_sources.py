"""The mixers' token steps (csrc/token_step.cu) read a slot's state only behind
the search that tells which row takes the slot's tokens along.

A CTA whose row is taken along by another one has no business with the state: in
place that other one may be writing it, and with tokens of few sequences in turn
nearly every row is such a one, whose reads cost a state each.  What is read too
early is dropped, so no run shows it: the sources are checked.
"""
import re

import pytest

from test_early_launch_sources import kernels, sources

READS = r"p\.state\s*\+\s*so|load\(state\b"
SEARCH = r"(?:first_rows|last_rows)\s*<"


def body(kernel):
    found = {re.search(r"(\w+_kernel)\s*\(", b).group(1): b for _, b in kernels(sources()["token_step.cu"])}
    return found[kernel]


@pytest.mark.parametrize("kernel", ["delta_step_kernel", "delta_step_vfirst_kernel", "conv1d_step_kernel"])
def test_states_are_read_behind_the_rows_search(kernel):
    text = body(kernel)
    searches = [m.start() for m in re.finditer(SEARCH, text)]
    reads = [m.start() for m in re.finditer(READS, text)]
    assert searches and reads
    assert max(searches) < min(reads)
    assert "kEarlier" not in text[min(reads):]        # nothing that was read is dropped
