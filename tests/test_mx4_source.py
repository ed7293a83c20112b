"""What the source of the 4-bit product has to say for its hand-overs to be sound,
read without a GPU: orderings whose absence no run shows."""
import os
import re

from doubly_stochastic_projection_b200 import build


def _read(name):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())


def test_no_operand_waits_for_word_of_another_cta():
    # a commit orders the tensor work of its thread, not what that thread has
    # waited for: it tells nobody that operands are there, least of all across
    # CTAs.  Barriers are the CTA's own; what others read of its shared memory
    # (the partial sums) lies between cluster barriers
    product, tc5 = _read("mhc_mx4.cu"), _read("tc5.cuh")
    assert "cta_group::2" not in tc5 and "multicast" not in tc5
    assert all(m.startswith("map_rank(tc5::smem_addr(epi") for m in re.findall(r"map_rank\([^)]*\)?", product))
    for bar in re.findall(r"(?:commit|mbar_arrive|mbar_expect_tx)\w*(?:<\w+>)?\(([^;]*);", product):
        assert "map_rank" not in bar, bar
