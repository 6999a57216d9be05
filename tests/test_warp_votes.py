"""A rule of the router's and the optimiser's kernels that no result shows, checked on their
sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_moe_routed_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["router.cu", "router.cuh", "router_choice.cuh", "router_group.cu",
                                  "router_bwd.cu", "adamw.cu"])
def test_no_lane_skips_what_its_warp_does_together(name):
    """A vote, a shuffle or a reduction of all lanes waits for all of them: none stands behind
    && or ||, whose left side may differ between the lanes."""
    together = r"(?:__any_sync|__all_sync|__ballot_sync|__shfl\w*|__reduce\w*|__match\w*|" \
               r"group_any|group_max|group_sum|warp_max|warp_sum|first_sum|lanes_max|lanes_sum)"
    text = code(name)
    assert re.search(together, text)
    assert not re.findall(r"(?:&&|\|\|)\s*\(?\s*!?\s*%s\s*[(<]" % together, text)
