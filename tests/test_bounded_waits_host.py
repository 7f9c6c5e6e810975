"""The bounded waits' control flow, read from the sources (no GPU).

A named barrier has no limit. Where the warps of a role time their waits each
for itself, one may give up while its neighbours go on, so they may meet only
at a barrier that every one of them reaches whatever its waits said, and leave
only by what that barrier told all of them.
"""

import glob
import os
import re

import pytest

from nsa_block_selection_gb300.build import CSRC


def _code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_named_barriers_carry_a_vote(path):
    code = _code(path)
    # PTX named barriers other than the one in bar_vote
    assert not re.search(r"\b(bar|barrier(\.cta)?)\.(sync|arrive)\b", code)
    # and each vote is heeded
    calls = len(re.findall(r"\bbar_vote\(", code)) - len(re.findall(r"\bbool bar_vote\(", code))
    assert calls == len(re.findall(r"if \(!bar_vote\(", code))


def _roles():
    """The auxiliary warpgroups' code in the sliding-window backward."""
    text = open(os.path.join(CSRC, "swa_bwd.cu")).read()
    for part in text.split("// ---- auxiliary warpgroup")[1:]:
        part = part.split("// ---- elementwise")[0]
        yield re.sub(r"//[^\n]*", "", part.split("----", 1)[1])


def test_the_auxiliary_warps_leave_together():
    roles = list(_roles())
    assert len(roles) == 2
    for code in roles:
        assert "bar_vote(1, 128, ok)" in code
        # `failed`, which ends the loop, is set only by what a vote said, and by
        # this warp's own waits once no barrier follows
        for m in re.finditer(r"failed = ([^;]*);", code):
            before = re.sub(r"\s+", " ", code[:m.start()])
            voted = before.endswith("if (!bar_vote(1, 128, ok)) { ")
            assert (m[1] == "true" and voted) or m[1] == "!ok || failed"
        last = code.index("failed = !ok || failed")
        assert "bar_vote" not in code[last:]
