"""What the attention over pages does once a wait has given up, read from its source
and counted out (no GPU): nothing of a CTA's copies stays in flight, and its warps
leave together."""

import os
import re

from nsa_block_selection_gb300.build import CSRC

CODE = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "paged_attn.cu")).read())


def _flat(text):
    return re.sub(r"\s+", " ", text)


def test_a_warp_drains_the_copy_that_it_has_issued_and_not_read():
    """Step t of an item is issued by warp t % 4: the first stages - 1 before any is
    read, step t + stages - 1 once t has been read. What a warp whose wait for step t
    gives up has in flight is then step t's or step t + 1's copy, if that is its own."""
    header = open(os.path.join(CSRC, "paged_attn.cuh")).read()
    warps = int(re.search(r"kPaWarps = (\d+)", header)[1])
    stages = int(re.search(r"kStages = Q4 \? (\d+)", CODE)[1])
    flat = _flat(CODE)
    assert "for (int t = 0; t < C::kStages - 1 && t < steps && !failed; ++t) if (t % kPaWarps == warp) issue(t);" in flat
    assert "const int next = t + C::kStages - 1; if (next < steps && next % kPaWarps == warp) issue(next);" in flat
    assert ("const int own = t % kPaWarps == warp ? t : t + 1; const uint32_t g = issued + own; "
            "if (own % kPaWarps == warp && own < steps) wait_phase(") in flat
    for steps in range(1, 14):
        for t in range(steps):
            issued = set(range(min(stages - 1, steps))) | {s + stages - 1 for s in range(t) if s + stages - 1 < steps}
            for warp in range(warps):
                open_ = {s for s in issued if s % warps == warp and s >= t}
                own = t if t % warps == warp else t + 1
                assert open_ == ({own} if own % warps == warp and own < steps else set())
                # a wait for a free slot that gives up (before step t + stages - 1 is issued)
                if t + stages - 1 < steps and (t + stages - 1) % warps == warp:
                    assert not {s for s in issued if s % warps == warp and s > t}


def test_the_warps_of_a_cta_leave_together():
    """A warp that gave up meets the others at the item's barrier, whose vote ends the
    loop for all before the ring is written over."""
    loop = CODE[CODE.index("for (bool more = !p.cut"):CODE.index("constexpr int kJoinThreads")]
    vote = loop.index("if (__syncthreads_or(failed)) {")
    assert _flat(loop[vote:]).startswith("if (__syncthreads_or(failed)) { failed = true; break; }")
    assert "__syncthreads();" not in loop[:vote]
    assert vote < loop.index("float* const joined")
