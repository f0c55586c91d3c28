"""Rules of the kernels' sources whose breach shows only when a wait runs out, which
no test can bring about on a device."""
import glob
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "compressive_fine_tuning_b200", "csrc")


def _structs(text):
    """(name, body) of every struct, by its braces."""
    for m in re.finditer(r"\bstruct (\w+) \{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at]


def test_epilogues_with_barriers_give_up_together():
    """A warp of the persistent product's epilogue that gives up on a tile leaves the
    tile's barriers to the others: the warps that meet there decide together."""
    seen = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for name, body in _structs(open(path).read()):
            team = re.search(r"static constexpr int kTeam = (\d);", body)
            if team or "void tile(" in body:
                meet = {int(n) // 32 for n in re.findall(r"named_bar_sync\([^,]+, (\d+)\)", body)}
                seen[name] = (team and int(team.group(1)), meet or {1})
    assert len(seen) >= 6
    for name, (team, meet) in seen.items():
        assert {team} == meet, name
    # the decision's barriers are away from the ids in use
    vote = int(re.search(r"kVoteBar = (\d+);", open(os.path.join(CSRC, "sk_gemm.cuh")).read()).group(1))
    assert 5 <= vote <= 12
