"""Properties of the CUDA sources that no run can show."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_11_b200", "csrc")


def test_no_inline_branch_is_declared_uniform():
    """A lane's answer from an mbarrier test is its own: the phase may complete between two lanes' polls, so no
    branch may promise that all lanes take it."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        assert not re.search(r"\b(bra|brx\.idx|call|ret)\.uni\b", open(path).read()), os.path.basename(path)


def test_whole_warps_wait_with_a_vote():
    """The roles of the prompts' scan are warps that go on, behind a wait, to instructions of all lanes: they poll
    with wait_warp, whose lanes leave together; the poll of a lane of its own is for the copying lane and the drain."""
    text = open(os.path.join(CSRC, "ss_tc.cuh")).read()
    body = text[text.index("bool wait_warp("):]
    body = body[:body.index("\n}\n")]
    assert "__all_sync(0xffffffffu, done)" in body and "try_wait" in body
    text = open(os.path.join(CSRC, "ss_ssd_prefill.cu")).read()
    whole = text[text.index("auto wait = [&]"):]
    assert "tc::wait_warp(" in whole[:whole.index("};")]
    assert text.count("tc::wait(") == 2
