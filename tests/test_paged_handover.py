"""The prompt kernel's hand-overs of tensor memory, read from its text: a thread
that read or wrote tensor memory fences before it arrives at a barrier, and one
that goes on to what another left there fences behind its wait.  (The order a
missing fence allows is not seen in results until a compiler or a machine makes
use of it.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dual_ar_tts_frame_gb300", "csrc")


def lines():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "paged_prompt.cu")).read())
    return [x.strip() for x in text.split("\n") if x.strip()]


@pytest.mark.parametrize("barrier", ["rowx", "pready"])
def test_arrivals_follow_a_fence(barrier):
    code = lines()
    at = [i for i, x in enumerate(code) if re.match(r"mbar_arrive\(&%s\b" % barrier, x)]
    assert at
    for i in at:
        assert code[i - 1] == "tc_fence_before();", code[i - 3:i + 1]


@pytest.mark.parametrize("barrier", ["rowx", "odone", "sfull"])
def test_waits_are_followed_by_a_fence(barrier):
    code = lines()
    at = [i for i, x in enumerate(code) if re.search(r"(mbar_wait|reached|ready)\(&%s\b" % barrier, x)]
    assert at
    for i in at:
        # (sfull's wait and the block's next are fenced together)
        assert "tc_fence_after();" in code[i + 1:i + 3], code[i:i + 3]
