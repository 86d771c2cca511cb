"""Order and waits in csrc/decode_tree_tc.cu that a run shows by chance only, looked up in the source."""
import os
import re

from long_context_sparse_dsa_gb300 import build as dsa_build


def _code():
    with open(os.path.join(dsa_build.CSRC, "decode_tree_tc.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text, head):
    """From `head` to the end of the block that opens behind it."""
    at = text.index(head)
    n, i = 0, text.index("{", at)
    for j in range(i, len(text)):
        n += {"{": 1, "}": -1}.get(text[j], 0)
        if n == 0:
            return text[i:j + 1]


def test_a_vote_over_barriers_is_followed_by_a_warp_barrier():
    """A warp's lanes may wait for two barriers at once; a vote says that all have completed but orders no memory for the lane that
    then issues."""
    body = _body(_code(), "bool tc_wait(uint32_t bar")
    votes = [m.end() for m in re.finditer(r"__all_sync", body)]
    assert len(votes) == 2
    for at in votes:
        rest = body[at:]
        assert rest.index("__syncwarp()") < rest.index("return")
