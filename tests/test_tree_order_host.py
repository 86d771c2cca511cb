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


def test_fetching_warps_wait_for_what_they_asked_for():
    """Each Q that a warp asks for is a phase of its barrier, so behind n of them the last phase has parity (n - 1) & 1; the last
    items of the ring are waited for too.  Both whether this warp gave up or not: another may have, and a TMA copy must not
    land behind the CTA's end."""
    code = _code()
    ask = _body(code, "if (pw == 0) {")
    assert len(re.findall(r"mbar_arrive_expect_tx\(qfull", code)) == 1 and "mbar_arrive_expect_tx(qfull" in ask and "++nq;" in ask
    assert code.count("++nq;") == 1 and "nq = 0;" in code
    fetch = _body(code, "if (warp >= 9) {")
    end = fetch[fetch.rindex("cp_async_wait<0>();"):]
    assert "if (nq > 0) mbar_wait(qfull, (nq - 1) & 1, nullptr);" in end and end.count("qfull") == 1
    assert "for (uint32_t i = it > C::NS ? it - C::NS : 0; i < it; ++i) mbar_wait(full(i), (i / C::NS) & 1, nullptr);" in end
    assert "{" not in end   # on every way out
