"""Rules of the paged cache's kernels that can be read off their sources, without a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(__file__), "..", "shared_prefix_decode_xattention_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_registers_are_exchanged_by_whole_warpgroups():
    """Every warp of a warpgroup has to execute the same register exchange: one place for each direction, both before
    the branch that parts the warps of a group (8 issues, 9 to 11 convert)."""
    src = source("cache_attend_tc.cu")
    up, down = ([m.start() for m in re.finditer(rf"tc::regs_{d}<", src)] for d in ("up", "down"))
    assert len(up) == 1 and len(down) == 1
    assert max(up[0], down[0]) < src.index("else if (warp > kIssueWarp)")
    assert re.search(r"if \(warp < 8\) tc::regs_up<\w+>\(\);\s*else tc::regs_down<\w+>\(\);", src)


def test_waits_of_whole_warps_have_one_verdict():
    """Softmax and conversion warps go on to instructions of all 32 lanes: no lane leaves a loop on its own wait's result,
    but all do by a vote on it."""
    src = source("cache_attend_tc.cu")
    roles = src[src.index("if (warp < 8) {\n"):src.index("idS = tc::idesc")]
    exits = [m.start() for m in re.finditer(r"if \(!ok\) break;", roles)]
    assert len(exits) == 3                          # a chunk's softmax, a segment's end, a chunk's conversion
    for at in exits:
        last = list(re.finditer(r"ok = (\w+)\(", roles[:at]))[-1]
        assert last.group(1) in ("warp_wait", "__all_sync"), roles[last.start():at]
    lane = [m.group(0) for m in re.finditer(r"[^;{}]*\bmbar_wait\(", roles)]
    assert len(lane) == 3                           # (put to those votes: the scores' and the two operand buffers')
