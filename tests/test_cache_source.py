"""Rules of the paged cache's kernels that can be read off their sources, without a GPU."""
import os
import re

import numpy as np

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
    """Softmax and conversion warps go on to instructions of all 32 lanes: no lane acts on its own wait's result, all ask
    for a vote on the flag that a wait which gave up has raised, at the end of a segment and before its result."""
    src = source("cache_attend_tc.cu")
    roles = src[src.index("if (warp < 8) {\n"):src.index("idS = tc::idesc")]
    assert len(re.findall(r"mbar_wait\(", roles)) == len(re.findall(r"(?<![=!&|(] )(?<!\()\bmbar_wait\([^;]*;", roles)) == 7
    assert not re.search(r"(=|&&|\|\||!|if \()\s*mbar_wait\(", roles)
    assert len(re.findall(r"if \(!went_well\(abort\)\) break;", roles)) == 2
    assert roles.index("went_well") < roles.index("a.lse[oi]")
    assert re.search(r"bool went_well\([^)]*\) \{ return __all_sync\(0xffffffffu, \*abort == 0\); \}", src)


def test_the_polynomial_for_small_capped_scores():
    """The committed coefficients against tanh in 64 bits over their range, |y| <= 1/2, and evaluated as the kernels do
    (in fp32, by y2 = 2 log2(e) y): within what the comment beside them states."""
    path = os.path.join(CSRC, "cache_plan.cuh")
    with open(path) as f:
        raw = " ".join(f.read().replace("\n//", " ").split())
    found = re.search(r"relative error is ([0-9.e-]+) \(([0-9.e-]+) with the roundings", raw)
    assert found, "the comment states both errors"
    fit, whole = float(found.group(1)), float(found.group(2))
    c = [1.0] + [float.fromhex(x) for x in re.findall(r"tanh_coef\((-?0x[0-9a-f.]+p[-+]?\d+), \d\)", raw)]
    assert len(c) == 5 and "constexpr float kTanhNear = kLog2e;" in raw
    y = np.linspace(1e-4, 0.5, 400001)
    err = np.abs(y * sum(k * y ** (2 * i) for i, k in enumerate(c)) / np.tanh(y) - 1).max()
    assert 0.9 * fit <= err <= fit
    unit = 2 * 1.4426950408889634
    f32 = [np.float32(k / unit ** (2 * i + 1)) for i, k in enumerate(c)]
    y2 = (y * unit).astype(np.float32)
    u, r = y2 * y2, np.full_like(y2, f32[4])
    for k in f32[3::-1]:
        r = (r.astype(np.float64) * u + k).astype(np.float32)          # one rounding, as the kernels' fused operation
    err = np.abs((r * y2).astype(np.float64) / np.tanh(y2.astype(np.float64) / unit) - 1).max()
    assert 0.8 * whole <= err <= whole
