"""Pins of the paged cache's oracle on cases worked by hand and on torch's own 8-bit type."""
import math

import numpy as np
import pytest
import torch

import oracle.cache as oc


def test_e4m3_codes_are_torchs():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, oc.E4M3, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.random.default_rng(1).integers(-12, 8, 4000),
                        oc.E4M3[:127], (oc.E4M3[:126] + oc.E4M3[1:127]) / 2, -(oc.E4M3[:126] + oc.E4M3[1:127]) / 2])
    x = np.clip(x, -448, 448)
    t = torch.tensor(x, dtype=torch.float32)
    ok = t.double().numpy() == x                  # ties and code values are fp32 numbers; the rest is rounded first
    want = t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = oc.encode(t.double().numpy(), "e4m3")
    assert ok.sum() > 300 and np.array_equal(oc.decode(want, "e4m3"), oc.decode(got, "e4m3"))


def test_int8_rounds_to_even_and_saturates():
    assert oc.encode([0.5, 1.5, -0.5, -2.5, 200, -200], "int8").view(np.int8).tolist() == [0, 2, 0, -2, 127, -127]


@pytest.mark.parametrize("x,fmt,want", [(448, "e4m3", 1), (449, "e4m3", 2), (224, "e4m3", 0.5), (127, "int8", 1),
                                        (128, "int8", 2), (0, "int8", 2.0 ** -126), (63.5, "int8", 0.5)])
def test_scale_is_the_smallest_power_of_two(x, fmt, want):
    assert oc.pow2_scale(x, fmt) == want


def _tiny():
    """Two pages of 16, one head, D = 2: keys (1,0),(0,1) at slots 0, 1 of page 1."""
    c = {"fmt": "int8", "k": np.zeros((2, 1, 16, 2), np.uint8), "v": np.zeros((2, 1, 16, 2), np.uint8),
         "ks": np.ones((2, 1), np.float32), "vs": np.full((2, 1), 0.5, np.float32)}
    c["k"][1, 0, :2] = [[1, 0], [0, 1]]
    c["v"][1, 0, :2] = [[4, 8], [12, 16]]
    return c


def test_attention_by_hand():
    c = _tiny()
    table, length, cu = np.array([[1, 0]]), np.array([2]), np.array([0, 1])
    q = np.array([[[math.log(3.0), 0.0]]])
    # scores ln 3 and 0: weights 3/4, 1/4; v = (2,4), (6,8); lse = ln 4
    o, z = oc.attend(c, table, length, cu, q, scale=1.0)
    assert np.allclose(o[0, 0], [3.0, 5.0], atol=1e-14) and abs(z[0, 0] - math.log(4)) < 1e-14
    # the cap: c tanh(ln 3 / c); the slope takes s * 1 from the far key
    o, z = oc.attend(c, table, length, cu, q, scale=1.0, softcap=2.0, slopes=[0.25])
    w = np.exp([2 * math.tanh(math.log(3) / 2) - 0.25, 0.0])
    assert np.allclose(o[0, 0], (w[0] * np.array([2, 4]) + w[1] * np.array([6, 8])) / w.sum())
    # a window of one key, a first key behind the query, an empty row
    assert oc.attend(c, table, length, cu, q, scale=1.0, window=1)[0][0, 0].tolist() == [6.0, 8.0]
    o, z = oc.attend(c, table, length, cu, q, first=[2])
    assert o.any() == False and z[0, 0] == -math.inf       # noqa: E712


def test_visible_intervals():
    assert oc.visible(10, 4, 1, "causal") == (0, 8, 7)
    assert oc.visible(10, 4, 1, "full") == (0, 10, 7)
    assert oc.visible(10, 4, 1, "prefix", prefix=9) == (0, 9, 7)
    assert oc.visible(10, 4, 1, "prefix", prefix=99) == (0, 10, 7)
    assert oc.visible(10, 4, 1, "causal", window=3) == (5, 8, 7)
    assert oc.visible(10, 4, 1, "causal", window=3, first=6) == (6, 8, 7)


def test_store_by_hand():
    c = _tiny()
    table, length = np.array([[1, 0]]), np.array([4])
    # slots 2, 3 get 300 and 1: scale 4 (127 * 2 < 300 <= 127 * 4); the older codes move to 1/4 (ties to even)
    k = np.array([[[300.0, 1.0]], [[2.0, 6.0]]])
    oc.store(c, table, length, np.array([0, 2]), k, k)
    assert c["ks"][1, 0] == 4 and c["k"][1, 0, :4].view(np.int8).tolist() == [[0, 0], [0, 0], [75, 0], [0, 2]]
    assert c["vs"][1, 0] == 4 and c["v"][1, 0, :2].view(np.int8).tolist() == [[0, 1], [2, 2]]   # 2,4,6,8 / 4: 0.5, 1, 1.5, 2


def test_fork_by_hand():
    # page 16, row 0: pages 0, 3 (len 20), row 1: page 5 (len 16), row 2: page 1 (len 3)
    rng = np.random.default_rng(0)
    c = {"fmt": "int8", "k": rng.integers(0, 256, (8, 1, 16, 2), dtype=np.uint8), "v": rng.integers(0, 256, (8, 1, 16, 2), dtype=np.uint8),
         "ks": rng.random((8, 1), dtype=np.float32), "vs": rng.random((8, 1), dtype=np.float32)}
    table = np.array([[0, 3, -1, -1], [5, -1, -1, -1], [1, -1, -1, -1]])
    was = {x: c[x].copy() for x in ("k", "v", "ks", "vs")}
    out, ln, st = oc.fork(c, table, [20, 16, 3], [1, 0, -1, 0], [1, 13, 4, 0])
    # held: 5; 0, 3.  free: 1, 2, 4, 6, 7.  row 0: full page 5, a new one 1; row 1 keeps 3 and grows to 33 tokens
    # (page 2); row 3 gets a copy of 3 in page 4
    assert out.tolist() == [[5, 1, -1, -1], [0, 3, 2, -1], [-1, -1, -1, -1], [0, 4, -1, -1]]
    assert ln.tolist() == [17, 33, 0, 20] and st == 0
    for x in was:
        assert np.array_equal(c[x][4], was[x][3]) and np.array_equal(c[x][3], was[x][3])
    out, ln, st = oc.fork(c, table, [20, 16, 3], [0, 0, 0, 0], [0, 40, 40, 0])
    # free: 1, 2, 4, 5, 6, 7, all taken by rows 1 and 2 (a copy and two pages each); row 3 ends before its copy
    assert st == 8 and ln.tolist() == [20, 60, 60, 16] and out[3].tolist() == [0, -1, -1, -1]
    out, ln, st = oc.fork(c, np.array([[0, 3], [5, -1], [1, -1]]), [20, 16, 3], [0, 1, 2], [14, 0, 0])
    assert st == 8 and ln.tolist() == [32, 16, 3]          # the table's width ends row 0


def test_compact_by_hand():
    c = _tiny()
    c = {x: (np.repeat(c[x], 4, axis=0) if x != "fmt" else c[x]) for x in c}
    c["ks"][:, 0] = np.arange(8)
    out, used = oc.compact(c, np.array([[6, 1, -1], [4, 6, 7]]), [20, 33])
    # held 1, 4, 6, 7: U = 4; 4 -> 0, 6 -> 2, 7 -> 3
    assert used == 4 and out.tolist() == [[2, 1, -1], [0, 2, 3]] and c["ks"][:4, 0].tolist() == [4, 1, 6, 7]
