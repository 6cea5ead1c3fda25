"""Hand-computed pins of the serving-step oracle (CPU)."""
import numpy as np

from oracle import serving as OV


def test_plan_pins():
    table, free = np.array([[5, 6, 0], [7, 0, 0], [8, 9, 0], [0, 0, 0]]), np.array([1, 2, 3, 0, 0, 0])
    # request 0 grows inside its second page, 1 has ended (page 7 goes back), 2 needs a third page, 3 is new
    r = OV.page_plan([70, 3, 128, 0], [2, -1, 1, 65], table, 64, free, 3, 80)
    assert r["granted"].tolist() == [2, 0, 1, 65] and r["lens"].tolist() == [72, 0, 129, 65]
    assert free.tolist() == [1, 2, 3, 7, 0, 0] and r["n_free"].tolist() == [1]
    assert table.tolist() == [[5, 6, 0], [7, 0, 0], [8, 9, 7], [3, 2, 0]]
    assert r["cu_new"].tolist() == [0, 2, 2, 3, 68]
    assert r["slots"][:4].tolist() == [6 * 64 + 6, 6 * 64 + 7, 7 * 64, 3 * 64] and r["slots"][67] == 2 * 64 and r["slots"][68:].tolist() == [-1] * 12
    assert r["positions"][:4].tolist() == [70, 71, 128, 0] and r["positions"][-1] == -1


def test_plan_waits_in_order():
    free = np.array([4, 5, 6])
    # one page each for the first two; the third needs three: it waits, and so does the fourth behind it; the fifth needs none
    r = OV.page_plan([0, 0, 0, 0, 10], [1, 64, 129, 1, 1], np.zeros((5, 3), int), 64, free, 3, 1000)
    assert r["granted"].tolist() == [1, 64, 0, 0, 1]
    # past the table's room: refused, without a place in the others' sums
    r = OV.page_plan([0, 0], [200, 1], np.zeros((2, 3), int), 64, free, 1, 1000)
    assert r["granted"].tolist() == [0, 1]
    # the step's tokens
    r = OV.page_plan([0, 0, 0], [5, 4, 1], np.zeros((3, 1), int), 64, free, 3, 8)
    assert r["granted"].tolist() == [5, 0, 0] and r["n_free"].tolist() == [2]
