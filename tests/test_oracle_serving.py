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


def test_e4m3_pins():
    assert OV.E4M3[[0, 1, 7, 8, 0x38, 0x7E]].tolist() == [0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 448.0]
    x = np.array([0.0, -0.0, 1.0, 1.0625, 1.1875, 448.0, 1e9, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11, 17.0, 19.0])
    assert OV.encode("e4m3_b64", x).tolist() == [0, 0x80, 0x38, 0x38, 0x3A, 0x7E, 0x7E, 0xFE, 0, 2, 0x80, 0x58, 0x5A]
    all_codes = np.concatenate((np.arange(0x7F), 0x80 + np.arange(0x7F))).astype(np.uint8)
    assert np.array_equal(OV.encode("e4m3_b64", OV.decode("e4m3_b64", all_codes)), all_codes)
    torch = __import__("torch")
    if hasattr(torch, "float8_e4m3fn"):
        y = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 40
        assert np.array_equal(OV.encode("e4m3_b64", y), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_block_append_pins():
    c = OV.BlockCache("int8_b64", 1, 1, 2, 128)
    row = lambda *v: np.array([[v]], np.float32)           # noqa: E731
    put = lambda x, pos: c.append("k", 0, x, pos)          # noqa: E731
    codes = lambda t: c.planes["k"]["payload"][0, 0, t].view(np.int8).tolist()     # noqa: E731
    put(row(127.0, -3.0), 0)
    assert c.planes["k"]["scale"][0, 0].tolist() == [1.0, 0.0] and codes(0) == [127, -3]
    put(row(100.0, 0.5), 1)                                # fits: the scale stays, half to even
    assert c.planes["k"]["scale"][0, 0, 0] == 1.0 and codes(1) == [100, 0]
    put(row(300.0, 8.0), 2)                                # needs 2.36: four times; 127 / 4 = 31.75, -0.75, 25, 0
    assert c.planes["k"]["scale"][0, 0, 0] == 4.0 and codes(0) == [32, -1] and codes(1) == [25, 0] and codes(2) == [75, 2]
    put(row(0.0, 0.0), 64)
    assert codes(64) == [0, 0] and c.planes["k"]["scale"][0, 0, 1] == 0.0
    put(row(254.0, 2.0), 65)                               # no scale yet: what the new row needs
    assert c.planes["k"]["scale"][0, 0, 1] == 2.0 and codes(65) == [127, 1]
    put(row(1.27, 0.01), 0)                                # a block begun again
    assert c.planes["k"]["scale"][0, 0, 0] == np.float32(np.float32(1.27) / np.float32(127)) and codes(0) == [127, 1] and codes(2) == [75, 2]


def test_growing_scales_cost_a_kept_row_at_most_a_step_more():
    """Appending row by row with ever larger values: each kept value is within 1.5 steps of the final scale."""
    rng = np.random.default_rng(3)
    c = OV.BlockCache("int8_b64", 1, 1, 8, 64)
    x = (rng.standard_normal((1, 64, 8)) * 1.09 ** np.arange(64)[:, None]).astype(np.float32)
    for t in range(64):
        c.append("k", 0, x[:, t:t + 1], t)
    s = c.planes["k"]["scale"][0, 0, 0]
    assert np.abs(c.values("k", 0, 0, 64) - x[0]).max() <= 1.5 * s


def test_attend_sees_blocks_and_rows():
    rng = np.random.default_rng(4)
    k, v, q = rng.standard_normal((200, 8)), rng.standard_normal((200, 8)), rng.standard_normal((1, 2, 3, 8))
    values = lambda t, b, h, n: (k if t == "k" else v)[:n]                         # noqa: E731
    full, _ = OV.attend(values, 1, q, 0.3, [200], True)
    listed, _ = OV.attend(values, 1, q, 0.3, [200], True, np.tile(np.arange(4), (1, 1, 3, 1)))
    assert np.array_equal(full, listed)
    one, _ = OV.attend(values, 1, q, 0.3, [200], False, np.array([[[[1, -1, 3]] * 3]]))
    x = 0.3 * (k[64:128] @ q[0, 0, 0])
    p = np.exp(x - x.max())
    assert np.allclose(one[0, 0, 0], p @ v[64:128] / p.sum(), rtol=1e-12)
    none, _ = OV.attend(values, 1, q, 0.3, [0], False)
    assert not none.any()


def test_bounds_and_selection_pins():
    rows = np.array([[1.0, -2.0], [3.0, 0.5], [-0.1, 0.0]], np.float32)
    codes, scale = OV.bounds(rows)
    s = np.float32(3) / np.float32(127)
    assert scale.tolist() == [s] and codes.tolist() == [[[-5, -85], [127, 22]]]     # -0.1 / s = -4.2, -2 / s = -84.7, 0.5 / s = 21.2
    assert OV.bounds(np.zeros((65, 2), np.float32))[1].tolist() == [0.0, 0.0]
    rng = np.random.default_rng(0)
    k, q = rng.standard_normal((64 * 9, 16)).astype(np.float32), rng.standard_normal((3, 1, 16)).astype(np.float32)
    codes, scale = OV.bounds(k)
    for blk in range(9):                                   # no product of a block passes its score
        for x in q[:, 0]:
            sq = np.abs(x).max() / 127
            q8 = np.rint(x / sq)
            top = np.maximum(q8 * codes[blk, 0].astype(float), q8 * codes[blk, 1].astype(float)).sum() * sq * scale[blk]
            assert (k[blk * 64:blk * 64 + 64] @ (q8 * sq)).max() <= top + 1e-5
    one = np.zeros((9, 2, 16), np.int8)
    one[3, 1], one[5, 1], one[7, 0] = 100, 100, -100
    x = np.ones((1, 2, 16), np.float32)
    x[:, 1] = -1
    got = OV.select(one, np.ones(9, np.float32), x, [64 * 9 - 1, 64 * 8 - 1], 3, 1, 1)
    assert got.tolist() == [[0, 3, 8], [0, 1, 7]]          # ties to the lowest; the recent block counts by itself
    assert OV.select(one, np.ones(9, np.float32), x, [-1, 100], 4, 0, 0).tolist() == [[-1] * 4, [0, 1, -1, -1]]
