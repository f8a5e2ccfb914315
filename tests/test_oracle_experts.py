"""Pins of the experts' oracle: the e4m3 grid, rounding, block scales and layouts by hand."""
import numpy as np

import oracle.experts_oracle as X


def test_e4m3_grid():
    v = X.VALUES
    assert v[0x7E] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0x80] == 0.0 and np.signbit(v[0x80])
    assert (np.diff(X._GRID) > 0).all()
    back = X.to_e4m3(v)
    ok = ~np.isnan(v)
    assert np.array_equal(back[ok], np.arange(256)[ok].astype(np.uint8))


def test_e4m3_rounds_to_nearest_even():
    x = np.array([1.0625, 1.1875, 1.0624, 1.0626, -1.0625, 2.0 ** -10, 1.5 * 2.0 ** -9, 440.0, 432.0, np.nan, np.inf])
    want = [0x38, 0x3A, 0x38, 0x39, 0xB8, 0x00, 0x02, 0x7E, 0x7E, 0x7F, 0x7F]
    # 1.0625 lies halfway between 1 (0x38) and 1.125 (0x39); 432 halfway between 416 (0x7D) and 448 (0x7E)
    assert X.to_e4m3(x).tolist() == want


def test_block_exponent():
    for a, e in ((448.0, 0), (448.5, 1), (224.0, -1), (225.0, 0), (1.0, -8), (0.875, -9), (0.0, 0), (2.0 ** -133, -126),
                 (3.3e38, 120), (np.inf, 0)):
        g = np.zeros((1, 128))
        g[0, 5] = -a
        assert X.block_exponent(g, 1)[0] == e, a


def test_rows_and_weights_share_their_values():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 200)) * np.exp(rng.standard_normal((5, 200)))
    q, s = X.quant_rows(x)
    assert q.shape == (5, 256) and s.shape == (5, 4) and (q[:, 200:] == 0).all() and (s[:, 2:] == 127).all()
    err = np.abs(X.rows_value(q, s)[:, :200] - x)
    e = np.repeat(X.block_exponent(np.pad(x, ((0, 0), (0, 56))).reshape(5, 2, 128), 2), 128, axis=1)[:, :200]
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e - 10))).all()  # half a step
    w = rng.standard_normal((130, 136))
    q, s = X.quant_weight(w)
    qt, st = X.quant_weight(w.T)
    assert np.array_equal(X.weight_value(q, s)[:, :136], X.weight_value(qt, st)[:, :130].T)


def test_columns_form_blocks_by_hand():
    off = [0, 130, 130, 131]                     # 2 blocks, none, 1
    assert X.first_blocks(off)[:3] == [0, 2, 3]  # 130 // 128 + 1, + 2
    x = np.arange(131.0)[:, None] * np.ones((1, 8))
    qt, s = X.quant_cols(x, off, 131 // 128 + 3, fill=9)
    assert (qt[2] == 9).all() and (s[2] == 9).all()
    assert X.VALUES[qt[1, 0, :3]].tolist() == [256.0, 256.0, 0.0]  # 128 and 129 at e = -1: 256 and 258, rounded
    assert s[1, 0] == 126 and X.VALUES[qt[3, 0, 0]] * 2.0 ** (int(s[3, 0]) - 127) == 128.0


def test_products_by_hand():
    one = X.to_e4m3(np.ones((2, 128)))
    scale = np.full((2, 4), 128, dtype=np.uint8)
    w = X.to_e4m3(np.full((3, 128), 2.0))
    y = X.expert_gemm(X.rows_value(one, scale), [X.weight_value(w, np.full((1, 4), 127, dtype=np.uint8))], [0, 2])
    assert (y == 128 * 2 * 2).all()
    x = np.zeros((130, 8))
    x[[0, 129], 3] = 1.0
    dy = np.zeros((130, 16))
    dy[[0, 129], 5] = [2.0, 3.0]
    a, b = X.quant_cols(dy, [0, 130], 2), X.quant_cols(x, [0, 130], 2)
    g = X.expert_wgrad(*a, *b, [0, 130])[0]
    assert g[5, 3] == 5.0 and np.count_nonzero(g) == 1


def test_clip_by_hand():
    norm, out = X.clip([np.array([3.0]), np.array([4.0, 0.0])], 2.5)
    assert norm == 5.0 and abs(out[1][0] - 4.0 * 2.5 / 5.000001) < 1e-15
    assert X.clip([np.array([0.3])], 1.0)[1][0][0] == 0.3
