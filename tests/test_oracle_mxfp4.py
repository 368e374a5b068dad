"""Pins of the MXFP4 oracle: hand values, exponent edges, error bound, the scale tile layout."""

import numpy as np

from oracle import mxfp4 as X


def row(*values):
    x = np.zeros((1, 32), np.float32)
    x[0, :len(values)] = values
    return x


def test_hand_values():
    c, s = X.quantize_rows(row(6.0, -3.0, 0.25, 0.75, -0.1, 5.0, 2.5))
    assert s.tolist() == [[127]] and c[0, :7].tolist() == [7, 13, 0, 2, 8, 6, 4]      # scale 1; ties to even
    c, s = X.quantize_rows(row(7.0, 4.0))
    assert s.tolist() == [[127]] and c[0, :2].tolist() == [7, 6]                      # 7 saturates to 6
    c, s = X.quantize_rows(row(8.0, 4.0))
    assert s.tolist() == [[128]] and c[0, :2].tolist() == [6, 4]
    c, s = X.quantize_rows(row())
    assert s.tolist() == [[0]] and not c.any()


def test_exponent_edges():
    big = np.float32(3.4028235e38)
    c, s = X.quantize_rows(row(big))
    assert s.tolist() == [[252]] and c[0, 0] == 7
    c, s = X.quantize_rows(row(2.0 ** -126))            # exponent -128 is held to -127
    assert s.tolist() == [[0]] and c[0, 0] == 4         # 2^-126 / 2^-127 = 2
    c, s = X.quantize_rows(row(np.inf, 1.0))
    assert s.tolist() == [[255]] and not c.any() and np.isnan(X.dequantize_rows(c, s)).all()


def test_error_bound():
    x = (np.random.default_rng(0).standard_normal((64, 128)) *
         np.exp2(np.random.default_rng(1).integers(-20, 20, (64, 1)))).astype(np.float32)
    c, s = X.quantize_rows(x)
    v = X.dequantize_rows(c, s)
    scale = np.repeat(np.exp2(s - 127.0), 32, axis=1)
    # half the widest step (4 to 6) below 6, up to 2 above it (values below 8 scales saturate at 6)
    assert np.all(np.abs(v - x) <= np.where(np.abs(x) <= 6 * scale, 1.0, 2.0) * scale)


def test_sf_index():
    for rows, cols in ((128, 128), (256, 384), (256, 160)):
        i = X.sf_byte_index(rows, cols)
        assert len(np.unique(i)) == i.size and i.max() < rows // 128 * -(-cols // 128) * 512
        assert i[0, 0] == 0 and i[0, 1] == 1 and i[32, 0] == 4 and i[1, 0] == 16
