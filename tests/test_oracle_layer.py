"""Pins of the layer operators' oracle: closed forms, numpy's own convolution, splits of a row."""
import numpy as np
import pytest

from oracle import layer as O


def test_codes_reconstruct_the_norm_and_use_the_whole_range():
    rs = np.random.default_rng(0)
    v, w = rs.standard_normal((7, 48)) * 3, rs.uniform(0.5, 1.5, 48)
    r = O.norm_codes(v, w)
    codes = np.rint(r["pos"])
    assert np.abs(codes).max(axis=1).tolist() == [127.0] * 7
    assert np.abs(codes * r["scale"][:, None] - r["u"]).max() <= r["scale"].max() / 2 * (1 + 1e-12)
    # the root mean square of an unweighted row is 1 (up to eps)
    np.testing.assert_allclose(np.mean(O.norm_codes(v)["u"] ** 2, axis=1), 1.0, atol=1e-5)


def test_codes_do_not_depend_on_the_root_mean_square():
    rs = np.random.default_rng(1)
    v = rs.standard_normal((3, 32))
    np.testing.assert_allclose(O.norm_codes(v)["pos"], O.norm_codes(1000 * v)["pos"], rtol=1e-12)
    np.testing.assert_allclose(O.norm_codes(v)["pos"], v * 127 / np.abs(v).max(axis=1, keepdims=True), rtol=1e-12)


def test_a_row_of_zeros_has_scale_one():
    r = O.norm_codes(np.zeros((2, 16)))
    assert r["scale"].tolist() == [1.0, 1.0] and not r["pos"].any()


def test_gate_closed_forms():
    np.testing.assert_allclose(O.gate([2.0, 2.0, 2.0, 2.0], [0.0, 40.0, -800.0, 1.0]),
                               [0.0, 80.0, 0.0, 2.0 / (1 + np.exp(-1.0))], rtol=1e-15)


def test_matmul_by_hand():
    r = O.matmul([[1, -2], [3, 4]], [0.5, 2.0], [[5, 6], [-7, 8], [1, 1]], [1.0, 0.25, 2.0], [1.0, 0.0, -1.0])
    np.testing.assert_array_equal(r["out"], [[0.5 * -7 + 1, 0.125 * -23, 1.0 * -1 - 1],
                                             [2.0 * 39 + 1, 0.5 * 11, 4.0 * 7 - 1]])


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_is_numpys_convolution_of_the_extended_row(W):
    rs = np.random.default_rng(W)
    L, C = 9, 3
    x, w, st = rs.standard_normal((1, L, C)), rs.standard_normal((W, C)), rs.standard_normal((1, W - 1, C))
    r = O.conv(x, w, None, st)
    for c in range(C):
        line = np.concatenate([st[0, :, c], x[0, :, c]])
        np.testing.assert_allclose(r["u"][0, :, c], np.convolve(line, w[::-1, c], "valid"), rtol=1e-12)
    np.testing.assert_array_equal(r["state"][0], x[0, L - W + 1:])


def test_conv_split_anywhere_and_padding():
    rs = np.random.default_rng(5)
    b, L, C, W = 2, 7, 4, 4
    x, w, bias = rs.standard_normal((b, L, C)), rs.standard_normal((W, C)), rs.standard_normal(C)
    whole = O.conv(x, w, bias)
    for cut in range(L + 1):
        a = O.conv(x[:, :cut], w, bias)
        z = O.conv(x[:, cut:], w, bias, a["state"])
        np.testing.assert_allclose(np.concatenate([a["out"], z["out"]], 1), whole["out"], rtol=1e-13)
        np.testing.assert_array_equal(z["state"], whole["state"])
    lens = [3, 0]
    pad = O.conv(x, w, bias, None, lens, rs.standard_normal((b, L, 2)), np.zeros(2))
    np.testing.assert_array_equal(pad["out"][0, :3], whole["out"][0, :3])
    assert not pad["out"][0, 3:].any() and not pad["out"][1].any() and not pad["dt"][1].any()
    np.testing.assert_array_equal(pad["state"][0], x[0, :3])
    assert not pad["state"][1].any()


def test_softplus_closed_forms():
    np.testing.assert_allclose(O.softplus([0.0, 100.0, -100.0]), [np.log(2.0), 100.0, np.exp(-100.0)], rtol=1e-14)
