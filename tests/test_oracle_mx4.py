"""Pins of the microscaled 4-bit oracle and of the selection of experts."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.cpu


def test_every_code_and_scale():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    v = oracle.mx4_values(codes, np.full((16, 1), 128, np.uint8))
    table = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    for b in range(256):
        assert v.flat[2 * b] == 2 * table[b & 15] and v.flat[2 * b + 1] == 2 * table[b >> 4]
    ends = oracle.mx4_values(np.full((4, 16), 0x22, np.uint8), np.array([[0], [1], [254], [255]], np.uint8))
    assert ends[0, 0] == 2.0 ** -127 and ends[1, 0] == 2.0 ** -126 and ends[2, 0] == 2.0 ** 127
    assert np.isnan(ends[3]).all()


def test_ties_go_to_the_even_code_and_the_top_saturates():
    x = np.zeros((1, 32))
    x[0, :10] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7.9, -2.5]
    c, s = oracle.mx4_quantize(x)
    assert s[0, 0] == 127
    assert oracle.mx4_values(c, s)[0, :10].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6, -2]
    c, s = oracle.mx4_quantize(2.0 ** 20 * x)
    assert s[0, 0] == 147 and oracle.mx4_values(c, s)[0, 6] == 4 * 2.0 ** 20


def test_zero_tiny_and_infinite_groups():
    x = np.zeros((5, 32))
    x[1, 0] = 2.0 ** -140                                # under half the smallest step: 0
    x[2, 0] = 2.0 ** -126
    x[3, 5] = np.inf
    x[4, 6] = np.nan
    c, s = oracle.mx4_quantize(x)
    assert s[:, 0].tolist() == [0, 0, 0, 255, 255] and not c[3:].any()
    v = oracle.mx4_values(c, s)
    assert not v[:2].any() and v[2, 0] == 2.0 ** -126 and np.isnan(v[3:]).all()


def test_error_of_a_group_is_at_most_a_quarter_of_its_largest():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(64, 256)) * np.exp(3 * rng.normal(size=(64, 1)))
    v = oracle.mx4_values(*oracle.mx4_quantize(x))
    a = np.abs(x.reshape(64, 8, 32)).max(-1)[..., None]
    assert (np.abs(v - x).reshape(64, 8, 32) <= a / 4).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_selection_without_groups_is_a_stable_sort(score):
    rng = np.random.default_rng(5)
    l = rng.integers(-4, 5, size=(50, 40)).astype(np.float64)      # many ties
    ids, w = oracle.moe_select(l, 7, score)
    want = np.argsort(-l, axis=1, kind="stable")[:, :7]
    assert (ids == want).all()
    t = torch.from_numpy(l)
    s = (torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)).numpy()
    assert np.abs(w - np.take_along_axis(s, want, 1)).max() < 1e-14


def test_selection_by_groups_by_hand():
    l = np.log(np.array([[8, 1, 1, 1, 5, 4, 1, 1, 7, 1, 1, 1.]]) / 32)     # softmax: these over 32
    ids, w = oracle.moe_select(l, 3, groups=3, top_groups=2, group_best=1)
    assert ids.tolist() == [[0, 8, 1]] and np.allclose(w * 32, [[8, 7, 1]])
    ids, w = oracle.moe_select(l, 3, groups=3, top_groups=2, group_best=2, renormalize=True, scale=2)
    assert ids.tolist() == [[0, 4, 5]] and np.allclose(w, [[16 / 17, 10 / 17, 8 / 17]])
    bias = np.zeros(12)
    bias[11] = 1                                         # seen by the choice, not by the weight
    ids, w = oracle.moe_select(l, 2, bias=bias)
    assert ids.tolist() == [[11, 0]] and np.allclose(w * 32, [[1, 8]])


def test_masked_experts_come_last_with_weight_zero():
    l = np.array([[-np.inf, 1, -np.inf, 0], [-np.inf] * 4, [np.nan, 1, 2, 3]])
    ids, w = oracle.moe_select(l, 3, renormalize=True)
    assert ids.tolist() == [[1, 3, 0], [0, 1, 2], [3, 2, 1]]
    assert w[0, 2] == 0 and not w[1].any() and np.isnan(w[2]).all()


def test_gated_activations_match_torch():
    g, u = np.random.default_rng(1).normal(size=(2, 1000)) * 4
    t = torch.from_numpy(g)
    assert np.abs(oracle.gated(g, u, "silu") - (torch.nn.functional.silu(t).numpy() * u)).max() < 1e-13
    assert np.abs(oracle.gated(g, u, "gelu_tanh")
                  - (torch.nn.functional.gelu(t, approximate="tanh").numpy() * u)).max() < 1e-13
