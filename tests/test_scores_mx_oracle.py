"""Pins of the oracle's routing by scores and MXFP4 (values worked out by hand), the host side
of their binding, and that the entry points refuse a null context."""
import ctypes

import numpy as np
import pytest

import oracle


def test_softmax_weights_by_hand():
    l = np.log(np.array([[1.0, 4.0, 3.0, 2.0]]))
    topk, w = oracle.route_scores(l, 2, renormalize=False)
    assert topk.tolist() == [[1, 2]] and np.allclose(w, [[0.4, 0.3]])
    topk, w = oracle.route_scores(l, 2, scale=2.0)
    assert np.allclose(w, [[8 / 7, 6 / 7]])


def test_bias_moves_the_choice_but_not_the_weight():
    l = np.zeros((1, 3))
    topk, w = oracle.route_scores(l, 1, score="sigmoid", bias=[0.0, 0.0, 0.5], renormalize=False)
    assert topk.tolist() == [[2]] and np.allclose(w, 0.5)


def test_ties_go_to_the_lower_index_and_group():
    l = np.zeros((1, 8))
    assert oracle.route_scores(l, 3)[0].tolist() == [[0, 1, 2]]
    assert oracle.route_scores(l, 3, groups=4, top_groups=2, group_score="top2")[0].tolist() == [[0, 1, 2]]


def test_groups_by_largest_and_by_top_two():
    l = np.log(np.array([[8.0, 0.1, 5.0, 4.9, 1.0, 1.0]]))
    assert oracle.route_scores(l, 2, groups=3, top_groups=1)[0].tolist() == [[0, 1]]
    assert oracle.route_scores(l, 2, groups=3, top_groups=1, group_score="top2")[0].tolist() == [[2, 3]]


def test_weights_are_zero_where_the_chosen_scores_are():
    _, w = oracle.route_scores(np.full((1, 2), -1e30), 2, score="sigmoid")
    assert w.tolist() == [[0.0, 0.0]]
    _, w = oracle.route_scores(np.array([[0.0, -3e38, -3e38]]), 2)
    assert w.tolist() == [[1.0, 0.0]]


def test_mx_levels_ties_and_scale():
    x = np.zeros((1, 32))
    x[0, :10] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1, 7.9]   # largest 7.9: 2^(2-2)
    codes, scales = oracle.mx_quantize(x)
    assert scales.tolist() == [[127]]
    assert oracle.mx_values(codes, scales)[0, :10].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -6, 6]
    assert codes[0, 0] == 0x06                                             # even element in the low half


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125),
                                       (3.4e38, 252), (np.inf, 255), (np.nan, 255)])
def test_mx_scale_bytes(amax, byte):
    assert int(oracle.mx_scale(np.array(amax))) == byte


def test_mx_experts_is_the_formula():
    rng = np.random.default_rng(5)
    x = oracle.mx_values(*oracle.mx_quantize(rng.normal(size=(3, 64))))
    wgu, wd = rng.normal(size=(2, 128, 64)), rng.normal(size=(2, 64, 64))
    topk, w = np.array([[0], [-1], [0]]), np.array([[0.5], [9.0], [2.0]])
    y, tol = oracle.mx_experts(x, topk, w, wgu, wd, 1)
    for t in range(3):
        want = np.zeros(64)
        for e, a in ((0, w[t, 0] * (topk[t, 0] == 0)), (1, 1.0)):
            gu = wgu[e] @ x[t]
            h = oracle.silu(gu[:64]) * gu[64:]
            want += a * (wd[e] @ oracle.mx_values(*oracle.mx_quantize(h[None]))[0])
        assert np.allclose(y[t], want)
    assert tol.min() >= 0


def test_entry_points_refuse_a_null_context():
    import gptq_calibration_moe_amd as g
    none, d = None, g.route_desc()
    assert g.lib.clha_route(none, ctypes.byref(d), 1, none, none, none, none, none) == g.ERR_INVALID_ARG
    assert g.lib.clha_collect_hessians_scored(none, 0, ctypes.byref(d), 1, none, none, none, none, none, none, none,
                                              none, 0, none) == g.ERR_INVALID_ARG
    assert g.lib.clha_mx_quantize(none, 1, 32, none, 0, 32, none, none, none) == g.ERR_INVALID_ARG
    assert g.lib.clha_mx_dequantize(none, 1, 32, none, none, none, 0, none) == g.ERR_INVALID_ARG
    assert g.lib.clha_mx_matmul(none, 1, 1, 32, none, none, none, none, none, 0, none) == g.ERR_INVALID_ARG
    assert g.lib.clha_mx_experts_workspace_bytes(none, 1, 128) == 0
    assert g.lib.clha_mx_experts(none, 1, 128, none, none, none, none, none, none, none, none, 0, none, 0,
                                 none) == g.ERR_INVALID_ARG


def test_route_desc_names():
    import gptq_calibration_moe_amd as g
    d = g.route_desc("sigmoid", groups=4, top_groups=2, group_score="top2", renormalize=False, scale=2.5)
    assert (d.score, d.n_groups, d.top_groups, d.group_score, d.renormalize, d.scale) == (1, 4, 2, 1, 0, 2.5)
    with pytest.raises(ValueError):
        g.route_desc("cosine")
    with pytest.raises(ValueError):
        g.route_desc(group_score="mean")
