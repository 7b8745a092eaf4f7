"""Routing by scores on the GPU against the fp64 oracle: expert ids equal, weights within their
rounding.

Weights are formed in 64 bits and rounded once (2^-24 relative), except that a softmax without
renormalization divides by a sum of fp32 exponentials: each has a relative error of at most
2 units in the last place plus its argument's rounding d 2^-24, which enters the sum weighted by
e^-d (d e^-d <= 0.37), so the quotient is off by less than 2^-20.  Tiny results below the fp32
normal range round to the subnormal grid (2^-150)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_util import bits_to_dev, dev, hess_err, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_calibration_moe_amd  # noqa: F401  (fails loudly if the library is missing)


def _ctx(E, K, n=70000, d=128, shared=0):
    import gptq_calibration_moe_amd as clha
    return clha.Context(d, E, K, shared, n, device=dev())


def _check(ctx, l, K, **kw):
    bias = kw.pop("bias", None)
    topk, w = ctx.route(to_dev(l), bias=None if bias is None else to_dev(bias), **kw)
    ctx.sync()
    want, ww = oracle.route_scores(l, K, bias=bias, **kw)
    assert np.array_equal(topk.cpu().numpy(), want)
    plain = kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True)
    rtol = 2.0 ** -20 if plain else 2.0 ** -23
    assert np.all(np.abs(w.cpu().numpy() - ww) <= rtol * np.abs(ww) + 2.0 ** -149)


SHAPES = [(1, 8, 2, 1, 1), (3, 1, 1, 1, 1), (17, 16, 16, 4, 4), (16, 20, 3, 5, 2), (257, 60, 6, 6, 3),
          (1000, 64, 6, 8, 4), (33, 127, 5, 1, 1), (64, 130, 16, 13, 2), (129, 256, 8, 8, 4), (40, 256, 1, 256, 7),
          (31, 96, 4, 3, 1)]


@pytest.mark.parametrize("n,E,K,groups,top", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_matches_oracle(n, E, K, groups, top, score, biased):
    rng = np.random.default_rng(n * 1000 + E)
    l = (rng.normal(0, 1.5, (n, E)) + rng.normal(0, 0.7, E)).astype(np.float32)
    bias = rng.normal(0, 0.05, E).astype(np.float32) if biased else None
    ctx = _ctx(E, K)
    for group_score in ("max", "top2") if groups > 1 else ("max",):
        for renorm in (True, False):
            _check(ctx, l, K, score=score, bias=bias, groups=groups, top_groups=top, group_score=group_score,
                   renormalize=renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_equal_close_and_extreme_logits(score, biased):
    """Ties, logits one unit apart, masks of the type's lowest value, saturated sigmoids, signed zeros."""
    E, K = 64, 6
    rng = np.random.default_rng(7)
    lowest = np.finfo(np.float32).min
    l = np.zeros((8, E), np.float32)
    l[1] = rng.integers(0, 3, E)                                   # many ties
    l[2] = np.nextafter(np.float32(1.0), np.float32(2.0)) * (rng.random(E) < 0.5) + 1.0
    l[3] = lowest
    l[3, 5], l[3, 40] = 1.0, 2.0                                   # fewer open experts than K
    l[4] = lowest                                                  # none open
    l[5] = rng.normal(0, 1, E)
    l[5, ::2] = -0.0
    l[5, 1::4] = 0.0
    l[6] = 1.0 + np.arange(E, dtype=np.float32)[::-1] * 2.0 ** -23   # neighbouring floats
    l[7] = rng.normal(0, 30, E)                                    # far apart: many scores next to 0 or 1
    bias = np.where(np.arange(E) % 3 == 0, 0.25, 0.0).astype(np.float32) if biased else None
    ctx = _ctx(E, K)
    for renorm in (True, False):
        _check(ctx, l, K, score=score, bias=bias, renormalize=renorm)
        _check(ctx, l[[0, 1, 2, 5, 6, 7]], K, score=score, bias=bias, renormalize=renorm, groups=8, top_groups=3,
               group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (256, 8, 4), (96, 4, 2), (128, 64, 5), (40, 5, 2)])
def test_groups_and_choices_next_to_each_other(score, group_score, E, groups, top):
    """Groups whose marks differ by a few units in the last place or not at all, with distinct members and
    with close ones; lists of close choices longer and shorter than the 16 lanes of a token."""
    rng = np.random.default_rng(E + groups)
    per, K, n = E // groups, 6 if top * (E // groups) >= 6 else top * (E // groups), 120
    l = rng.normal(-2.0, 0.7, (n, E)).astype(np.float32)
    for t in range(n):
        v = l[t].reshape(groups, per)
        if t % 3 < 2:                                     # the same largest members in every group, moved a little
            big = np.float32(1.5) + np.arange(min(per, 2), dtype=np.float32) * np.float32(0.25)
            v[:, :big.size] = big
            v[:, 0] += rng.integers(0, 3, groups) * np.float32(2.0 ** -22) * (t % 3)
            rng.shuffle(v, axis=1)
        else:                                             # everything close
            v[:] = np.float32(0.5) + rng.integers(0, 6, (groups, per)) * np.float32(2.0 ** -23)
    bias = (rng.integers(0, 2, E) * np.float32(0.125)).astype(np.float32)
    ctx = _ctx(E, K)
    for b in (None, bias, np.zeros(E, np.float32)):
        _check(ctx, l, K, score=score, bias=b, groups=groups, top_groups=top, group_score=group_score)
        _check(ctx, l, K, score=score, bias=b)


def test_many_tokens_and_optional_outputs():
    E, K, n = 256, 8, 40961
    rng = np.random.default_rng(3)
    l = rng.normal(0, 1.5, (n, E)).astype(np.float32)
    b = rng.normal(0, 0.05, E).astype(np.float32)
    ctx = _ctx(E, K)
    _check(ctx, l, K, score="sigmoid", bias=b, groups=8, top_groups=4, group_score="top2")
    import gptq_calibration_moe_amd as clha
    ld = to_dev(l)
    topk = torch.empty(n, K, dtype=torch.int32, device=dev())
    d = clha.route_desc()
    st = clha.lib.clha_route(ctx._h, ctypes.byref(d), n, ld.data_ptr(), None, topk.data_ptr(), None,
                             torch.cuda.current_stream().cuda_stream)
    assert st == clha.OK
    assert np.array_equal(topk.cpu().numpy(), oracle.route_scores(l, K)[0])


def test_no_tokens_and_unaligned_rows():
    ctx = _ctx(64, 6)
    topk, w = ctx.route(torch.empty(0, 64, device=dev()))
    assert topk.shape == w.shape == (0, 6)
    rng = np.random.default_rng(9)
    flat = torch.from_numpy(rng.normal(size=5 * 64 + 1).astype(np.float32)).to(dev())
    view = flat[1:].view(5, 64)                       # rows 4-byte aligned only
    topk, _ = ctx.route(view)
    assert np.array_equal(topk.cpu().numpy(), oracle.route_scores(view.cpu().numpy(), 6)[0])


def test_non_finite_logits_are_latched_and_stay_in_range():
    import gptq_calibration_moe_amd as clha
    ctx = _ctx(20, 4)
    l = np.random.default_rng(1).normal(size=(6, 20)).astype(np.float32)
    good = oracle.route_scores(l, 4)[0]
    l[2] = np.nan
    l[4, 3] = np.inf
    for bias in (None, to_dev(np.zeros(20, np.float32))):
        for groups in (1, 5):
            topk, _ = ctx.route(to_dev(l), bias=bias, groups=groups, top_groups=groups)
            with pytest.raises(clha.ClhaError) as ei:
                ctx.sync()
            assert ei.value.status == clha.ERR_NONFINITE and "routing" in str(ei.value)
            ctx.sync()                                   # the latch was cleared
            t = topk.cpu().numpy()
            assert t.min() >= 0 and t.max() < 20
            assert all(len(set(r)) == 4 for r in t.tolist())
            assert np.array_equal(t[[0, 1, 3, 5]], good[[0, 1, 3, 5]])
    bad = torch.zeros(20, device=dev())
    bad[7] = float("nan")
    ctx.route(torch.zeros(3, 20, device=dev()), bias=bad)
    with pytest.raises(clha.ClhaError):
        ctx.sync()


def test_refusals():
    import gptq_calibration_moe_amd as clha
    ctx = _ctx(64, 6)
    l = torch.zeros(4, 64, device=dev())
    for kw, st in ((dict(groups=5), clha.ERR_SHAPE), (dict(groups=0), clha.ERR_SHAPE),
                   (dict(groups=8, top_groups=0), clha.ERR_SHAPE), (dict(groups=8, top_groups=9), clha.ERR_SHAPE),
                   (dict(groups=16, top_groups=1), clha.ERR_SHAPE),          # four experts left for six choices
                   (dict(scale=float("inf")), clha.ERR_INVALID_ARG), (dict(scale=float("nan")), clha.ERR_INVALID_ARG)):
        with pytest.raises(clha.ClhaError) as ei:
            ctx.route(l, **kw)
        assert ei.value.status == st, kw
    d = clha.route_desc()
    lib, h, p = clha.lib, ctx._h, l.data_ptr()
    assert lib.clha_route(h, None, 4, p, None, p, None, None) == clha.ERR_INVALID_ARG
    assert lib.clha_route(h, ctypes.byref(d), 4, None, None, p, None, None) == clha.ERR_INVALID_ARG
    assert lib.clha_route(h, ctypes.byref(d), 4, p, None, None, None, None) == clha.ERR_INVALID_ARG
    assert lib.clha_route(h, ctypes.byref(d), 4, p + 2, None, p, None, None) == clha.ERR_ALIGN
    assert lib.clha_route(h, ctypes.byref(d), -1, p, None, p, None, None) == clha.ERR_SHAPE
    assert lib.clha_route(h, ctypes.byref(d), (1 << 27) + 1, p, None, p, None, None) == clha.ERR_SHAPE
    for field, v in (("score", 2), ("score", -1), ("renormalize", 2)):
        e = clha.route_desc()
        setattr(e, field, v)
        assert lib.clha_route(h, ctypes.byref(e), 4, p, None, p, None, None) == clha.ERR_INVALID_ARG
    e = clha.route_desc(groups=2)
    e.group_score = 5
    e.top_groups = 2
    assert lib.clha_route(h, ctypes.byref(e), 4, p, None, p, None, None) == clha.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ctx.route(torch.zeros(4, 63, device=dev()))
    with pytest.raises(TypeError):
        ctx.route(l.double())
    with pytest.raises(ValueError):
        ctx.collect_hessians(0, torch.zeros(4, 128, dtype=torch.bfloat16, device=dev()), l, bias=l[0])


def test_collection_by_scores_matches_oracle():
    """clha_collect_hessians_scored: the sums, counts and lists of the chosen experts."""
    import gptq_calibration_moe_amd as clha
    import gen
    d, E, K, n = 256, 20, 3, 700
    rng = np.random.default_rng(21)
    x = gen.bf16_bits(rng.normal(size=(n, d)).astype(np.float32))
    l = rng.normal(0, 1.5, (n, E)).astype(np.float32)
    b = rng.normal(0, 0.3, E).astype(np.float32)
    ctx = _ctx(E, K, n=n, d=d, shared=1)
    S, cnt = ctx.new_layer_buffers()
    ctx.register_layer(0, S, cnt)
    kw = dict(score="sigmoid", groups=5, top_groups=2, group_score="top2")
    topk = torch.empty(n, K, dtype=torch.int32, device=dev())
    w = torch.empty(n, K, dtype=torch.float32, device=dev())
    off = torch.empty(E + 1, dtype=torch.int64, device=dev())
    ids = torch.empty(n * K, dtype=torch.int32, device=dev())
    ctx.collect_hessians(0, bits_to_dev(x), to_dev(l), topk_out=topk, offsets_out=off, token_ids_out=ids,
                         routing=clha.route_desc(**kw), bias=to_dev(b), weights_out=w)
    ctx.sync()
    want, ww = oracle.route_scores(l, K, bias=b, **kw)
    assert np.array_equal(topk.cpu().numpy(), want)
    assert np.all(np.abs(w.cpu().numpy() - ww) <= 2.0 ** -23 * ww)
    for e in range(E):
        t = np.nonzero((want == e).any(axis=1))[0]
        o = off.cpu().numpy()
        assert np.array_equal(ids.cpu().numpy()[o[e]:o[e + 1]], t)
        assert int(cnt[e]) == t.size
        R = oracle.gram(gen.bf16_value(x[t])) if t.size else np.zeros((d, d))
        assert hess_err(np.tril(S[e].cpu().numpy()), np.tril(R)) <= 1e-4
    assert int(cnt[E]) == n
    assert hess_err(np.tril(S[E].cpu().numpy()), np.tril(oracle.gram(gen.bf16_value(x)))) <= 1e-4
    nan = l.copy()
    nan[3, 3] = np.nan
    ctx.collect_hessians(0, bits_to_dev(x), to_dev(nan), routing=clha.route_desc(**kw), bias=to_dev(b))
    with pytest.raises(clha.ClhaError) as ei:
        ctx.sync()
    assert "layer 0" in str(ei.value)
