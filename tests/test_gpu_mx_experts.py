"""The pass through MXFP4 experts on the GPU against the fp64 oracle, alone and with the routing
and the quantization it is used with.

The oracle's tolerance follows from fp32 sums of k products (each addition off by at most 2^-23
of the running magnitude: k 2^-23 of the sum of magnitudes) and from the 4-bit codes of h that
such an error can turn; the sum over a token's experts adds at most 2^-23 per term, and the output
rounds by half a step."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_calibration_moe_amd  # noqa: F401  (fails loudly if the library is missing)


class Block:
    def __init__(self, seed, d, f, E, K, shared, max_tokens):
        import gptq_calibration_moe_amd as clha
        rng = np.random.default_rng(seed)
        self.rng, self.d, self.f, self.E, self.K, self.shared = rng, d, f, E, K, shared
        self.ctx = clha.Context(d, E, K, shared, max_tokens, device=dev())
        slots = E + shared
        self.wgu = oracle.mx_quantize(rng.normal(0, d ** -0.5, (slots, 2 * f, d)))
        self.wd = oracle.mx_quantize(rng.normal(0, f ** -0.5, (slots, d, f)))
        self.dev = [to_dev(v) for v in (*self.wgu, *self.wd)]
        self.gu_values, self.d_values = oracle.mx_values(*self.wgu), oracle.mx_values(*self.wd)

    def tokens(self, n):
        x = torch.from_numpy(self.rng.normal(size=(n, self.d)).astype(np.float32)).to(dev()).bfloat16()
        l = self.rng.normal(0, 1.5, (n, self.E)) + self.rng.normal(0, 0.7, self.E)
        topk, w = oracle.route_scores(l, self.K)
        return x, topk, w.astype(np.float32)

    def run(self, x, topk, w, **kw):
        return self.ctx.mx_experts(x, to_dev(topk), to_dev(w), *self.dev, **kw)

    def check(self, got, x, topk, w):
        n = x.shape[0]
        terms = self.K + self.shared
        want, tol = oracle.mx_experts(x.double().cpu().numpy(), topk, w, self.gu_values, self.d_values, self.E,
                                      sum_eps=max(self.d, self.f) * 2.0 ** -23,
                                      pair_eps=2 / 65534 + 2.0 ** -23 if got.dtype == torch.bfloat16 else 0.0,
                                      add_eps=(terms + 1) * 2.0 ** -23)   # a product and terms - 1 sums, 2^-24 each
        tol = tol + (np.abs(want) + tol) * (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24)
        g = got.double().cpu().numpy()
        assert g.shape == want.shape and np.isfinite(g).all()
        off = np.abs(g - want) - tol
        assert off.max() <= 0, (n, float(off.max()), float(tol.max()))


CASES = [(128, 128, 4, 2, 0, 1), (128, 128, 4, 2, 1, 2), (256, 128, 3, 1, 2, 5), (256, 384, 8, 2, 0, 16),
         (384, 256, 5, 3, 1, 17), (256, 128, 16, 16, 1, 9), (128, 256, 1, 1, 0, 33), (128, 128, 7, 3, 2, 65),
         (256, 640, 4, 2, 1, 100), (640, 128, 6, 2, 0, 129), (256, 256, 4, 2, 1, 300), (128, 128, 3, 2, 0, 700),
         (256, 128, 2, 2, 2, 513), (128, 384, 200, 8, 0, 64)]


@pytest.mark.parametrize("d,f,E,K,shared,n", CASES)
def test_experts_match_oracle(d, f, E, K, shared, n):
    b = Block(d + f + E + n, d, f, E, K, shared, n)
    x, topk, w = b.tokens(n)
    b.check(b.run(x, topk, w, dtype=torch.float32), x, topk, w)
    b.check(b.run(x, topk, w), x, topk, w)


@pytest.mark.parametrize("n", [1, 3, 40, 400])
def test_ids_that_name_no_expert_and_experts_named_twice(n):
    """Masked tokens give the shared experts' answer alone, or zeros; a repeated expert counts twice."""
    for shared in (0, 1):
        b = Block(50 + n, 128, 128, 6, 3, shared, n)
        x, topk, w = b.tokens(n)
        topk = topk.copy()
        topk[::3] = [-1, 6, 2 ** 31 - 1]
        topk[1::3] = [2, 2, 2]
        topk[2::3, 1] = -(2 ** 31)
        got = b.run(x, topk, w, dtype=torch.float32)
        b.check(got, x, topk, w)
        if not shared:
            assert not got[::3].any()
    none = np.full_like(topk, -1)
    b.check(b.run(x, none, w, dtype=torch.float32), x, none, w)


def test_all_tokens_to_one_expert_and_one_token_each():
    b = Block(60, 128, 128, 64, 1, 0, 300)
    x, topk, w = b.tokens(300)
    one = np.full_like(topk, 63)
    b.check(b.run(x, one, w, dtype=torch.float32), x, one, w)
    each = (np.arange(300) % 64).astype(np.int32)[:, None]
    b.check(b.run(x, each, w, dtype=torch.float32), x, each, w)


def test_no_tokens():
    b = Block(61, 128, 128, 4, 2, 1, 4)
    assert b.run(torch.empty(0, 128, dtype=torch.bfloat16, device=dev()), np.zeros((0, 2), np.int32),
                 np.zeros((0, 2), np.float32)).shape == (0, 128)


def test_rows_behind_the_last_token_stay():
    b = Block(62, 256, 128, 4, 2, 1, 21)
    x, topk, w = b.tokens(21)
    out = torch.full((22, 256), 5.0, device=dev())
    b.run(x, topk, w, dtype=torch.float32, out=out[:21])
    assert bool((out[21] == 5.0).all())
    b.check(out[:21], x, topk, w)


def test_large_values_and_zero_tokens():
    """A token of zeros answers zeros; h past fp32's range is a NaN block and spoils its own token only."""
    b = Block(63, 128, 128, 4, 2, 0, 40)
    x, topk, w = b.tokens(40)
    x[3] = 0
    x[7] = 3e38
    got = b.run(x, topk, w, dtype=torch.float32)
    assert not got[3].any()
    keep = [i for i in range(40) if i != 7]
    assert bool(torch.isfinite(got[keep]).all())
    b.check(got[keep], x[keep], topk[keep], w[keep])


@pytest.mark.parametrize("n", [1, 30, 500])
def test_same_bits_on_every_run_workspace_and_stream(n):
    b = Block(70 + n, 256, 256, 12, 3, 1, n)
    x, topk, w = b.tokens(n)
    tk, wt = to_dev(topk), to_dev(w)
    want = b.ctx.mx_experts(x, tk, wt, *b.dev, dtype=torch.float32)
    need = b.ctx.mx_experts_workspace_bytes(n, b.f)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev())           # nothing in it is read before written
    assert torch.equal(b.ctx.mx_experts(x, tk, wt, *b.dev, dtype=torch.float32, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.ctx.mx_experts(x, tk, wt, *b.dev, dtype=torch.float32, stream=s)
    again = b.ctx.mx_experts(x, tk, wt, *b.dev, dtype=torch.float32)         # both at once, a workspace each
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


@pytest.mark.parametrize("n", [2, 150])
def test_block_answer_in_a_captured_graph(n):
    """Quantize the experts, then route and answer in one graph, replayed on new inputs."""
    b = Block(80 + n, 256, 128, 16, 4, 1, n)
    logits = torch.randn(n, 16, generator=torch.Generator(device=dev()).manual_seed(1), device=dev())
    x, _, _ = b.tokens(n)
    bias = torch.linspace(-0.1, 0.1, 16, device=dev())

    def step():
        topk, w = b.ctx.route(logits, score="sigmoid", bias=bias, groups=4, top_groups=2, group_score="top2", scale=2.0)
        return b.ctx.mx_experts(x, topk, w, *b.dev, dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for seed in (2, 3, 4):
        gen = torch.Generator(device=dev()).manual_seed(seed)
        logits.copy_(torch.randn(n, 16, generator=gen, device=dev()))
        x.copy_(torch.randn(n, 256, generator=gen, device=dev()))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, step())
        torch.cuda.synchronize()
    topk, w = oracle.route_scores(logits.cpu().numpy(), 4, score="sigmoid", bias=bias.cpu().numpy(), groups=4,
                                  top_groups=2, group_score="top2", scale=2.0)
    b.check(got, x, topk, w.astype(np.float32))


def test_refusals():
    import gptq_calibration_moe_amd as clha
    b = Block(90, 128, 128, 4, 2, 1, 8)
    x, topk, w = b.tokens(8)
    tk, wt = to_dev(topk), to_dev(w)
    out = torch.empty(8, 128, device=dev())
    ws = torch.empty(b.ctx.mx_experts_workspace_bytes(8, 128), dtype=torch.uint8, device=dev())
    good = dict(n=8, f=128, x=x.data_ptr(), topk=tk.data_ptr(), w=wt.data_ptr(), gu=b.dev[0].data_ptr(),
                gs=b.dev[1].data_ptr(), d=b.dev[2].data_ptr(), ds=b.dev[3].data_ptr(), out=out.data_ptr(), dt=clha.F32,
                ws=ws.data_ptr(), nb=ws.numel())

    def call(**kw):
        a = {**good, **kw}
        return clha.lib.clha_mx_experts(b.ctx._h, a["n"], a["f"], a["x"], a["topk"], a["w"], a["gu"], a["gs"], a["d"],
                                        a["ds"], a["out"], a["dt"], a["ws"], a["nb"],
                                        torch.cuda.current_stream().cuda_stream)
    assert call() == clha.OK
    for kw in (dict(n=-1), dict(n=9), dict(f=0), dict(f=64), dict(f=192), dict(f=8320)):
        assert call(**kw) == clha.ERR_SHAPE, kw
    for k in ("x", "topk", "w", "gu", "gs", "d", "ds", "out", "ws"):
        assert call(**{k: None}) == clha.ERR_INVALID_ARG, k
        assert call(**{k: good[k] + 2}) == clha.ERR_ALIGN, k
    assert call(dt=9) == clha.ERR_INVALID_ARG
    assert call(nb=ws.numel() - 1) == clha.ERR_WORKSPACE
    assert call(n=0, x=None) == clha.OK
    assert b.ctx.mx_experts_workspace_bytes(9, 128) == b.ctx.mx_experts_workspace_bytes(8, 100) == 0
    with pytest.raises(ValueError):
        b.ctx.mx_experts(x, tk[:, :1].contiguous(), wt, *b.dev)
    with pytest.raises(ValueError):
        b.ctx.mx_experts(x, tk, wt, b.dev[0][:4].contiguous(), *b.dev[1:])
    with pytest.raises(TypeError):
        b.ctx.mx_experts(x, tk.long(), wt, *b.dev)
    torch.cuda.synchronize()
    b.check(out, x, topk, w)


def test_other_stages_are_timed():
    b = Block(91, 128, 128, 4, 2, 0, 8)
    x, topk, w = b.tokens(8)
    b.ctx.set_timing(True)
    b.run(x, topk, w)
    b.ctx.mx_quantize(x)
    t = b.ctx.read_timing()
    b.ctx.set_timing(False)
    assert t["mx_experts"][1] == 1 and t["mx_quantize"][1] == 1 and t["mx_experts"][0] > 0


@pytest.mark.parametrize("d,f", [(128, 8192), (8192, 128), (2048, 1408)])
def test_passes_beyond_one_launch_are_refused(d, f):
    """Threads of a launch are counted in 32 bits: the pairs times the wider of d and f
    end at 2^36."""
    import gptq_calibration_moe_amd as clha
    ctx = clha.Context(d, 4, 2, 1, 1 << 27)
    most = min((1 << 27) // 3, (1 << 36) // (3 * max(d, f)), (1 << 33) // d)
    assert ctx.mx_experts_workspace_bytes(most, f) > 0
    assert ctx.mx_experts_workspace_bytes(most + 1, f) == 0
    t = torch.zeros(64, dtype=torch.uint8, device=dev())
    p = t.data_ptr()
    st = clha.lib.clha_mx_experts(ctx._h, most + 1, f, p, p, p, p, p, p, p, p, clha.F32, p, 64, None)
    assert st == clha.ERR_SHAPE
    for tile, threads in ((128, 256), (256, 512)):
        tiles = 3 * most // tile + 4 + 1 + 32
        assert tiles * (f // (tile // 2)) * threads < 1 << 32 and tiles * -(-d // tile) * threads < 1 << 32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_pairs_than_one_share_of_the_plan_each(dtype):
    """A plan of 300 thousand pairs: 500 tokens over and over give the same rows each time."""
    b = Block(91, 128, 128, 16, 6, 1, 50000)
    x, topk, w = b.tokens(500)
    topk[::7, 3] = -1
    many = b.run(x.repeat(100, 1), np.tile(topk, (100, 1)), np.tile(w, (100, 1)), dtype=dtype).view(100, 500, 128)
    b.check(many[0], x, topk, w)
    assert torch.equal(many, many[:1].expand_as(many))


# mean positions of a slot from 6 to 192 and beyond: every tile, with scale rows of whole words
# (d, f from 512) and without, contractions that end inside a stage
TILES = [(512, 512, 8, 2, 1, 60), (640, 128, 5, 1, 0, 33), (128, 640, 6, 3, 0, 40), (384, 384, 4, 2, 2, 50),
         (512, 640, 4, 2, 1, 80), (640, 128, 3, 1, 1, 150), (128, 512, 4, 4, 0, 60), (256, 384, 5, 2, 0, 160),
         (1408, 512, 4, 2, 0, 200), (512, 128, 4, 2, 1, 300), (128, 512, 2, 1, 0, 200), (896, 640, 3, 2, 1, 350)]


@pytest.mark.parametrize("d,f,E,K,shared,n", TILES)
def test_every_tile_matches_oracle(d, f, E, K, shared, n):
    b = Block(d + f + E + n + 1, d, f, E, K, shared, n)
    x, topk, w = b.tokens(n)
    topk[1::9, 0] = -1
    b.check(b.run(x, topk, w, dtype=torch.float32), x, topk, w)
    b.check(b.run(x, topk, w), x, topk, w)
