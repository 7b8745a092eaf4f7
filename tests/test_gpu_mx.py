"""MXFP4 quantization and the MXFP4 product on the GPU against the fp64 oracle.

Codes and scales are equal bit for bit, and so are dequantized values.  The product sums k
products of exactly representable values in fp32, in any order, each addition off by at most one
unit in the last place (2^-23, the matrix cores may truncate): |error| <= k 2^-23 sum |a w|, plus
half a step of the output type.  Where all scales are 1 and the sum of magnitudes stays below
2^22 quarters, every partial sum is a multiple of 1/4 that fp32 holds, so the fp32 result is exact."""
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


@pytest.fixture(scope="module")
def ctx():
    import gptq_calibration_moe_amd as clha
    return clha.Context(128, 8, 2, 0, 1, device=dev())


def _as(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev())
    return t if dtype == torch.float32 else t.to(dtype)


def _check_quantize(ctx, t):
    codes, scales = ctx.mx_quantize(t)
    x = t.float().cpu().numpy().astype(np.float64)
    cw, sw = oracle.mx_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), sw)
    assert np.array_equal(codes.cpu().numpy(), cw)
    v = oracle.mx_values(cw, sw)
    for dt in (torch.float32, torch.bfloat16):
        got = ctx.mx_dequantize(codes, scales, dtype=dt).double().cpu().numpy()
        assert np.array_equal(got, v, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (37, 2048), (257, 1440), (64, 8192)])
def test_quantize_matches_oracle(ctx, dtype, rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(size=(rows, cols)) * np.exp2(rng.normal(0, 8, (rows, 1)))
    _check_quantize(ctx, _as(x, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_every_kind_of_value(ctx, dtype):
    """Borders and their neighbours, zeros, the smallest and largest numbers, NaN and infinities."""
    rng = np.random.default_rng(2)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99])
    near = np.concatenate([mids, np.nextafter(mids.astype(np.float32), np.float32(0)),
                           np.nextafter(mids.astype(np.float32), np.float32(9))])
    x = np.zeros((40, 64), np.float32)
    for r in range(20):
        e = [-126, -125, -60, 0, 100, 124][r % 6]
        x[r] = np.ldexp(rng.choice(near, 64) * rng.choice([-1, 1], 64), e)
        x[r, [0, 40]] = np.ldexp(4.0, e)
    x[20] = 0.0
    x[21] = -0.0
    x[22, :32] = np.ldexp(rng.integers(0, 1 << 20, 32).astype(np.float64), -149)   # subnormals
    x[23] = rng.choice([1.0, -1.0], 64) * np.finfo(np.float32).max
    x[24, 5] = np.nan
    x[25, 33] = np.inf
    x[26, 63] = -np.inf
    x[27] = 2.0 ** -149
    x[28] = np.ldexp(1.0, rng.integers(-149, 128, 64))
    x[29, 1] = 1.0
    x[30:] = rng.integers(0, 1 << 32, (10, 64), dtype=np.uint32).view(np.float32)  # any bits
    with np.errstate(invalid="ignore"):
        _check_quantize(ctx, _as(x, dtype))


def test_quantize_strided_rows_and_given_outputs(ctx):
    rng = np.random.default_rng(4)
    for dt, pad in ((torch.bfloat16, 8), (torch.float32, 4)):
        big = _as(rng.normal(size=(9, 160 + pad)), dt)
        view = big[:, :160]
        codes = torch.full((9, 80), 7, dtype=torch.uint8, device=dev())
        scales = torch.full((9, 5), 7, dtype=torch.uint8, device=dev())
        ctx.mx_quantize(view, codes_out=codes, scales_out=scales)
        cw, sw = oracle.mx_quantize(view.double().cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), cw) and np.array_equal(scales.cpu().numpy(), sw)
    three = _as(rng.normal(size=(2, 3, 64)), torch.float32)
    codes, scales = ctx.mx_quantize(three)
    assert codes.shape == (2, 3, 32) and scales.shape == (2, 3, 2)
    empty, es = ctx.mx_quantize(torch.empty(0, 64, device=dev()))
    assert empty.shape == (0, 32) and ctx.mx_dequantize(empty, es).shape == (0, 64)


def test_dequantize_every_code_and_scale(ctx):
    codes = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1))
    codes[:, 1::2] ^= 0x5A
    scales = np.arange(256, dtype=np.uint8)[:, None]
    want = oracle.mx_values(codes, scales)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)                     # past the type's range: infinity
    for dt in (torch.float32, torch.bfloat16):
        got = ctx.mx_dequantize(to_dev(codes), to_dev(scales), dtype=dt).float().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


# ------------------------------------------------------------------ product

def _random_mx(rng, rows, k, spread=6):
    codes = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    scales = (127 + rng.integers(-spread, spread + 1, (rows, k // 32))).astype(np.uint8)
    return codes, scales


def _check_matmul(ctx, rng, m, n, k, dtypes=(torch.float32, torch.bfloat16)):
    a, sa = _random_mx(rng, m, k)
    w, sw = _random_mx(rng, n, k)
    av, wv = oracle.mx_values(a, sa), oracle.mx_values(w, sw)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    for dt in dtypes:
        got = ctx.mx_matmul(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), dtype=dt).double().cpu().numpy()
        tol = k * 2.0 ** -23 * mag
        tol = tol + (np.abs(want) + tol) * (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24)
        assert got.shape == (m, n)
        assert np.all(np.abs(got - want) <= tol), (m, n, k, dt, np.max(np.abs(got - want) - tol))


SIZES = [(1, 1, 32), (1, 2816, 2048), (2, 17, 64), (5, 33, 96), (15, 100, 128), (16, 256, 2048), (17, 16, 160),
         (31, 130, 224), (32, 64, 288), (33, 500, 256), (48, 31, 1440), (63, 129, 320), (64, 1408, 512),
         (65, 257, 352), (77, 401, 1440), (100, 1000, 416), (127, 255, 1056), (128, 512, 1024), (129, 128, 480),
         (192, 320, 1408), (255, 257, 544), (256, 256, 8192), (300, 700, 608), (511, 1409, 256), (513, 640, 2048),
         (1000, 513, 1440), (1025, 1024, 640), (2049, 300, 128), (4100, 2816, 96)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul_matches_oracle(ctx, m, n, k):
    _check_matmul(ctx, np.random.default_rng(m * 7 + n * 3 + k), m, n, k)


@pytest.mark.parametrize("m,n,k", [(1, 300, 2048), (40, 64, 1440), (130, 130, 1056), (600, 520, 1440), (1500, 1100, 96)])
def test_matmul_is_exact_on_quarters(ctx, m, n, k):
    rng = np.random.default_rng(k)
    a, w = (rng.integers(0, 256, (r, k // 2)).astype(np.uint8) for r in (m, n))
    one = lambda r: np.full((r, k // 32), 127, np.uint8)                     # noqa: E731
    want = oracle.mx_values(a, one(m)) @ oracle.mx_values(w, one(n)).T
    got = ctx.mx_matmul(to_dev(a), to_dev(one(m)), to_dev(w), to_dev(one(n)), dtype=torch.float32)
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("m,n,k", [(1, 40, 128), (70, 50, 160), (300, 600, 1440), (700, 1300, 256)])
def test_matmul_nan_blocks_and_zero_scales(ctx, m, n, k):
    """A NaN block spoils its own row or column and no other; neighbours of the last rows stay as they are."""
    rng = np.random.default_rng(m)
    a, sa = _random_mx(rng, m, k)
    w, sw = _random_mx(rng, n, k)
    ra, rw = m - 1, n // 2
    sa[ra, -1] = 255
    sw[rw, 0] = 255
    sw[n - 1, 0] = 0
    av, wv = oracle.mx_values(a, sa), oracle.mx_values(w, sw)
    out = torch.full((m + 1, n), 77.0, device=dev())
    ctx.mx_matmul(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), dtype=torch.float32, out=out[:m])
    got = out.double().cpu().numpy()
    assert np.all(got[m] == 77.0)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert np.array_equal(np.isnan(got[:m]), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(got[:m] - want)[ok] <= (k * 2.0 ** -23 * mag + 2.0 ** -24 * np.abs(want))[ok])


def test_quantize_then_multiply(ctx):
    """A linear layer as it is used: both operands quantized, then multiplied."""
    rng = np.random.default_rng(8)
    x, w = rng.normal(size=(37, 512)), rng.normal(0, 0.02, (200, 512))
    xt, wt = _as(x, torch.bfloat16), _as(w, torch.float32)
    y = ctx.mx_matmul(*ctx.mx_quantize(xt), *ctx.mx_quantize(wt), dtype=torch.float32).double().cpu().numpy()
    xv = oracle.mx_values(*oracle.mx_quantize(xt.double().cpu().numpy()))
    wv = oracle.mx_values(*oracle.mx_quantize(wt.double().cpu().numpy()))
    assert np.all(np.abs(y - xv @ wv.T) <= 512 * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + 1e-30)


def test_same_bits_on_every_run_and_stream(ctx):
    rng = np.random.default_rng(11)
    a, sa = _random_mx(rng, 333, 2048)
    w, sw = _random_mx(rng, 777, 2048)
    args = [to_dev(v) for v in (a, sa, w, sw)]
    want = ctx.mx_matmul(*args, dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ctx.mx_matmul(*args, dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(ctx.mx_matmul(*args, dtype=torch.float32), want)


def test_refusals(ctx):
    import gptq_calibration_moe_amd as clha
    lib, h = clha.lib, ctx._h
    t = torch.zeros(4096, dtype=torch.uint8, device=dev())
    p = t.data_ptr()

    def quant(rows=2, cols=64, x=p, dt=clha.F32, ld=64, codes=p, scales=p):
        return lib.clha_mx_quantize(h, rows, cols, x, dt, ld, codes, scales, None)
    assert quant(cols=48) == quant(cols=0) == quant(cols=-32) == quant(rows=-1) == clha.ERR_SHAPE
    assert quant(ld=63) == quant(ld=32) == quant(ld=66) == quant(dt=clha.BF16, ld=68) == clha.ERR_SHAPE
    assert quant(rows=1 << 40) == clha.ERR_SHAPE
    assert quant(dt=2) == quant(x=None) == quant(codes=None) == quant(scales=None) == clha.ERR_INVALID_ARG
    assert quant(x=p + 4) == quant(codes=p + 8) == quant(scales=p + 2) == clha.ERR_ALIGN
    assert quant(rows=0, x=None) == clha.OK

    def deq(rows=2, cols=64, codes=p, scales=p, out=p, dt=clha.F32):
        return lib.clha_mx_dequantize(h, rows, cols, codes, scales, out, dt, None)
    assert deq(cols=16) == deq(rows=-1) == clha.ERR_SHAPE
    assert deq(dt=7) == deq(codes=None) == deq(out=None) == clha.ERR_INVALID_ARG
    assert deq(out=p + 4) == deq(codes=p + 4) == clha.ERR_ALIGN

    def mm(m=2, n=2, k=32, a=p, sa=p, w=p, sw=p, out=p, dt=clha.F32):
        return lib.clha_mx_matmul(h, m, n, k, a, sa, w, sw, out, dt, None)
    assert mm(k=0) == mm(k=33) == mm(k=65568) == mm(n=0) == mm(n=524289) == mm(m=-1) == mm(m=1 << 31) == clha.ERR_SHAPE
    assert mm(a=None) == mm(sa=None) == mm(w=None) == mm(sw=None) == mm(out=None) == mm(dt=3) == clha.ERR_INVALID_ARG
    assert mm(a=p + 8) == mm(w=p + 8) == mm(out=p + 4) == mm(sa=p + 1) == mm(sw=p + 2) == clha.ERR_ALIGN
    assert mm(m=0, a=None) == clha.OK
    x = torch.zeros(4, 64, device=dev())
    for bad in (x.double(), x.cpu(), x.t()):
        with pytest.raises((TypeError, ValueError)):
            ctx.mx_quantize(bad)
    codes, scales = ctx.mx_quantize(x)
    with pytest.raises(ValueError):
        ctx.mx_dequantize(codes, scales[:, :1].contiguous())
    with pytest.raises(TypeError):
        ctx.mx_dequantize(codes, scales, dtype=torch.float16)
    with pytest.raises(ValueError):
        ctx.mx_matmul(codes, scales, *ctx.mx_quantize(torch.zeros(4, 96, device=dev())))
    with pytest.raises(clha.ClhaError):
        ctx.mx_quantize(x[:1].expand(4, 64))


def test_products_beyond_one_launch_are_refused(ctx):
    """A launch counts its threads in 32 bits: 256 for a tile of 128 x 128 results, so
    m rows of one column need m / 128 * 256 of them."""
    import gptq_calibration_moe_amd as clha
    t = torch.zeros(64, dtype=torch.uint8, device=dev())
    p = t.data_ptr()
    for m, n in (((1 << 30) + 1, 1), (1 << 31, 1), ((1 << 26) + 1, 1024), ((1 << 17) + 1, 524288)):
        st = clha.lib.clha_mx_matmul(ctx._h, m, n, 32, p, p, p, p, p, clha.F32, None)
        assert st == clha.ERR_SHAPE, (m, n)
    for tile, threads in ((128, 256), (256, 512)):   # the largest calls that are taken
        for m in (129, 1 << 17, 1 << 20, 1 << 26, 1 << 30):
            n = min((1 << 36) // m, 524288)
            tiles = -(-m // tile) * -(-n // tile)
            assert (tiles + 7) // 8 * 8 * threads < 1 << 32


@pytest.mark.parametrize("m,n,k", [(20, 8300, 96), (40, 8300, 512), (65, 4097, 160), (100, 8193, 512), (128, 4096, 544)])
def test_few_rows_against_many_columns(ctx, m, n, k):
    _check_matmul(ctx, np.random.default_rng(m + n + k), m, n, k)
