"""GPU tests of the microscaled operators against plain forms in 64 bits.

Quantised codes and scales, and values read back, are compared bit for bit:
the format determines them.  Tolerances elsewhere are counted in half steps
(2^-8 for bf16, 2^-11 for fp16, 2^-24 for fp32) as each test derives."""
import concurrent.futures
import copy
import gc
import io
import sys
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import expert_ffn_execution_b200 as sm  # noqa: E402
import oracle  # noqa: E402
from expert_ffn_execution_b200 import mx  # noqa: E402
from tests import mx_reference as ref  # noqa: E402
from tests.harness import OUT_REL_L2, check_routing, rel_l2_rows  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FMTS = [sm.MX_FP4, sm.MX_FP8]
LAYOUTS = [sm.MX_ROWS, sm.MX_TILES]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def n64(t):
    return t.double().cpu().numpy()


def hard_rows(rows, K, dtype, seed):
    """Normal values over many magnitudes, with blocks of zeros, of signed
    zeros, of subnormals, of the type's largest, exact ties, powers of two and
    their neighbours, Inf and NaN."""
    g = gen(seed)
    x = torch.randn(rows, K, device=DEV, generator=g)
    x *= torch.exp2(torch.randint(-12, 13, (rows, K // 32, 1), device=DEV, generator=g).float()).expand(
        -1, -1, 32).reshape(rows, K)
    x = x.to(dtype)
    b = x.view(-1, 32)
    info = torch.finfo(dtype)
    special = [torch.zeros(32), -torch.zeros(32), torch.full((32,), info.tiny), torch.full((32,), info.smallest_normal / 4),
               torch.full((32,), info.max), torch.arange(32) * 0.25, torch.arange(32) * -0.125, torch.arange(32) * 14.0,
               torch.tensor([2.0 ** (i - 16) for i in range(32)]), torch.full((32,), 4.0).index_fill(0, torch.tensor([5]), float("inf")),
               torch.ones(32).index_fill(0, torch.tensor([31]), float("nan")),
               torch.full((32,), 8.0).index_fill(0, torch.tensor([0]), 8.0 - 8 * info.eps)]
    for i, v in enumerate(special):
        if (3 * i + 1) < b.shape[0]:
            b[3 * i + 1] = v.to(device=DEV, dtype=dtype)
    return x


def host_codes(q):
    c = q.codes.cpu().numpy()
    return ref.unpack(c.reshape(q.rows, -1), q.fmt)


def assert_quantised(q, x):
    codes, scales = ref.quantize(n64(x), q.fmt)
    s = q.scales.cpu().numpy()
    if q.layout == sm.MX_TILES:
        assert np.array_equal(s, ref.tile_scales(scales))
    else:
        assert np.array_equal(s, scales)
    assert np.array_equal(host_codes(q), codes)


@pytest.fixture(autouse=True, scope="module")
def armed():
    """The native calls are those that run."""
    sm.mx_quantize(torch.zeros(1, 32, device=DEV), sm.MX_FP8)
    assert mx._fast is not None


# ---------------------------------------------------------------- quantiser
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (128, 128), (130, 160), (67, 2592)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_quantize(dtype, fmt, layout, rows, K):
    x = hard_rows(rows, K, dtype, 1 + rows)
    assert_quantised(sm.mx_quantize(x, fmt, layout), x)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_strided_rows(fmt):
    wide = hard_rows(37, 256, torch.bfloat16, 2)
    x = wide[:, 64:160]
    assert_quantised(sm.mx_quantize(x, fmt), x)
    x = wide[::3, 96:256]
    assert_quantised(sm.mx_quantize(x, fmt, sm.MX_ROWS), x)
    row = wide[5:6].expand(9, 256)  # one row nine times: stride 0
    assert_quantised(sm.mx_quantize(row, fmt), row)


def test_quantize_leaves_the_rest():
    """Rows behind the last, and bytes between batches, stay as they were."""
    E, rows, K = 3, 5, 64
    x = hard_rows(E * rows, K, torch.float32, 3).view(E, rows, K)
    cs, ss = rows * 32 + 48, rows * 2 + 7
    codes = torch.full((E * cs + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((E * ss + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    sm.moe_mx_quantize(x, sm.DTYPE_F32, E, rows, K, K, rows * K, sm.MX_FP4, codes, cs, scales, sm.MX_ROWS, ss)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    for e in range(E):
        rc, rs = ref.quantize(n64(x[e]), sm.MX_FP4)
        assert np.array_equal(c[e * cs:][:rows * 32].reshape(rows, 32), ref.pack(rc, sm.MX_FP4))
        assert np.array_equal(s[e * ss:][:rows * 2].reshape(rows, 2), rs)
        assert (c[e * cs + rows * 32:(e + 1) * cs] == 0xA5).all()
        assert (s[e * ss + rows * 2:(e + 1) * ss] == 0xA5).all()


def test_quantize_nothing():
    for layout in LAYOUTS:
        q = sm.mx_quantize(torch.empty(0, 64, device=DEV), sm.MX_FP4, layout)
        assert q.codes.shape == (0, 32) and q.scales.numel() == 0
        assert q.dequantize().shape == (0, 64)


# ---------------------------------------------------------------- read-back
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_code(fmt, layout, dtype):
    """Every code under scales from the smallest to the largest and NaN."""
    n = 16 if fmt == sm.MX_FP4 else 256
    exps = np.array([0, 1, 20, 100, 118, 127, 130, 141, 240, 254, 255], np.uint8)
    codes = np.tile(np.arange(n, dtype=np.uint8), (len(exps), 256 // n))
    scales = np.repeat(exps[:, None], 8, 1)
    want = ref.dequantize(codes, scales, fmt)
    stored = torch.from_numpy(ref.pack(codes, fmt)).to(DEV)
    s = torch.from_numpy(scales).to(DEV)
    q = sm.MXTensor(stored, s, fmt, len(exps), 256, sm.MX_ROWS)
    if layout == sm.MX_TILES:
        q = sm.mx_tile_scales(q)
        assert np.array_equal(q.scales.cpu().numpy(), ref.tile_scales(scales))
    got = q.dequantize(dtype).cpu()
    # exact in fp32, then one rounding: torch's own from the exact fp64 value through fp32
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want.astype(np.float32)).to(dtype)
    assert np.array_equal(got.float().numpy(), want.float().numpy(), equal_nan=True)


@pytest.mark.parametrize("rows,K", [(1, 32), (129, 160), (300, 1056)])
def test_tile_scales(rows, K):
    s = torch.randint(0, 256, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=gen(4))
    q = sm.MXTensor(torch.zeros(rows, K, dtype=torch.uint8, device=DEV), s, sm.MX_FP8, rows, K, sm.MX_ROWS)
    assert np.array_equal(sm.mx_tile_scales(q).scales.cpu().numpy(), ref.tile_scales(s.cpu().numpy()))


# ---------------------------------------------------------------- norm
def norm64(x, delta, gain, eps):
    r = n64(x) + (0 if delta is None else n64(delta))
    h = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r, h * (1 if gain is None else n64(gain))


# fp32 steps of h: the addition (half a step), the sum of H squares (each thread adds up to 32
# squares in turn, then 5 + 16 partial sums: under 64 half steps, halved by the root), the mean, eps,
# root, division and two products (half a step each, together under 8).
H_REL = (1 + 32 + 8) * 2.0 ** -24


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2560), (3, 40), (5, 2592), (130, 4096), (2, 16384)])
@pytest.mark.parametrize("xt,dt,ot", [(torch.float32, torch.bfloat16, torch.bfloat16),
                                      (torch.bfloat16, torch.bfloat16, torch.float16),
                                      (torch.float16, torch.float32, torch.float32),
                                      (torch.float32, None, torch.bfloat16)])
def test_norm(xt, dt, ot, T, H):
    g = gen(T + H)
    x = torch.randn(T, H, device=DEV, generator=g).to(xt)
    delta = None if dt is None else torch.randn(T, H, device=DEV, generator=g).to(dt)
    gain = 1 + 0.1 * torch.randn(H, device=DEV, generator=g) if T != 3 else None
    n = sm.add_rmsnorm(x, delta, gain, 1e-5, out_dtype=ot)
    r, h = norm64(x, delta, gain, 1e-5)
    if delta is None:
        assert n.residual is x
    else:
        # one fp32 addition, one rounding to the dtype of x
        want = (x.float() + delta.float()).to(xt)
        assert torch.equal(n.residual, want)
    # r's rounding is relative to r, so where x and delta cancel h's error is relative to |x| + |delta|
    size = np.abs(h)
    if delta is not None:
        k = np.abs(h) / np.maximum(np.abs(r), 1e-300)
        size = np.maximum(size, k * (np.abs(n64(x)) + np.abs(n64(delta))))
    assert n.out.dtype == ot
    tol = HALF_STEP[ot] * np.abs(h) + H_REL * (1 + HALF_STEP[ot]) * size + 2.0 ** -25  # fp16 subnormals
    assert (np.abs(n64(n.out) - h) <= tol).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H", [(1, 32), (4, 2560), (131, 2592), (3, 16384)])
def test_norm_quantised(T, H, fmt, layout):
    """The codes are those of h to within h's own rounding: the scale is that
    of a largest magnitude within H_REL of h's, every value within half a step
    of h on that scale, or saturated."""
    g = gen(T * H)
    x = torch.randn(T, H, device=DEV, generator=g)
    delta = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    x[:, : min(H, 4)] *= 30
    gain = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
    n = sm.add_rmsnorm(x, delta, gain, 1e-6, out_dtype=torch.float32, fmt=fmt, layout=layout)
    # the codes are the format's of the fp32 rows that `out` holds, bit for bit
    assert_quantised(n.mx, n.out)
    r, h = norm64(x, delta, gain, 1e-6)
    size = np.abs(h) / np.maximum(np.abs(r), 1e-300) * (np.abs(n64(x)) + np.abs(n64(delta)))
    assert (np.abs(n64(n.out) - h) <= (H_REL + 2.0 ** -24) * size).all()
    only = sm.add_rmsnorm(x, delta, gain, 1e-6, fmt=fmt, layout=layout)
    assert only.out is None and torch.equal(only.mx.codes, n.mx.codes) and torch.equal(only.mx.scales, n.mx.scales)


@pytest.mark.parametrize("T,H", [(4099, 128), (5003, 256), (1203, 1056), (9481, 1024), (9481, 1536), (150, 16384)])
@pytest.mark.parametrize("xt,dt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                   (torch.float32, None), (torch.bfloat16, None)])
def test_norm_of_many_rows(xt, dt, T, H):
    """Rows that share a CTA, and several groups a thread."""
    g = gen(T + H)
    x = torch.randn(T, H, device=DEV, generator=g).to(xt)
    delta = None if dt is None else torch.randn(T, H, device=DEV, generator=g).to(dt)
    gain = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
    n = sm.add_rmsnorm(x, delta, gain, 1e-6, out_dtype=torch.float32, fmt=sm.MX_FP8)
    q = sm.mx_quantize(n.out, sm.MX_FP8)
    assert torch.equal(n.mx.codes, q.codes) and torch.equal(n.mx.scales, q.scales)
    r = size = x.double()
    if delta is not None:
        assert torch.equal(n.residual, (x.float() + delta.float()).to(xt))
        r, size = r + delta.double(), r.abs() + delta.double().abs()
    k = gain.double() / (r.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    assert ((n.out.double() - r * k).abs() <= (H_REL + 2.0 ** -24) * (size * k).abs()).all()


def test_norm_in_place_and_zero_rows():
    x = torch.randn(6, 256, device=DEV, generator=gen(5))
    x[2] = 0
    d = torch.randn(6, 256, device=DEV, generator=gen(6))
    d[2] = 0
    want = sm.add_rmsnorm(x, d, out_dtype=torch.bfloat16, fmt=sm.MX_FP8)
    y = x.clone()
    got = sm.add_rmsnorm(y, d, out_dtype=torch.bfloat16, fmt=sm.MX_FP8, residual_out=y)
    assert got.residual is y and torch.equal(y, want.residual) and torch.equal(got.out, want.out)
    assert (want.out[2] == 0).all() and (want.mx.dequantize()[2] == 0).all()
    x[4, 7] = float("nan")
    n = sm.add_rmsnorm(x, d, out_dtype=torch.float32, fmt=sm.MX_FP4)
    assert n.out[4].isnan().all() and n.mx.dequantize()[4].isnan().all()
    assert torch.equal(n.mx.codes[:4], sm.mx_quantize(n.out, sm.MX_FP4).codes[:4])
    assert not n.out[[0, 1, 3, 5]].isnan().any()


def test_norm_matches_the_layers_norm():
    """Without delta and gain: within a step of moe_rmsnorm (bf16)."""
    x = torch.randn(9, 2560, device=DEV, generator=gen(7))
    a = torch.empty(9, 2560, dtype=torch.bfloat16, device=DEV)
    sm.moe_rmsnorm(x, 9, 2560, 1e-6, a)
    b = sm.add_rmsnorm(x, out_dtype=torch.bfloat16).out
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs()).all()


# ---------------------------------------------------------------- product
PAIRS = [(sm.MX_FP8, sm.MX_FP4), (sm.MX_FP4, sm.MX_FP4), (sm.MX_FP8, sm.MX_FP8)]


def random_mx(rows, K, fmt, seed, lo=120, hi=130):
    g = gen(seed)
    if fmt == sm.MX_FP4:
        codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    else:
        codes = torch.randint(0, 127, (rows, K), dtype=torch.uint8, device=DEV, generator=g)
        codes |= torch.randint(0, 2, (rows, K), dtype=torch.uint8, device=DEV, generator=g) << 7
    s = torch.randint(lo, hi, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    q = sm.MXTensor(codes, s, fmt, rows, K, sm.MX_ROWS)
    v = torch.from_numpy(ref.dequantize(host_codes(q), s.cpu().numpy(), fmt)).to(DEV)
    return sm.mx_tile_scales(q), v


def assert_product(y, xv, wv, bias=None):
    """|error| <= one rounding of the result + the fp32 sum's: products of codes are exact, an
    instruction adds 32 or 64 of them and the sum so far, each kept to 24 bits of the largest: at most
    K/32 + 64 truncations (a whole fp32 step each, 2^-23) of at most sum |x w|, and 8 joined parts and
    a bias."""
    want = xv @ wv.T
    mag = xv.abs() @ wv.abs().T
    if bias is not None:
        want = want + bias.double()
        mag = mag + bias.double().abs()
    steps = xv.shape[1] / 32 + 64 + 9
    tol = HALF_STEP[y.dtype] * want.abs() + steps * 2.0 ** -23 * mag + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    bad = ~((y.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float((y.double() - want).norm() / want.norm()))


SHAPES = [(1, 128, 128), (1, 1, 128), (3, 100, 256), (16, 129, 384), (17, 300, 640), (33, 128, 1024), (64, 127, 128),
          (65, 257, 512), (128, 128, 128), (129, 385, 896), (300, 641, 2688), (513, 1000, 256), (4, 4100, 2560),
          (2, 40000, 128), (8, 64, 16384)]


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear(T, N, K, xf, wf):
    x, xv = random_mx(T, K, xf, T + N)
    w, wv = random_mx(N, K, wf, T + N + 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = sm.mx_linear(x, w, out_dtype=torch.float32, dev_status=status)
    assert sm.strata_read_status(status) == 0
    assert_product(y, xv, wv)


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("T", [2, 200])
def test_linear_is_exact_on_small_integers(T, xf, wf):
    """Whole numbers whose sums stay below 2^24: no rounding anywhere."""
    N, K = 200, 640
    g = gen(T)
    xi = torch.randint(-3, 4, (T, K), device=DEV, generator=g).float()
    wi = torch.randint(-3, 4, (N, K), device=DEV, generator=g).float()
    xi.view(T, -1, 32)[..., 0] = 4  # every block's largest is 4: scales of 1 (FP4)
    wi.view(N, -1, 32)[..., 0] = 4
    y = sm.mx_linear(sm.mx_quantize(xi, xf), sm.mx_quantize(wi, wf), out_dtype=torch.float32)
    assert torch.equal(y.double(), xi.double() @ wi.double().T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,N", [(5, 300), (150, 259), (1100, 2050), (1100, 2047), (1030, 2176)])
def test_linear_bias_dtypes_and_row_stride(T, N, dtype):
    K = 512
    x, xv = random_mx(T, K, sm.MX_FP8, 1, 118, 122)
    w, wv = random_mx(N, K, sm.MX_FP4, 2, 118, 122)
    bias = torch.randn(N, device=DEV, generator=gen(3))
    for extra, at in ((13, 3), (14, 2), (32, 8)):  # rows on odd, 4-byte and 16-byte boundaries
        wide = torch.full((T + 2, (N + extra + 15) // 16 * 16 + extra % 16), 7.0, dtype=dtype, device=DEV)
        out = wide[1:-1, at:N + at]
        got = sm.mx_linear(x, w, bias, out=out)
        assert got is out
        assert_product(out, xv, wv, bias)
        wide[1:-1, at:N + at] = 7.0
        assert (wide == 7.0).all()  # nothing else was written


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("T", [4, 140])
def test_linear_nan_blocks_stay_in_their_rows(T, xf, wf):
    N, K = 140, 384
    x, xv = random_mx(T, K, xf, 5)
    w, wv = random_mx(N, K, wf, 6)
    xs = x.scales.clone()
    xs[(1 % 32) * 16 + 2] = 255       # row 1, block 2
    ws = w.scales.clone()
    ws[2 * 512 + (7 % 32) * 16 + 3] = 255  # row 7, block 11, the last
    y = sm.mx_linear(sm.MXTensor(x.codes, xs, xf, T, K, sm.MX_TILES),
                     sm.MXTensor(w.codes, ws, wf, N, K, sm.MX_TILES), out_dtype=torch.float32)
    assert y[1].isnan().all() and y[:, 7].isnan().all()
    keep_t = [t for t in range(T) if t != 1]
    keep_n = [n for n in range(N) if n != 7]
    assert_product(y[keep_t][:, keep_n].contiguous(), xv[keep_t], wv[keep_n])


def test_linear_extreme_scales():
    """Scale bytes far apart whose products are in fp32's range."""
    T, N, K = 7, 130, 256
    x, xv = random_mx(T, K, sm.MX_FP8, 8, 10, 12)
    w, wv = random_mx(N, K, sm.MX_FP8, 9, 240, 242)
    assert_product(sm.mx_linear(x, w, out_dtype=torch.float32), xv, wv)


def test_linear_same_bits_every_time_and_in_any_batch_of_a_tile():
    x, _ = random_mx(200, 1024, sm.MX_FP8, 10)
    w, _ = random_mx(700, 1024, sm.MX_FP4, 11)
    a = sm.mx_linear(x, w, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(a, sm.mx_linear(x, w, out_dtype=torch.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,N", [(3900, 4000), (4096, 4096), (3841, 4003), (4100, 3850)])
@pytest.mark.parametrize("xf,wf,K", [(sm.MX_FP8, sm.MX_FP4, 1024), (sm.MX_FP4, sm.MX_FP4, 2176),
                                     (sm.MX_FP8, sm.MX_FP8, 1152)])
def test_linear_many_rounds_of_tiles(xf, wf, K, T, N, dtype):
    """Small integers, exact in any order; rows of y further apart than they
    are long, on 16-byte boundaries or not, and nothing behind them written."""
    g = gen(71)
    x = torch.randint(-3, 4, (T, K), device=DEV, generator=g).float()
    w = torch.randint(-3, 4, (N, K), device=DEV, generator=g).float()
    bias = torch.randint(-9, 10, (N,), device=DEV, generator=g).float()
    want = (x @ w.T + bias).to(dtype)
    q, wq = sm.mx_quantize(x, xf), sm.mx_quantize(w, wf)
    for pitch in (N, N + 16 - N % 8, N + 1):
        out = torch.full((T, pitch), 7, dtype=dtype, device=DEV)
        sm.mx_linear(q, wq, bias, out=out[:, :N])
        assert torch.equal(out[:, :N], want) and (out[:, N:] == 7).all()
    assert torch.equal(sm.mx_linear(q, wq, out_dtype=dtype), (x @ w.T).to(dtype))


@pytest.mark.parametrize("T", [1 << 22, (1 << 20) + 1])
def test_linear_most_tokens(T):
    """Small integers, exact in any order; N too small for many tiles."""
    g = gen(70)
    x = torch.randint(-3, 4, (1024, 128), device=DEV, generator=g).float()
    w = torch.randint(-3, 4, (3, 128), device=DEV, generator=g).float()
    q = sm.mx_quantize(x, sm.MX_FP8, sm.MX_ROWS)
    n = -(-T // 1024)
    many = sm.mx_tile_scales(sm.MXTensor(q.codes.repeat(n, 1)[:T], q.scales.repeat(n, 1)[:T], sm.MX_FP8, T, 128,
                                         sm.MX_ROWS))
    y = sm.mx_linear(many, sm.mx_quantize(w, sm.MX_FP4), out_dtype=torch.float32)
    assert torch.equal(y, (x @ w.T).repeat(n, 1)[:T])


def test_linear_nothing():
    w, _ = random_mx(64, 128, sm.MX_FP4, 12)
    x = sm.mx_quantize(torch.empty(0, 128, device=DEV), sm.MX_FP8)
    assert sm.mx_linear(x, w).shape == (0, 64)


@pytest.mark.parametrize("xf,wf", PAIRS)
def test_linear_tiles_that_start_inside_a_scale_tile(xf, wf):
    """Two tiles of 64 tokens in one tile of scales, every row's scales its own."""
    for T, N, K in ((128, 256, 2048), (100, 512, 1024), (192, 384, 1024)):
        x, xv = random_mx(T, K, xf, T, 110, 140)
        w, wv = random_mx(N, K, wf, T + 1)
        assert_product(sm.mx_linear(x, w, out_dtype=torch.float32), xv, wv)


def test_linear_on_two_streams_at_once():
    """Calls of every form (split and not, single CTAs and pairs) side by side
    on two streams give the bits of the calls in turn."""
    cases = [(4, 2560, 2560), (600, 4000, 512), (64, 1024, 4096), (128, 4096, 1024), (1, 12000, 768)]
    made = []
    for i, (T, N, K) in enumerate(cases):
        x, w = (sm.mx_quantize(torch.randn(r, K, device=DEV, generator=gen(70 + 2 * i + j)), f)
                for j, (r, f) in enumerate(((T, sm.MX_FP8), (N, sm.MX_FP4))))
        made.append((x, w, sm.mx_linear(x, w, out_dtype=torch.float32)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, (x, w, want) in enumerate(made):
            for s in streams:
                with torch.cuda.stream(s):
                    got.append((sm.mx_linear(x, w, out_dtype=torch.float32, dev_status=status), want))
        made.append(made.pop(0))  # another neighbour each time
    torch.cuda.synchronize()
    assert sm.strata_read_status(status) == 0
    for y, want in got:
        assert torch.equal(y, want)


# ---------------------------------------------------------------- past 32 bits
def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of a call with them alone."""
    rows, K, tail = (1 << 19) + 5 + 128 * 37, 4096, 133
    first = rows - rows % 128 - 128  # where a tile of scales starts
    x = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
    x[:1 << 17].normal_(generator=gen(90))
    for at in range(1 << 17, rows, 1 << 17):
        n = min(1 << 17, rows - at)
        x[at:at + n] = x[:n]
    x[first:].normal_(generator=gen(91))
    for fmt in FMTS:
        q = sm.mx_quantize(x, fmt)
        alone = sm.mx_quantize(x[first:], fmt)
        assert torch.equal(q.codes[first:], alone.codes)
        assert torch.equal(q.scales[first * K // 32:], alone.scales)
        v = q.dequantize(torch.bfloat16)
        assert torch.equal(v[-tail:], alone.dequantize(torch.bfloat16)[-tail:])
        assert torch.equal(v[:300], sm.mx_quantize(x[:300], fmt).dequantize(torch.bfloat16))
        del v, q
    n = sm.add_rmsnorm(x, fmt=sm.MX_FP8, residual_out=x)
    alone = sm.add_rmsnorm(x[first:].clone(), fmt=sm.MX_FP8)
    assert torch.equal(n.mx.codes[first:], alone.mx.codes)
    assert torch.equal(n.mx.scales[first * K // 32:], alone.mx.scales)
    del x, n, alone
    torch.cuda.empty_cache()
    T, N, K = (1 << 17) + 77, 17000, 128
    a, w = sm.mx_quantize(torch.randn(T, K, device=DEV), sm.MX_FP8), sm.mx_quantize(torch.randn(N, K, device=DEV), sm.MX_FP4)
    last = T - T % 128 - 256
    z = sm.MXTensor(a.codes[last:], a.scales[last * K // 32:].clone(), sm.MX_FP8, T - last, K, sm.MX_TILES)
    for dtype in (torch.bfloat16, torch.float32):
        y = sm.mx_linear(a, w, out_dtype=dtype)
        assert y.numel() > 1 << 31
        assert torch.equal(y[last:], sm.mx_linear(z, w, out_dtype=dtype))
        del y
        torch.cuda.empty_cache()


# ---------------------------------------------------------------- together
def step(x, d, gain, w, out):
    n = sm.add_rmsnorm(x, d, gain, fmt=sm.MX_FP8, residual_out=x)
    return sm.mx_linear(n.mx, w, out=out)


def test_two_graphs_and_a_side_stream():
    """Steps captured in two graphs, replayed in turn, and run on another
    stream, give the bits of the eager calls."""
    T, H, N = 4, 2560, 1000
    w, _ = random_mx(N, H, sm.MX_FP4, 13, 116, 120)
    gain = torch.ones(H, device=DEV)
    ins = [(torch.randn(T, H, device=DEV, generator=gen(20 + i)),
            torch.randn(T, H, device=DEV, generator=gen(30 + i)).bfloat16()) for i in range(2)]
    want = []
    for x, d in ins:
        r, o = x.clone(), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        step(r, d, gain, w, o)
        want.append((r, o))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r, o = ins[0][0].clone(), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        step(r, ins[0][1], gain, w, o)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r, want[0][0]) and torch.equal(o, want[0][1])
    held = []
    for x, d in ins:
        r, o = x.clone(), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(r, d, gain, w, o)
        held.append((g, r, o, x))
    for _ in range(3):
        for g, r, o, x in held:
            r.copy_(x)
            o.zero_()
        for g, *_ in held:
            g.replay()
        for (g, r, o, x), (wr, wo) in zip(held, want):
            assert torch.equal(r, wr) and torch.equal(o, wo)


@pytest.mark.parametrize("rows", [1, 4096])
def test_a_residual_behind_an_early_release(rows):
    """moe_combine reads its residual before it waits, and the quantiser lets
    it start early: what the norm before both wrote is there."""
    T, H = 64, 2560
    big = torch.randn(rows, 1024, device=DEV, generator=gen(60))
    codes = sm.mx_quantize(big, sm.MX_FP8).codes.clone()
    y = torch.zeros(T, H, device=DEV)
    inv = torch.arange(T, dtype=torch.int32, device=DEV)
    w = torch.ones(T, 1, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, acc = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, device=DEV)
    r = torch.zeros(T, H, device=DEV)
    for i in range(20):
        x = torch.randn(T, H, device=DEV, generator=gen(61 + i))
        torch.cuda.synchronize()
        sm.add_rmsnorm(x, x, fmt=sm.MX_FP8, residual_out=r)
        q = sm.mx_quantize(big, sm.MX_FP8)
        sm.moe_combine(y, sm.DTYPE_F32, inv, w, None, sm.DTYPE_F32, r, T, 1, H, out, acc, status)
        assert torch.equal(acc, x + x) and torch.equal(q.codes, codes)
    assert sm.strata_read_status(status) == 0


@pytest.mark.parametrize("T", [4, 48])
def test_packed_experts_in_the_layer(T):
    """bf16 weights -> blobs -> the MoE layer -> the norm after it -> a
    projection: the blobs are the format's bit for bit, the layer agrees with
    the oracle on them, and the projection with 64 bits on its own input."""
    H, I, E, k, N = 512, 256, 16, 4, 300
    g = gen(40)
    gate, up = (0.05 * torch.randn(E, I, H, device=DEV, generator=g).bfloat16() for _ in range(2))
    down = 0.05 * torch.randn(E, H, I, device=DEV, generator=g).bfloat16()
    ex = sm.pack_experts(gate, up, down)
    for t, v in zip((gate, up, down), ex.dequantize()):
        c, s = ref.quantize(n64(t).reshape(-1, t.shape[2]), sm.MX_FP4)
        assert np.array_equal(n64(v).reshape(c.shape), ref.dequantize(c, s, sm.MX_FP4))
    x = torch.randn(T, H, device=DEV, generator=g)
    wr = (0.02 * torch.randn(H, E, device=DEV, generator=g)).bfloat16()
    layer = sm.MoELayer(wr, None, ex, k)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = layer.forward(x, topk_ids=ids, dev_status=status)
    assert sm.strata_read_status(status) == 0
    hid = oracle.rmsnorm(x.cpu().numpy())
    wr16 = wr.cpu().view(torch.int16).numpy().view(np.uint16)
    lg = oracle.router_logits(hid, wr16, None)
    assert check_routing(lg, ids.cpu().numpy(), k)[0]
    r = oracle.moe_layer(hid, wr16, None, E, k, sm.FMT_MXFP4_32, I, ex.blobs.cpu().numpy(),
                         forced_ids=ids.cpu().numpy())
    assert rel_l2_rows(out.float().cpu().numpy(), r["out_f32"]).max() <= OUT_REL_L2
    n = sm.add_rmsnorm(x, out, fmt=sm.MX_FP8)
    assert torch.equal(n.residual, x + out.float())
    w, wv = random_mx(N, H, sm.MX_FP4, 41, 118, 122)
    y = sm.mx_linear(n.mx, w, dev_status=status)
    assert sm.strata_read_status(status) == 0
    assert_product(y, n.mx.dequantize().double(), wv)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("E,I,H", [(1, 128, 128), (5, 128, 384), (3, 640, 2560)])
def test_pack_experts_strides(E, I, H, dtype):
    """Weights whose experts or rows are further apart than they are long."""
    g = gen(50)
    gate = torch.randn(E, I, H + 16, device=DEV, generator=g).to(dtype)[:, :, 8:H + 8]
    up = torch.randn(2 * E, I, H, device=DEV, generator=g).to(dtype)[::2]
    down = torch.randn(E, H, I, device=DEV, generator=g).to(dtype)
    blob = sm.pack_experts(gate, up, down)
    assert blob.blobs.shape == (E, sm.strata_expert_bytes(sm.FMT_MXFP4_32, H, I))
    for t, v in zip((gate, up, down), blob.dequantize(torch.bfloat16)):
        c, s = ref.quantize(n64(t).reshape(-1, t.shape[2]), sm.MX_FP4)
        assert np.array_equal(n64(v).reshape(c.shape), ref.dequantize(c, s, sm.MX_FP4))


def test_pack_experts_leaves_the_rest():
    """Blobs further apart than they are long keep the bytes between them."""
    E, I, H = 3, 128, 128
    size = sm.strata_expert_bytes(sm.FMT_MXFP4_32, H, I)
    ws = [torch.randn(E, r, k, device=DEV, generator=gen(60 + i)) for i, (r, k) in enumerate(((I, H), (I, H), (H, I)))]
    blobs = torch.full((E, size + 512), 0xA5, dtype=torch.uint8, device=DEV)
    sm.moe_mx_pack_experts(*ws, sm.DTYPE_F32, [w.stride(1) for w in ws], [w.stride(0) for w in ws], E, H, I, blobs,
                           size + 512)
    assert (blobs[:, size:] == 0xA5).all()
    want = sm.pack_experts(*ws).blobs
    planes = torch.zeros(size, dtype=torch.bool)
    at = 0
    for r, k in ((I, H), (I, H), (H, I)):
        for n in (r * k // 2, r * k // 32):
            planes[at:at + n] = True
            at = (at + n + 255) // 256 * 256
    assert torch.equal(blobs[:, :size].cpu()[:, planes], want.cpu()[:, planes])
    assert (blobs[:, :size].cpu()[:, ~planes] == 0xA5).all()


# ---------------------------------------------------------------- the native calls
def every_call(x, d, gain, w, bias):
    n = sm.add_rmsnorm(x, d, gain, 1e-5, out_dtype=torch.bfloat16, fmt=sm.MX_FP8)
    p = sm.add_rmsnorm(x, gain=gain, fmt=sm.MX_FP4, layout=sm.MX_ROWS)
    r = x.clone()
    q = sm.add_rmsnorm(r, d, out_dtype=torch.float32, residual_out=r)
    out = torch.empty(x.shape[0], w.rows + 8, dtype=torch.float16, device=DEV)[:, :w.rows]
    z = sm.mx_quantize(x, sm.MX_FP8)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    return (n.residual, n.out, n.mx.codes, n.mx.scales, p.mx.codes, p.mx.scales, q.residual, q.out,
            p.mx.dequantize(torch.float16), z.codes, z.scales, sm.mx_linear(n.mx, w),
            sm.mx_linear(z, w, bias, torch.float32, dev_status=status), sm.mx_linear(z, w, bias, out=out).clone())


def test_native_calls_are_the_python_ones(monkeypatch):
    g = gen(80)
    x = torch.randn(5, 256, device=DEV, generator=g)
    args = (x, torch.randn(5, 256, device=DEV, generator=g).half(), 1 + torch.rand(256, device=DEV, generator=g),
            sm.mx_quantize(torch.randn(70, 256, device=DEV, generator=g), sm.MX_FP4),
            torch.randn(70, device=DEV, generator=g))
    native = every_call(*args)
    as_parameters = every_call(args[0], args[1], torch.nn.Parameter(args[2]), *args[3:])
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
        aside = every_call(*args)
        torch.cuda.synchronize()
    monkeypatch.setattr(mx, "_fast", None)
    monkeypatch.setattr(mx, "_mxcalls", None)
    for got in (native, as_parameters, aside):
        for a, b in zip(got, every_call(*args)):
            assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_native_tensors_are_the_python_ones(monkeypatch):
    q = sm.mx_quantize(torch.randn(5, 160, device=DEV), sm.MX_FP4, sm.MX_ROWS)
    made = []
    for fast in (mx._fast, None):
        monkeypatch.setattr(mx, "_fast", fast)
        m = sm.MXTensor(q.codes, q.scales, sm.MX_FP4, 5, 160, sm.MX_ROWS)
        made.append(tuple(getattr(m, f) for f in mx._FIELDS))
        assert m.codes is q.codes and m.scales is q.scales
    assert made[0] == made[1]


def test_native_calls_keep_nothing():
    x = torch.randn(64, 256, device=DEV)
    d = torch.randn(64, 256, device=DEV)
    w = sm.mx_quantize(torch.randn(128, 256, device=DEV), sm.MX_FP4)
    b = torch.randn(128, device=DEV)
    held = [sys.getrefcount(o) for o in (x, d, w, b, torch.float32, x.device, sm.MXTensor)]
    for _ in range(3):
        every_call(x, d, None, w, b)
    torch.cuda.synchronize()
    gc.collect()
    used = torch.cuda.memory_allocated()
    for _ in range(50):
        every_call(x, d, None, w, b)
        sm.MXTensor(w.codes, w.scales, w.fmt, w.rows, w.K, w.layout)
    gc.collect()
    assert torch.cuda.memory_allocated() == used
    for before, o in zip(held, (x, d, w, b, torch.float32, x.device, sm.MXTensor)):
        assert sys.getrefcount(o) <= before + 2


def test_native_calls_leave_refusals_to_python():
    """The messages of mx.py, with the native calls armed."""
    x = torch.zeros(4, 128, device=DEV)
    q = sm.mx_quantize(x, sm.MX_FP8)
    rows = sm.mx_quantize(x, sm.MX_FP8, sm.MX_ROWS)
    w4 = sm.mx_quantize(x, sm.MX_FP4)
    c, s = rows.codes, rows.scales
    for call, error, match in (
            (lambda: sm.MXTensor(c, s, 3, 4, 128, sm.MX_ROWS), ValueError, "fmt"),
            (lambda: sm.MXTensor(c, s, sm.MX_FP8, 4, 120, sm.MX_ROWS), ValueError, "multiple of 32"),
            (lambda: sm.MXTensor(c, s, sm.MX_FP4, 4, 128, sm.MX_ROWS), ValueError, "codes"),
            (lambda: sm.MXTensor(c, s[:3], sm.MX_FP8, 4, 128, sm.MX_ROWS), ValueError, "scales"),
            (lambda: sm.MXTensor(c[:, ::2], s, sm.MX_FP4, 4, 128, sm.MX_ROWS), ValueError, "codes"),
            (lambda: sm.MXTensor(c.int(), s, sm.MX_FP8, 4, 128, sm.MX_ROWS), ValueError, "codes"),
            (lambda: sm.MXTensor(c, s.cpu(), sm.MX_FP8, 4, 128, sm.MX_ROWS), ValueError, "scales on"),
            (lambda: sm.mx_quantize(x.T, sm.MX_FP8), ValueError, "rows"),
            (lambda: sm.mx_quantize(x[:, 1:97], sm.MX_FP8), ValueError, "16-byte"),
            (lambda: sm.mx_quantize(x[:, :48], sm.MX_FP8), ValueError, "multiple of 32"),
            (lambda: sm.mx_quantize(x.double(), sm.MX_FP8), TypeError, "dtype"),
            (lambda: sm.mx_quantize(x.cpu(), sm.MX_FP8), ValueError, "CUDA"),
            (lambda: sm.mx_quantize(x, 7), ValueError, "fmt"),
            (lambda: sm.mx_quantize(x, sm.MX_FP8, 7), ValueError, "layout"),
            (lambda: sm.mx_quantize(x[0], sm.MX_FP8), ValueError, "matrix"),
            (lambda: q.dequantize(torch.int32), TypeError, "dtype"),
            (lambda: sm.add_rmsnorm(x, x.cpu(), fmt=sm.MX_FP8), ValueError, "on c"),
            (lambda: sm.add_rmsnorm(x, x[:2], fmt=sm.MX_FP8), ValueError, "delta"),
            (lambda: sm.add_rmsnorm(x, gain=x[0].half(), fmt=sm.MX_FP8), ValueError, "gain"),
            (lambda: sm.add_rmsnorm(x), ValueError, "out_dtype"),
            (lambda: sm.add_rmsnorm(x, eps=-1.0, fmt=sm.MX_FP8), sm.StrataError, "invalid"),
            (lambda: sm.add_rmsnorm(x, residual_out=x.half(), fmt=sm.MX_FP8), TypeError, "residual_out"),
            (lambda: sm.mx_linear(rows, q), ValueError, "tiles"),
            (lambda: sm.mx_linear(q, sm.mx_quantize(x[:, :64], sm.MX_FP8)), ValueError, "K = "),
            (lambda: sm.mx_linear(w4, q), sm.StrataError, "unsupported"),
            (lambda: sm.mx_linear(q, q, x[0]), ValueError, "bias"),
            (lambda: sm.mx_linear(q, q, out=x), ValueError, "out"),
            (lambda: sm.mx_linear(q, q, dev_status=x), ValueError, "dev_status"),
            (lambda: sm.mx_linear(q, q, out_dtype=torch.int32), TypeError, "dtype")):
        with pytest.raises(error, match=match):
            call()


def test_native_calls_leave_dispatch_modes_to_python():
    """A mode that watches torch's allocations sees those of these calls."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            names.append(func.name())
            return func(*args, **(kwargs or {}))

    names = []
    x = torch.randn(3, 64, device=DEV)
    want = sm.mx_quantize(x, sm.MX_FP8)
    with Seen():
        got = sm.mx_quantize(x, sm.MX_FP8)
    assert any(n.startswith("aten::empty") for n in names)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


def test_native_calls_leave_tensors_without_memory_to_python():
    sm.mx_quantize(torch.randn(3, 64, device=DEV), sm.MX_FP8)
    with pytest.raises(RuntimeError):
        torch.vmap(lambda r: sm.mx_quantize(r, sm.MX_FP8).codes)(torch.randn(2, 3, 64, device=DEV))


def test_native_calls_out_of_memory():
    x = torch.zeros(1, 4096, device=DEV).expand(1 << 26, 4096)  # its codes: 256 GiB
    with pytest.raises(torch.OutOfMemoryError):
        sm.mx_quantize(x, sm.MX_FP8)
    assert (sm.mx_quantize(x[:3], sm.MX_FP8).codes == 0).all()


def test_native_calls_of_several_threads():
    g = gen(81)
    xs = [torch.randn(5, 256, device=DEV, generator=g) for _ in range(4)]
    w = sm.mx_quantize(torch.randn(70, 256, device=DEV, generator=g), sm.MX_FP4)

    def calls(x):
        n = sm.add_rmsnorm(x, x, fmt=sm.MX_FP8, out_dtype=torch.float16)
        return n.residual, n.out, sm.mx_linear(n.mx, w), n.mx.dequantize()

    want = [calls(x) for x in xs]
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        gots = list(pool.map(lambda i: [calls(xs[i]) for _ in range(100)], range(4)))
    torch.cuda.synchronize()
    for i, got in enumerate(gots):
        for once in got:
            assert all(torch.equal(a, b) for a, b in zip(once, want[i]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_native_expert_calls_are_the_python_ones(monkeypatch, dtype):
    g = gen(82)
    ws = [torch.randn(3, *s, device=DEV, generator=g).to(dtype) for s in ((128, 384), (128, 384), (384, 128))]
    made = []
    for fast in (mx._fast, None):
        monkeypatch.setattr(mx, "_fast", fast)
        if fast is None:
            monkeypatch.setattr(mx, "_mxcalls", None)
        e = sm.pack_experts(*ws)
        made.append((e, e.dequantize(), e.dequantize(torch.float16)))
    (a, *x), (b, *y) = made
    assert (a.fmt, a.hidden, a.inter, a.num_experts, a.blobs.shape, a.qw.expert_stride) == \
        (b.fmt, b.hidden, b.inter, b.num_experts, b.blobs.shape, b.qw.expert_stride) and a.hidden == 384
    for p, q in zip(x, y):
        for u, v in zip(p, q):
            assert u.dtype == v.dtype and u.shape == v.shape and torch.equal(u, v)


def test_native_expert_calls_leave_refusals_to_python():
    w = torch.zeros(2, 128, 256, device=DEV)
    d = torch.zeros(2, 256, 128, device=DEV)
    e = sm.pack_experts(w, w, d)
    for call, error, match in (
            (lambda: sm.pack_experts(w[0], w, d), ValueError, "gate and up"),
            (lambda: sm.pack_experts(w, w, w), ValueError, "down"),
            (lambda: sm.pack_experts(w[:, :96], w[:, :96], d[:, :, :96]), ValueError, "128"),
            (lambda: sm.pack_experts(w[:0], w[:0], d[:0]), ValueError, "positive"),
            (lambda: sm.pack_experts(w, w.half(), d), TypeError, "one dtype"),
            (lambda: sm.pack_experts(w, w, d.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "rows"),
            (lambda: sm.pack_experts(w.cpu(), w, d), ValueError, "CUDA"),
            (lambda: e.dequantize(torch.int32), TypeError, "dtype")):
        with pytest.raises(error, match=match):
            call()


# ---------------------------------------------------------------- a matrix's memory
@pytest.mark.parametrize("fast", [True, False])
def test_matrix_follows_its_tensors(monkeypatch, fast):
    """Calls read a matrix where it is: copied, saved, given other memory."""
    x, w = torch.randn(5, 256, device=DEV, generator=gen(90)), torch.randn(70, 256, device=DEV, generator=gen(91))
    if not fast:
        monkeypatch.setattr(mx, "_fast", None)
        monkeypatch.setattr(mx, "_mxcalls", None)
    q = sm.mx_quantize(x, sm.MX_FP8)
    v = q.dequantize()
    for made in (sm.mx_quantize(w, sm.MX_FP4), sm.mx_tile_scales(sm.mx_quantize(w, sm.MX_FP4, sm.MX_ROWS))):
        want, values = sm.mx_linear(q, made), made.dequantize()
        other = sm.mx_quantize(2 * w, sm.MX_FP4)
        twice = sm.mx_linear(q, other)
        r = copy.deepcopy(made)
        p = sm.MXTensor(torch.nn.Parameter(made.codes.clone(), requires_grad=False),
                        torch.nn.Parameter(made.scales.clone(), requires_grad=False), sm.MX_FP4, 70, 256, sm.MX_TILES)
        made.codes.zero_()
        assert torch.equal(sm.mx_linear(q, r), want) and torch.equal(r.dequantize(), values)
        assert torch.equal(sm.mx_linear(q, p), want)
        for m in (r, p):
            m.codes.data, m.scales.data = other.codes.clone(), other.scales.clone()
            assert torch.equal(sm.mx_linear(q, m), twice) and torch.equal(m.dequantize(), 2 * values)
            m.codes.data = m.codes.data[:64]
            for call in (m.dequantize, lambda: sm.mx_linear(q, m)):
                with pytest.raises(ValueError, match="codes must be"):
                    call()
    f = io.BytesIO()
    torch.save(q, f)
    f.seek(0)
    assert torch.equal(torch.load(f, weights_only=False).dequantize(), v)


# ---------------------------------------------------------------- calls of several threads
def test_linear_of_several_threads_and_shapes():
    """Products of one tile width that want different amounts of shared memory,
    side by side: the amount is a property of the kernel, not of the call."""
    shapes = [(4, 128, 128), (4, 4100, 2560), (4, 40000, 128), (4, 2560, 8192)]
    made = []
    for i, (T, N, K) in enumerate(shapes):
        x, _ = random_mx(T, K, sm.MX_FP8, 100 + i)
        w, _ = random_mx(N, K, sm.MX_FP4, 200 + i)
        y = torch.empty(T, N, device=DEV)
        made.append((x, w, y, sm.mx_linear(x, w, out_dtype=torch.float32)))
    torch.cuda.synchronize()
    start = threading.Barrier(len(shapes))

    def calls(i):
        (T, N, K), (x, w, y, _) = shapes[i], made[i]
        torch.cuda.synchronize()  # the device is this thread's too
        stream = torch.cuda.Stream().cuda_stream
        a = (x.codes, sm.MX_FP8, x.scales, T, w.codes, sm.MX_FP4, w.scales, N, K, None, y, sm.DTYPE_F32, N, None)
        start.wait()
        return [rc for _ in range(4000) if (rc := sm.moe_mx_linear(*a, stream, check=False))]

    with concurrent.futures.ThreadPoolExecutor(len(shapes)) as pool:
        failed = list(pool.map(calls, range(len(shapes))))
    torch.cuda.synchronize()
    assert failed == [[]] * len(shapes)
    for *_, y, want in made:
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,N,K", [(4, 300, 256), (200, 300, 256), (2000, 2048, 1024)])
def test_linear_from_a_thread_that_has_not_used_the_device(T, N, K):
    x, _ = random_mx(T, K, sm.MX_FP8, 110)
    w, _ = random_mx(N, K, sm.MX_FP4, 111)
    want = sm.mx_linear(x, w)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        pool.submit(sm.mx_linear, x, w, out=out).result()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- a stream that is not the current one
def owner(t):
    """The stream whose memory a tensor is in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


@pytest.mark.parametrize("fast", [True, False])
def test_results_are_the_streams_that_writes_them(monkeypatch, fast):
    """Memory that the current stream has given back may still be written by
    what it has yet to do: a call on another stream takes none of it."""
    if not fast:
        monkeypatch.setattr(mx, "_fast", None)
        monkeypatch.setattr(mx, "_mxcalls", None)
    x, d = (torch.randn(5, 256, device=DEV, generator=gen(120 + i)) for i in range(2))
    gate = torch.randn(2, 128, 256, device=DEV, generator=gen(122))
    down = torch.randn(2, 256, 128, device=DEV, generator=gen(123))

    def every(stream):
        q = sm.mx_quantize(x, sm.MX_FP8, stream=stream)
        r = sm.mx_tile_scales(sm.mx_quantize(x, sm.MX_FP8, sm.MX_ROWS, stream=stream), stream)
        n = sm.add_rmsnorm(x, d, out_dtype=torch.float16, fmt=sm.MX_FP4, stream=stream)
        e = sm.pack_experts(gate, gate, down, stream)
        return [q.codes, q.scales, q.dequantize(stream=stream), r.scales, n.residual, n.out, n.mx.codes,
                sm.mx_linear(q, r, stream=stream), e.blobs, *e.dequantize(stream=stream)]

    want = every(None)
    torch.cuda.synchronize()
    current, side = torch.cuda.current_stream(), torch.cuda.Stream()
    assert all(owner(t) == current.cuda_stream for t in want)
    for stream in (side, side.cuda_stream):
        got = every(stream)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == current
        for a, b in zip(got, want):
            assert owner(a) == side.cuda_stream and a.shape == b.shape and a.dtype == b.dtype
            assert a.dtype == torch.uint8 or torch.equal(a, b)
    with torch.cuda.stream(side):  # the default stream by its handles, from another one
        for handle in (0, 1, torch.cuda.default_stream()):
            got = every(handle)
            torch.cuda.synchronize()
            assert all(owner(t) == 0 for t in got) and torch.equal(got[7], want[7])
        assert torch.cuda.current_stream() == side
    with pytest.raises(ValueError, match="default stream"):
        sm.mx_quantize(x, sm.MX_FP8, stream=2)


def test_a_stream_inside_a_capture():
    """A step whose product runs on a second stream, captured and replayed."""
    x, d = (torch.randn(4, 512, device=DEV, generator=gen(124 + i)) for i in range(2))
    w, _ = random_mx(300, 512, sm.MX_FP4, 126, 116, 120)
    want = sm.mx_linear(sm.add_rmsnorm(x, d, fmt=sm.MX_FP8).mx, w)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        n = sm.add_rmsnorm(x, d, fmt=sm.MX_FP8)
        side.wait_stream(torch.cuda.current_stream())
        y = sm.mx_linear(n.mx, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ---------------------------------------------------------------- the norm's mean
@pytest.mark.parametrize("H", [32, 392, 2560, 2592])
def test_norm_rounds_the_mean_once(H):
    """Rows of m ones: their squares sum to m exactly, so that the mean has one rounding, m / H's,
    and the ones become its inverse root as the device's function gives it."""
    x = torch.ones(H, H, device=DEV).tril()
    mean = (torch.arange(1, H + 1, device=DEV).double() / H).float()
    assert torch.equal(sm.add_rmsnorm(x, eps=0.0, out_dtype=torch.float32).out[:, 0], torch.rsqrt(mean))


# fp32 steps of h where nothing is added: a sum of up to 16 squares in turn (16 half steps, halved by
# the root), the mean's one rounding (a half, halved), the device's inverse root (4 half steps), two
# products (2).
H_REL_ALONE = (8 + 0.5 + 4 + 2) * 2.0 ** -24


@pytest.mark.parametrize("T,H", [(1, 32), (7, 256), (5, 512), (3, 392), (130, 2592), (9481, 1024), (40, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_alone_is_within_its_steps(dtype, T, H):
    x = torch.randn(T, H, device=DEV, generator=gen(T + H)).to(dtype)
    gain = 1 + 0.1 * torch.randn(H, device=DEV, generator=gen(1))
    h = x.double() / (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
    out = sm.add_rmsnorm(x, gain=gain, out_dtype=torch.float32).out
    assert ((out.double() - h).abs() <= H_REL_ALONE * h.abs()).all()


# rows whose squares leave fp32's range, above and below: (largest magnitude, eps)
FAR = [(2.0 ** 127, 1e-6), (1e30, 1e-6), (3e19, 0.0), (2.0 ** 60, 1e-6), (1e-12, 0.0), (1e-25, 0.0), (1e-38, 0.0),
       (2.0 ** -140, 0.0), (1e-25, 1e-50), (1e-18, 1e-36), (1e-25, 1e-6)]


@pytest.mark.parametrize("T,H", [(1, 32), (7, 256), (5, 512), (6, 1024), (131, 2592), (3, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_rows_far_from_one(dtype, T, H):
    """h is about one whatever the rows' magnitude; neighbours in a CTA are ordinary rows.  Rows of
    2^-140 are subnormals: what they are is exact, and so is all that is done to them."""
    x = torch.randn(T, H, device=DEV, generator=gen(T + H)).clamp(-3, 3)
    gain = 1 + 0.1 * torch.randn(H, device=DEV, generator=gen(1))
    for size, eps in FAR:
        far = x.clone()
        far[::2] *= size / 4
        far = far.to(dtype)
        if eps == 0 and not far.any(1).all():
            continue  # bf16 has nothing that small
        eps32 = torch.tensor(eps, dtype=torch.float32).double().item()
        h = far.double() / (far.double().pow(2).mean(-1, keepdim=True) + eps32).sqrt() * gain.double()
        n = sm.add_rmsnorm(far, gain=gain, eps=eps, out_dtype=torch.float32, fmt=sm.MX_FP8)
        assert n.out.isfinite().all()
        # (an element 2^56 below a row of 2^61 and more may lose its last bits: below 2^-120 of h)
        assert ((n.out.double() - h).abs() <= H_REL_ALONE * h.abs() + 2.0 ** -120).all(), (size, eps)
        q = sm.mx_quantize(n.out, sm.MX_FP8)
        assert torch.equal(n.mx.codes, q.codes) and torch.equal(n.mx.scales, q.scales)


def test_norm_of_mixed_and_infinite_rows():
    """One large element among ordinary ones; an infinite one makes its row 0 and itself NaN, as the
    formula has it; rows of zeros without eps are 0 / 0."""
    H = 1024
    x = torch.randn(6, H, device=DEV, generator=gen(3))
    x[0, 5] = 1e30
    x[1, 7] = float("inf")
    x[2] = 0
    x[3, 9] = -float("inf")
    x[3, 8] = float("nan")
    n = sm.add_rmsnorm(x, eps=0.0, out_dtype=torch.float32, fmt=sm.MX_FP4)
    h = x[0].double() / x[0].double().pow(2).mean().sqrt()
    assert ((n.out[0].double() - h).abs() <= H_REL_ALONE * h.abs() + 2.0 ** -120).all()
    assert n.out[1, 7].isnan() and (torch.cat([n.out[1, :7], n.out[1, 8:]]) == 0).all()
    assert n.out[2].isnan().all() and n.out[3].isnan().all()
    assert torch.equal(n.out[4:], sm.add_rmsnorm(x[4:].clone(), eps=0.0, out_dtype=torch.float32).out)
    v = n.mx.dequantize()
    assert v[1, :32].isnan().all() and (v[1, 32:] == 0).all() and v[2:4].isnan().all() and v[4:].isfinite().all()
