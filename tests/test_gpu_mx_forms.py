"""GPU tests of every form of the microscaled product: each shape of
tests/mx_shapes.py against the plain product in 64 bits, with scales of their
own in every block, a bias, each output type, rows of y further apart than
they are long, and NaN blocks; and the forms side by side on two streams."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import expert_ffn_execution_b200 as sm  # noqa: E402
from tests import mx_reference as ref  # noqa: E402
from tests import mx_shapes  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FORMATS = {"8x4": (sm.MX_FP8, sm.MX_FP4), "8x8": (sm.MX_FP8, sm.MX_FP8), "4x4": (sm.MX_FP4, sm.MX_FP4)}
CASES = [(f, form, s) for f in FORMATS for form, shapes in
         (mx_shapes.NARROW_K if f == "4x4" else mx_shapes.WIDE_K).items() for s in shapes]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def scale_byte(row, block, K):
    """Where a block's scale is in the plane of tiles."""
    return (row // 128 * (K // 128) + block // 4) * 512 + row % 32 * 16 + row // 32 % 4 * 4 + block % 4


def matrix(rows, K, fmt, seed):
    """A matrix whose blocks have scales of their own, and its values in 64 bits by table."""
    g = gen(seed)
    n = 16 if fmt == sm.MX_FP4 else 127  # E4M3: no NaN
    codes = torch.randint(0, n, (rows, K), dtype=torch.uint8, device=DEV, generator=g)
    if fmt == sm.MX_FP8:
        codes |= torch.randint(0, 2, (rows, K), dtype=torch.uint8, device=DEV, generator=g) << 7
    scales = torch.randint(116, 122, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    table = torch.from_numpy(ref.values(fmt)).to(DEV)
    values = table[codes.int()]
    values.view(rows, -1, 32).mul_(torch.ldexp(torch.ones_like(scales, dtype=torch.float64),
                                               scales.int() - 127).unsqueeze(-1))
    stored = codes if fmt == sm.MX_FP8 else codes[:, 0::2] | codes[:, 1::2] << 4
    tiles = torch.zeros(-(-rows // 128) * (K // 128) * 512, dtype=torch.uint8, device=DEV)
    r = torch.arange(rows, device=DEV).unsqueeze(1)
    b = torch.arange(K // 32, device=DEV).unsqueeze(0)
    tiles[scale_byte(r, b, K).flatten()] = scales.flatten()
    return sm.MXTensor(stored.contiguous(), tiles, fmt, rows, K, sm.MX_TILES), values


def output(T, N, dtype, aligned):
    """[T, N] with other elements on all sides, rows on 16-byte boundaries or on odd ones."""
    wide = torch.full((T + 2, (N + 31) // 16 * 16 + (0 if aligned else 1)), 7.0, dtype=dtype, device=DEV)
    at = 8 if aligned else 3
    return wide, wide[1:-1, at:N + at]


@pytest.mark.parametrize("formats,form,shape", CASES, ids=str)
def test_form(formats, form, shape):
    """|error| <= one rounding of the result + the fp32 sums': products of codes are exact; a 32-wide
    block is added to the sum so far with every term kept to 24 bits of the largest, a whole step 2^-23 of
    at most sum |x w| for each of its 32 terms' tails together, so K/32 steps; 8 joined parts and a bias 9."""
    T, N, K = shape
    xf, wf = FORMATS[formats]
    x, xv = matrix(T, K, xf, T + N)
    w, wv = matrix(N, K, wf, T + N + 1)
    bias = torch.randn(N, device=DEV, generator=gen(2))
    want, mag = xv @ wv.T, xv.abs() @ wv.abs().T
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    aligned = form != (0, False)
    for dtype in HALF_STEP:
        for add in (None, bias):
            wide, out = output(T, N, dtype, aligned)
            assert sm.mx_linear(x, w, add, out=out, dev_status=status) is out
            exact = want if add is None else want + add.double()
            size = mag if add is None else mag + add.double().abs()
            tol = HALF_STEP[dtype] * exact.abs() + (K / 32 + 9) * 2.0 ** -23 * size + \
                (2.0 ** -25 if dtype == torch.float16 else 0)
            bad = ~((out.double() - exact).abs() <= tol)
            assert not bad.any(), (dtype, int(bad.sum()), bad.nonzero()[:5].tolist())
            out.fill_(7.0)
            assert (wide == 7.0).all()  # nothing else was written
    # blocks of NaN: in x's first and last row, in w's last
    wide, out = output(T, N, torch.float32, aligned)
    clean = sm.mx_linear(x, w, out=out).clone()
    blocks = K // 32
    x.scales[scale_byte(T - 1, blocks - 1, K)] = 255
    if T > 2:
        x.scales[scale_byte(0, blocks // 2, K)] = 255
    w.scales[scale_byte(N - 1, blocks - 2, K)] = 255
    got = sm.mx_linear(x, w, out=out)
    assert got[T - 1].isnan().all() and got[:, N - 1].isnan().all() and (T <= 2 or got[0].isnan().all())
    rest = slice(1 if T > 2 else 0, T - 1), slice(0, N - 1)
    assert torch.equal(got[rest], clean[rest])
    assert sm.strata_read_status(status) == 0


@pytest.mark.parametrize("formats", list(FORMATS))
def test_forms_on_two_streams_at_once(formats):
    """Calls of every form side by side on two streams give the bits of the calls in turn."""
    xf, wf = FORMATS[formats]
    made = []
    for form, shapes in (mx_shapes.NARROW_K if formats == "4x4" else mx_shapes.WIDE_K).items():
        T, N, K = shapes[0]
        x, w = matrix(T, K, xf, 3)[0], matrix(N, K, wf, 4)[0]
        outs = [output(T, N, torch.bfloat16, form != (0, False))[1] for _ in range(3)]
        made.append((x, w, outs))
        sm.mx_linear(x, w, out=outs[0])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(4):
        for i in range(len(made)):
            for j, s in enumerate(streams):  # another neighbour each turn
                x, w, outs = made[(i + j * (turn + 1)) % len(made)]
                with torch.cuda.stream(s):
                    sm.mx_linear(x, w, out=outs[1 + j], dev_status=status)
        torch.cuda.synchronize()
        for _, _, (want, *got) in made:
            for y in got:
                assert torch.equal(y, want)
                y.zero_()
        torch.cuda.synchronize()
    assert sm.strata_read_status(status) == 0
