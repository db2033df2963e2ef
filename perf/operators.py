"""Cases of the microscaled (MX) operators: the residual's addition with the
root-mean-square norm and an 8- or 4-bit output, the quantiser and its
read-back, and the product of two quantised matrices.

Every case can be run in two ways.  With `own` false, run() computes the
operators in elementary torch operations in 32 bits; with `own` true it makes
the calls that a user of expert_ffn_execution_b200 makes.  exact() gives the
same outputs from the definitions in 64 bits.

The format (OCP Microscaling v1.0): blocks of 32 consecutive elements of a row
share one E8M0 scale byte e, worth 2^(e-127); elements are E2M1 (FP4: 0, 0.5,
1, 1.5, 2, 3, 4, 6 and their negatives) or E4M3 (FP8, largest 448).  For a
block of largest magnitude m the scale is 2^s, s = floor(log2 m) - emax
clamped to -127..127 (emax 2 for FP4, 8 for FP8; s = -127 for a block of
zeros), and an element is x / 2^s rounded to nearest even and saturated.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EMAX = {"fp4": 2, "fp8": 8}
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # One decode step of 1 token and 3 drafts between two layers: the attention output joins
        # the fp32 residual stream and the next projection's input is normalised to MXFP8.
        {"name": "norm step", "op": "norm", "T": 4, "H": 2560, "x": "f32", "delta": "bf16", "out": "bf16", "fmt": "fp8"},
        # A prefill chunk of the large-expert layer: the normalised rows are wanted in bf16 (the
        # router) and in MXFP8 (the projections).
        {"name": "norm chunk", "op": "norm", "T": 8192, "H": 4096, "x": "f32", "delta": "bf16", "out": "bf16", "fmt": "fp8"},
        # A ragged batch with a 16-bit residual stream, a width of 81 blocks, 4-bit output.
        {"name": "norm odd", "op": "norm", "T": 1001, "H": 2592, "x": "bf16", "delta": "bf16", "out": "f16", "fmt": "fp4"},
        # Loading a checkpoint: 32 experts' bf16 weights become the layer's MXFP4 blobs, and are
        # read back to check them.
        {"name": "pack experts", "op": "experts", "E": 32, "H": 2560, "I": 640},
        # The activations of one decode step, quantised and read back.
        {"name": "quantize step", "op": "quantize", "rows": 4, "K": 2560, "x": "bf16", "fmt": "fp8"},
        # An fp32 weight matrix of odd height and 23 blocks a row.
        {"name": "quantize odd", "op": "quantize", "rows": 7777, "K": 736, "x": "f32", "fmt": "fp4"},
        # Decode, one token, 8-bit activations and 4-bit weights: a dense up projection.
        {"name": "linear step", "op": "linear", "T": 1, "K": 2560, "N": 10240, "a": "fp8", "w": "fp4", "bias": False},
        # Decode, a verify window over a vocabulary-sized matrix, both sides in 4 bits.
        {"name": "linear verify", "op": "linear", "T": 4, "K": 8192, "N": 32768, "a": "fp4", "w": "fp4", "bias": False},
        # A few hundred tokens into an odd number of features, with a bias.
        {"name": "linear odd", "op": "linear", "T": 300, "K": 2688, "N": 5001, "a": "fp8", "w": "fp8", "bias": True},
        # A prefill chunk, 8-bit activations and 4-bit weights.
        {"name": "linear chunk 8x4", "op": "linear", "T": 8192, "K": 2560, "N": 10240, "a": "fp8", "w": "fp4", "bias": False},
        # A prefill chunk, both sides in 4 bits: the most arithmetic.
        {"name": "linear chunk 4x4", "op": "linear", "T": 8192, "K": 4096, "N": 16384, "a": "fp4", "w": "fp4", "bias": False},
        # The operators together, as between two layers of a decode step: addition, norm to
        # MXFP8, and the projection that reads it.
        {"name": "norm and linear", "op": "norm+linear", "T": 16, "H": 4096, "N": 4096, "x": "f32", "delta": "bf16", "a": "fp8", "w": "fp4"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "experts", "quantize", "linear", "linear", "linear", "norm+linear"])
    if op == "norm":
        H = 32 * _log_int(rng, 4, 256)
        return {"op": op, "T": _log_int(rng, 1, min(8192, 8192 * 4096 // H)), "H": H, "x": rng.choice(["f32", "bf16"]),
                "delta": rng.choice(["bf16", "f32", "f16", "none"]), "out": rng.choice(["none", "bf16", "f16"]),
                "fmt": rng.choice(["fp8", "fp4"])}
    if op == "experts":
        H, I = 128 * rng.randint(2, 32), 128 * rng.randint(1, 16)
        return {"op": op, "E": _log_int(rng, 1, max(1, min(64, 32 * 2560 * 640 // (H * I)))), "H": H, "I": I}
    if op == "quantize":
        K = 32 * _log_int(rng, 1, 256)
        return {"op": op, "rows": _log_int(rng, 1, min(16384, (1 << 25) // K)), "K": K, "x": rng.choice(["bf16", "f32", "f16"]),
                "fmt": rng.choice(["fp8", "fp4"])}
    K, N = 128 * _log_int(rng, 2, 64), _log_int(rng, 1, 32768)
    T = _log_int(rng, 1, max(1, min(8192, 8192 * 4096 * 16384 // (N * K))))
    a, w = rng.choice([("fp8", "fp4"), ("fp4", "fp4"), ("fp8", "fp8")])
    if op == "norm+linear":
        return {"op": op, "T": T, "H": K, "N": N, "x": "f32", "delta": rng.choice(["bf16", "none"]), "a": a, "w": w}
    return {"op": op, "T": T, "K": K, "N": N, "a": a, "w": w, "bias": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _matrix(g, rows, K, fmt):
    """A quantised weight matrix as a program holds it: codes, and the scales by rows and in the
    product's tiles of 128 rows x 4 blocks (row r, block b at byte (r%32)*16 + (r//32%4)*4 + b%4)."""
    if fmt == "fp4":
        codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    else:  # E4M3 codes of magnitudes 1 to 30: exponent fields 7..11
        codes = torch.randint(7 << 3, 12 << 3, (rows, K), dtype=torch.uint8, device=DEV, generator=g)
        codes |= torch.randint(0, 2, (rows, K), dtype=torch.uint8, device=DEV, generator=g) << 7
    lo = 118 if fmt == "fp4" else 115
    scales = torch.randint(lo, lo + 4, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    rt, kt = -(-rows // 128), -(-K // 128)
    tiles = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=DEV)
    tiles[:rows, : K // 32] = scales
    tiles = tiles.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes, scales, tiles


def _acts(g, rows, K, dtype):
    """Rows as they leave a layer: normal values, a few channels ten times as large."""
    x = torch.randn(rows, K, device=DEV, generator=g)
    x[:, torch.randint(0, K, (max(1, K // 256),), device=DEV, generator=g)] *= 10
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"].startswith("norm"):
        T, H = case["T"], case["H"]
        s["res"] = _acts(g, T, H, DTYPES[case["x"]])
        s["dlt"] = None if case["delta"] == "none" else torch.randn(T, H, device=DEV, generator=g).to(DTYPES[case["delta"]])
        s["gain"] = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
    if case["op"] == "experts":
        E, H, I = case["E"], case["H"], case["I"]
        for name, shape in (("gate", (E, I, H)), ("up", (E, I, H)), ("down", (E, H, I))):
            s[name] = (0.02 * torch.randn(shape, device=DEV, generator=g)).bfloat16()
    if case["op"] == "quantize":
        s["data"] = _acts(g, case["rows"], case["K"], DTYPES[case["x"]])
    if case["op"] == "linear":
        s["data"] = _acts(g, case["T"], case["K"], torch.bfloat16)
        s["add"] = torch.randn(case["N"], device=DEV, generator=g) if case["bias"] else None
    if case["op"].endswith("linear"):
        s["codes"], s["scales"], s["tiles"] = _matrix(g, case["N"], case.get("K") or case["H"], case["w"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------- the plain forms, in 32 bits
def _pow2(s):
    """2^s in fp32 for whole s in -126..127, from its bits."""
    return ((s + 127) << 23).view(torch.float32)


def _mx(x, fmt):
    """The values that x's rows have in the format: fp32, each block rounded on its own scale."""
    b = x.float().unflatten(-1, (-1, 32))
    m = b.abs().amax(-1, keepdim=True)
    s = (torch.frexp(m)[1] - 1 - EMAX[fmt]).clamp(-126, 126)  # the inputs here are far from the clamps
    a = b * _pow2(-s)
    if fmt == "fp4":
        r = a.abs()
        r = torch.where(r < 2, torch.round(2 * r) / 2, torch.where(r < 4, torch.round(r), 2 * torch.round(r / 2))).clamp(max=6)
    else:
        r = a.abs()
        q = _pow2((torch.frexp(r)[1] - 1).clamp(min=-6) - 3)
        r = (torch.round(r / q) * q).clamp(max=448)
    return (torch.copysign(r, a) * _pow2(s) * (m > 0)).flatten(-2)


def _values(codes, scales, fmt, wide=torch.float32):
    """The values of a quantised matrix."""
    if fmt == "fp4":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=wide, device=codes.device)
        table = torch.cat([table, -table])
        v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    else:
        c = codes.int()
        e, m = (c >> 3) & 15, (c & 7).to(wide)
        v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).to(wide)), m * 2.0 ** -9)
        v = torch.where(c >= 128, -v, v)
    return (v.unflatten(-1, (-1, 32)) * _pow2(scales.int() - 127).to(wide).unsqueeze(-1)).flatten(-2)


def _plain_norm(s):
    r = s["res"].float() if s["dlt"] is None else s["res"].float() + s["dlt"].float()
    h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["gain"]
    return r.to(s["res"].dtype), h


def _plain(s):
    op = s["op"]
    if op == "norm":
        r, h = _plain_norm(s)
        return {"residual": r, "out": None if s["out"] == "none" else h.to(DTYPES[s["out"]]), "quantised": _mx(h, s["fmt"]).bfloat16()}
    if op == "experts":
        return {n: _mx(s[n], "fp4").bfloat16() for n in ("gate", "up", "down")}
    if op == "quantize":
        return _mx(s["data"], s["fmt"]).bfloat16()
    if op == "linear":
        y = _mx(s["data"], s["a"]) @ _values(s["codes"], s["scales"], s["w"]).T
        return (y if s["add"] is None else y + s["add"]).bfloat16()
    r, h = _plain_norm(s)
    return {"residual": r, "y": (_mx(h, s["a"]) @ _values(s["codes"], s["scales"], s["w"]).T).bfloat16()}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import expert_ffn_execution_b200 as sm

    op = s["op"]
    code = {"fp4": sm.MX_FP4, "fp8": sm.MX_FP8}
    if op == "norm":
        n = sm.add_rmsnorm(s["res"], s["dlt"], s["gain"], EPS, out_dtype=None if s["out"] == "none" else DTYPES[s["out"]], fmt=code[s["fmt"]])
        return {"residual": n.residual, "out": n.out, "quantised": n.mx.dequantize(torch.bfloat16)}
    if op == "experts":
        w = sm.pack_experts(s["gate"], s["up"], s["down"])
        return dict(zip(("gate", "up", "down"), w.dequantize(torch.bfloat16)))
    if op == "quantize":
        return sm.mx_quantize(s["data"], code[s["fmt"]]).dequantize(torch.bfloat16)
    K = s.get("K") or s["H"]
    w = sm.MXTensor(s["codes"], s["tiles"], code[s["w"]], s["N"], K, sm.MX_TILES)
    if op == "linear":
        return sm.mx_linear(sm.mx_quantize(s["data"], code[s["a"]]), w, s["add"], dev_status=s["status"])
    n = sm.add_rmsnorm(s["res"], s["dlt"], s["gain"], EPS, fmt=code[s["a"]])
    return {"residual": n.residual, "y": sm.mx_linear(n.mx, w, dev_status=s["status"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _bits(fmt):
    return (4.25 if fmt == "fp4" else 8.25) / 8


def _size(name):
    return {"f32": 4, "none": 0}.get(name, 2)


def work(case):
    op = case["op"]
    by = fl = 0
    if op.startswith("norm"):
        n = case["T"] * case["H"]
        by += n * _size(case["x"]) + 4 * case["H"]
        by += 0 if case["delta"] == "none" else n * (_size(case["delta"]) + _size(case["x"]))  # the new residual is written
        fl += 6 * n
    if op == "norm":
        by += n * (_size(case["out"]) + _bits(case["fmt"]) + 2)  # written in 8 or 4 bits, read back in 16
    if op == "experts":
        n = 3 * case["E"] * case["H"] * case["I"]
        by, fl = n * (2 + _bits("fp4") + 2), 4 * n
    if op == "quantize":
        n = case["rows"] * case["K"]
        by, fl = n * (_size(case["x"]) + _bits(case["fmt"]) + 2), 4 * n
    if op.endswith("linear"):
        K = case.get("K") or case["H"]
        by += K * case["N"] * _bits(case["w"]) + 2 * case["T"] * case["N"] + (4 * case["N"] if case.get("bias") else 0)
        by += 2 * case["T"] * K if op == "linear" else 0
        fl += 2 * case["T"] * case["N"] * K
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------- the definitions in 64 bits
def _nearest(a, grid):
    """a's magnitude rounded to the nearest of `grid` (ascending, an even number of steps apart
    from its first: a tie goes to the even index), saturating; fp64."""
    a = a.abs().clamp(max=grid[-1].item())
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    return grid[torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)]


def _exact_mx(x, fmt):
    if fmt == "fp4":
        grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    else:
        grid = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    flat, to = x.reshape(-1, 32), out.view(-1, 32)
    for at in range(0, flat.shape[0], 1 << 20):  # in parts: the search takes several times the data
        b = flat[at : at + (1 << 20)].double()
        m = b.abs().amax(1, keepdim=True)
        # floor(log2 m) from the 64-bit number's own exponent
        e = ((m.view(torch.int64) >> 52) & 2047) - 1023
        scale = torch.ldexp(torch.ones_like(m), (e - EMAX[fmt]).clamp(-127, 127))
        to[at : at + (1 << 20)] = torch.where(m > 0, torch.copysign(_nearest(b / scale, grid), b) * scale, torch.zeros_like(b))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        r = s["res"].double()
        if s["dlt"] is not None:
            r = r + s["dlt"].double()
        h = r / torch.sqrt(r.square().sum(-1, keepdim=True) / case["H"] + EPS) * s["gain"].double()
    if op == "norm":
        # None for "quantised": next to a border between two codes the last bit of a 32-bit norm
        # decides which of them a value gets, and either stands for it as well.  The quantiser's own
        # cases, whose inputs are given, compare its roundings exactly.
        return {"residual": r, "out": None if case["out"] == "none" else h, "quantised": None}
    if op == "experts":
        return {n: _exact_mx(s[n], "fp4") for n in ("gate", "up", "down")}
    if op == "quantize":
        return _exact_mx(s["data"], case["fmt"])
    w = _values(s["codes"], s["scales"], case["w"], torch.float64)
    if op == "linear":
        y = _exact_mx(s["data"], case["a"]) @ w.T
        return y if s["add"] is None else y + s["add"].double()
    return {"residual": r, "y": _exact_mx(h, case["a"]) @ w.T}
