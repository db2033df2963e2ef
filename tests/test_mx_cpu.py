"""CPU checks of the microscaled operators: the C entry points refuse bad
arguments before anything is enqueued, the torch-level calls refuse what the
library could not read, and the reference the GPU tests use is pinned."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import expert_ffn_execution_b200 as sm
from expert_ffn_execution_b200 import _binding as B
from tests import mx_reference as ref

P = 4096  # an aligned address nothing reads: every call here ends in the host checks


def test_reference_values():
    assert ref.values(ref.FP4).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]
    v = ref.values(ref.FP8)
    assert v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448 and v[0xfe] == -448
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, v.astype(np.float32), equal_nan=True)


def test_reference_quantize():
    x = np.zeros((1, 32))
    c, s = ref.quantize(x, ref.FP4)
    assert s[0, 0] == 0 and not c.any()
    x[0, :8] = [4, 7.9, -5, 5, 2.5, 3.5, 0.25, 0.75]  # scale 1: ties to even, saturation
    c, s = ref.quantize(x, ref.FP4)
    assert s[0, 0] == 127
    assert ref.values(ref.FP4)[c[0, :8]].tolist() == [4, 6, -4, 4, 2, 4, 0, 1]
    x[0, 0] = np.inf
    c, s = ref.quantize(x, ref.FP8)
    assert s[0, 0] == 255 and not c.any()


@pytest.mark.parametrize("rows,K", [(0, 32), (1, 32), (128, 128), (129, 160), (5001, 2688)])
def test_scale_bytes(rows, K):
    assert sm.moe_mx_scale_bytes(rows, K, sm.MX_ROWS) == rows * K // 32
    assert sm.moe_mx_scale_bytes(rows, K, sm.MX_TILES) == -(-rows // 128) * -(-K // 128) * 512
    if rows and rows * K < 1 << 20:
        assert ref.tile_scales(np.zeros((rows, K // 32), np.uint8)).size == sm.moe_mx_scale_bytes(
            rows, K, sm.MX_TILES)


def test_scale_bytes_of_bad_arguments():
    for a in ((-1, 32, 0), (1, 0, 0), (1, 48, 0), (1, 32, 2)):
        assert sm.moe_mx_scale_bytes(*a) == 0


def quant(**k):
    a = dict(src=P, src_dtype=sm.DTYPE_BF16, batch=1, rows=4, K=64, src_row_stride=64,
             src_batch_stride=256, fmt=sm.MX_FP4, codes=P, codes_batch_stride=128, scales=P,
             scale_layout=sm.MX_ROWS, scales_batch_stride=8)
    a.update(k)
    return sm.moe_mx_quantize(**a, stream=0, check=False)


def dequant(**k):
    a = dict(codes=P, codes_batch_stride=128, scales=P, scale_layout=sm.MX_ROWS,
             scales_batch_stride=8, fmt=sm.MX_FP4, batch=1, rows=4, K=64, dst=P,
             dst_dtype=sm.DTYPE_BF16, dst_row_stride=64, dst_batch_stride=256)
    a.update(k)
    return sm.moe_mx_dequantize(**a, stream=0, check=False)


BAD_BATCH = [dict(fmt=0), dict(fmt=3), dict(scale_layout=2), dict(batch=-1), dict(rows=-1),
             dict(K=48), dict(K=0), dict(codes=None), dict(scales=None), dict(codes=P + 8),
             dict(scale_layout=sm.MX_TILES, scales=P + 8),
             dict(batch=2, codes_batch_stride=112), dict(batch=2, codes_batch_stride=136),
             dict(batch=2, scales_batch_stride=7),
             dict(batch=2, scale_layout=sm.MX_TILES, scales_batch_stride=511),
             dict(batch=1 << 20, rows=1 << 11, codes_batch_stride=1 << 16, scales_batch_stride=1 << 12)]


@pytest.mark.parametrize("k", BAD_BATCH + [
    dict(src=None), dict(src=P + 2), dict(src_dtype=3), dict(src_row_stride=-64),
    dict(src_row_stride=68), dict(batch=2, src_batch_stride=257)], ids=str)
def test_quantize_refuses(k):
    assert quant(**k) == B.EINVAL


@pytest.mark.parametrize("k", BAD_BATCH + [
    dict(dst=None), dict(dst=P + 2), dict(dst_dtype=3), dict(dst_row_stride=68),
    dict(dst_row_stride=56), dict(batch=2, dst_batch_stride=248)], ids=str)
def test_dequantize_refuses(k):
    assert dequant(**k) == B.EINVAL


@pytest.mark.parametrize("k", [
    dict(batch=2, dst_row_stride=512, dst_batch_stride=0), dict(batch=2, rows=1, dst_batch_stride=0),
    dict(batch=2, rows=1, dst_batch_stride=56), dict(batch=3, dst_row_stride=128, dst_batch_stride=64)],
    ids=str)
def test_dequantize_refuses_matrices_that_overlap(k):
    assert dequant(**k) == B.EINVAL


def test_tile_scales_refuses_planes_past_memory():
    assert sm.moe_mx_tile_scales(P, (1 << 31) - 1, 1 << 30, P, stream=0, check=False) == B.EINVAL


def test_tile_scales_refuses():
    for a in ((P, -1, 64, P), (P, 4, 48, P), (None, 4, 64, P), (P, 4, 64, None), (P, 4, 64, P + 8)):
        assert sm.moe_mx_tile_scales(*a, stream=0, check=False) == B.EINVAL


def pack(**k):
    a = dict(gate=P, up=P, down=P, dtype=sm.DTYPE_BF16, row_strides=(256, 256, 128),
             expert_strides=(1 << 15,) * 3, E=2, H=256, I=128, blobs=P, blob_stride=1 << 20)
    a.update(k)
    return sm.moe_mx_pack_experts(**a, stream=0, check=False)


def unpack(**k):
    a = dict(blobs=P, blob_stride=1 << 20, E=2, H=256, I=128, gate=P, up=P, down=P,
             dtype=sm.DTYPE_BF16)
    a.update(k)
    return sm.moe_mx_unpack_experts(**a, stream=0, check=False)


BAD_EXPERTS = [dict(gate=None), dict(up=P + 2), dict(down=None), dict(dtype=5), dict(E=-1), dict(H=192),
               dict(I=0), dict(blobs=None), dict(blobs=P + 128), dict(blob_stride=(1 << 20) + 64),
               dict(blob_stride=256)]


@pytest.mark.parametrize("k", BAD_EXPERTS + [
    dict(row_strides=None), dict(expert_strides=None), dict(row_strides=(260, 256, 128)),
    dict(row_strides=(256, -256, 128)), dict(expert_strides=(1 << 15, 1 << 15, 9))], ids=str)
def test_pack_experts_refuses(k):
    assert pack(**k) == B.EINVAL


@pytest.mark.parametrize("k", BAD_EXPERTS, ids=str)
def test_unpack_experts_refuses(k):
    assert unpack(**k) == B.EINVAL


def norm(**k):
    a = dict(x=P, x_dtype=0, delta=P, delta_dtype=2, gain=P, T=4, H=64, eps=1e-6, residual_out=P,
             out=P, out_dtype=2, mx_fmt=sm.MX_FP8, codes=P, scales=P, scale_layout=sm.MX_TILES)
    a.update(k)
    return sm.moe_add_rmsnorm(**a, stream=0, check=False)


@pytest.mark.parametrize("k", [
    dict(x=None), dict(x=P + 8), dict(x_dtype=3), dict(delta_dtype=-1), dict(delta=P + 4),
    dict(gain=P + 4), dict(T=-1), dict(H=24), dict(H=16392), dict(H=68), dict(H=72),
    dict(eps=-1.0), dict(eps=float("nan")), dict(residual_out=P + 8), dict(out=P + 8),
    dict(out_dtype=7), dict(mx_fmt=3), dict(codes=None), dict(scales=None), dict(codes=P + 8),
    dict(scales=P + 8), dict(scale_layout=5), dict(residual_out=None, out=None, mx_fmt=0)], ids=str)
def test_norm_refuses(k):
    assert norm(**k) == B.EINVAL


def linear(**k):
    a = dict(x_codes=P, x_fmt=sm.MX_FP8, x_scales=P, T=4, w_codes=P, w_fmt=sm.MX_FP4, w_scales=P,
             N=100, K=256, bias=None, y=P, y_dtype=2, ldy=100, dev_status=None)
    a.update(k)
    return sm.moe_mx_linear(**a, stream=0, check=False)


@pytest.mark.parametrize("k", [
    dict(x_fmt=0), dict(w_fmt=3), dict(T=-1), dict(T=(1 << 22) + 1), dict(N=0), dict(N=(1 << 24) + 1),
    dict(K=0), dict(K=192), dict(K=1 << 25), dict(ldy=99), dict(y_dtype=3), dict(x_codes=None),
    dict(x_scales=None), dict(w_codes=None), dict(w_scales=None), dict(y=None),
    dict(x_codes=P + 16), dict(w_codes=P + 16), dict(x_scales=P + 8), dict(w_scales=P + 8),
    dict(y=P + 1), dict(bias=P + 2)], ids=str)
def test_linear_refuses(k):
    assert linear(**k) == B.EINVAL


def test_linear_pair_without_a_kernel():
    assert linear(x_fmt=sm.MX_FP4, w_fmt=sm.MX_FP8) == B.EUNSUPPORTED


def test_empty_is_a_noop():
    assert quant(rows=0, src=None, codes=None, scales=None) == B.OK
    assert quant(batch=0, src=None, codes=None, scales=None) == B.OK
    assert dequant(rows=0, dst=None, codes=None, scales=None) == B.OK
    assert sm.moe_mx_tile_scales(None, 0, 64, None, stream=0, check=False) == B.OK
    assert pack(E=0, gate=None, blobs=None) == B.OK
    assert unpack(E=0, gate=None, blobs=None) == B.OK
    assert norm(T=0, x=None) == B.OK
    assert linear(T=0, x_codes=None, y=None) == B.OK


def test_torch_level_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sm.mx_quantize(x, sm.MX_FP8)
    with pytest.raises(ValueError, match="CUDA"):
        sm.add_rmsnorm(x, fmt=sm.MX_FP8)
    with pytest.raises(TypeError):
        sm.mx_quantize(x.double(), sm.MX_FP8)
    with pytest.raises(ValueError, match="rows"):
        sm.mx_quantize(torch.zeros(64, 4).T, sm.MX_FP8)
    with pytest.raises(ValueError, match="16-byte"):
        sm.mx_quantize(torch.zeros(4, 66)[:, :64], sm.MX_FP8)
    with pytest.raises(ValueError, match="matrix"):
        sm.mx_quantize(torch.zeros(2, 4, 64), sm.MX_FP8)
    with pytest.raises(ValueError, match="multiple of 32"):
        sm.mx_quantize(torch.zeros(4, 48), sm.MX_FP8)
    with pytest.raises(ValueError, match="out_dtype"):
        sm.add_rmsnorm(x)
    with pytest.raises(ValueError, match="delta"):
        sm.add_rmsnorm(x, torch.zeros(4, 32), fmt=sm.MX_FP8)
    with pytest.raises(ValueError, match="gain"):
        sm.add_rmsnorm(x, gain=torch.ones(64).bfloat16(), fmt=sm.MX_FP8)
    with pytest.raises(TypeError, match="residual_out"):
        sm.add_rmsnorm(x, fmt=sm.MX_FP8, residual_out=x.bfloat16())
    c, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    q = sm.MXTensor(c, s, sm.MX_FP8, 4, 128, sm.MX_ROWS)
    with pytest.raises(ValueError, match="tiles"):
        sm.mx_linear(q, q)
    with pytest.raises(ValueError, match="K = "):
        sm.mx_linear(q, sm.MXTensor(c[:, :64].contiguous(), s[:, :2].contiguous(), sm.MX_FP8, 4, 64, sm.MX_ROWS))
    for bad in ((c, s, 3, 4, 128, 0), (c, s, 2, 4, 128, 2), (c, s, 2, 4, 120, 0), (c, s, 1, 4, 128, 0),
                (c, s, 2, 4, 128, 1), (c.int(), s, 2, 4, 128, 0), (c, s, 2, 5, 128, 0)):
        with pytest.raises(ValueError):
            sm.MXTensor(*bad)
    w = torch.zeros(2, 128, 256)
    with pytest.raises(ValueError, match="CUDA"):
        sm.pack_experts(w, w, torch.zeros(2, 256, 128))
    with pytest.raises(ValueError, match="down"):
        sm.pack_experts(w, w, w)
    with pytest.raises(ValueError, match="gate"):
        sm.pack_experts(w, w[:1], w)
    e = sm.ExpertWeights(torch.zeros(2, 1 << 17, dtype=torch.uint8), sm.FMT_Q2_32, 256, 128)
    with pytest.raises(ValueError, match="MXFP4"):
        e.dequantize()


# ---------------------------------------------------------------- a matrix's memory
HELD = """
import copy, io, pickle, sys
if {plain}:
    sys.modules["expert_ffn_execution_b200._mxcalls"] = None
import torch
import expert_ffn_execution_b200 as sm
from expert_ffn_execution_b200 import mx
assert (mx._mxcalls is None) == {plain}


def make():
    c = torch.randint(0, 256, (4, 64), dtype=torch.uint8)
    s = torch.randint(0, 256, (4, 4), dtype=torch.uint8)
    return sm.MXTensor(c, s, sm.MX_FP4, 4, 128, sm.MX_ROWS)


def whole(q):
    assert q.codes_ptr == q.codes.data_ptr() and q.scales_ptr == q.scales.data_ptr()
    assert (q.fmt, q.layout, q.rows, q.K, q.index, q.device.type) == (sm.MX_FP4, sm.MX_ROWS, 4, 128, -1, "cpu")


def refuses(error, f, *a):
    try:
        f(*a)
    except error:
        return
    raise AssertionError("not refused")


both = sm.MXTensor._empty(sm.MX_FP4, 4, 128, sm.MX_ROWS, torch.device("cpu"))
assert both.scales_ptr == both.codes_ptr + 256
both.codes.copy_(torch.arange(256).view(4, 64) % 251)
both.scales.fill_(120)
for q in (make(), both):
    whole(q)
    f = io.BytesIO()
    torch.save(q, f)
    f.seek(0)
    for r in (copy.deepcopy(q), pickle.loads(pickle.dumps(q)), torch.load(f, weights_only=False)):
        whole(r)
        assert torch.equal(r.codes, q.codes) and torch.equal(r.scales, q.scales)
        assert r.codes_ptr != q.codes_ptr and r.scales_ptr != q.scales_ptr
    r = copy.copy(q)
    whole(r)
    assert r.codes is q.codes and r.scales is q.scales
    # other memory of the same form is followed, another form refused
    q.codes.data = torch.zeros(4, 64, dtype=torch.uint8)
    q.scales.data = torch.zeros(4, 4, dtype=torch.uint8)
    whole(q)
    for t, bad in ((q.codes, torch.zeros(3, 64, dtype=torch.uint8)), (q.scales, torch.zeros(4, 4)),
                   (q.codes, torch.zeros(4, 128, dtype=torch.uint8)[:, ::2])):
        kept = t.data
        t.data = bad
        refuses(ValueError, mx._planes, q)
        t.data = kept
        whole(q)
    for n in ("fmt", "layout", "rows", "K"):
        refuses(AttributeError, setattr, q, n, 1000)
    whole(q)
"""


@pytest.mark.parametrize("plain", [False, True])
def test_matrix_follows_its_tensors(plain):
    """Copied, saved, given other memory: a matrix's addresses are those of its
    tensors, with the native fields and without."""
    if not plain:
        pytest.importorskip("expert_ffn_execution_b200._mxcalls")
    r = subprocess.run([sys.executable, "-c", HELD.format(plain=plain)], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


# ---------------------------------------------------------------- the native module's build
@pytest.mark.parametrize("missing", ["compiler", "torch"])
def test_library_is_built_where_the_native_module_is_not(monkeypatch, tmp_path, missing):
    """No compiler for it, no torch: a warning, the library all the same, and
    no module of other sources left behind."""
    from expert_ffn_execution_b200 import build
    calls = tmp_path / "_mxcalls.so"
    calls.write_bytes(b"old")
    monkeypatch.setattr(build, "CALLS", str(calls))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    os.utime(calls, (0, 0))
    if missing == "compiler":
        monkeypatch.setenv("CXX", "/bin/false")
    else:
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(UserWarning, match="_mxcalls was not built"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not calls.exists()


def test_native_module_is_this_interpreters(monkeypatch, tmp_path):
    """Named so that no other interpreter imports it; one under the name that
    any would import goes."""
    import importlib.machinery
    from expert_ffn_execution_b200 import build
    assert os.path.basename(build.CALLS) == "_mxcalls" + importlib.machinery.EXTENSION_SUFFIXES[0]
    (tmp_path / "_mxcalls.so").write_bytes(b"old")
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "build_calls", lambda force: "built")
    assert build.try_build_calls() == "built"
    assert not (tmp_path / "_mxcalls.so").exists()


def test_negated_views_are_refused():
    """The calls read memory, and a lazily negated view is not what its memory holds."""
    x = torch.zeros(4, 64)
    n = torch._neg_view(x)
    w, d = torch.zeros(2, 128, 256), torch.zeros(2, 256, 128)
    q = sm.MXTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), sm.MX_FP8, 4, 128,
                    sm.MX_TILES)
    r = sm.MXTensor(q.codes[:1], q.scales, sm.MX_FP8, 1, 128, sm.MX_TILES)
    bias = torch.zeros(1, dtype=torch.complex64).conj().imag
    assert bias.is_neg() and bias.is_contiguous()
    for call in (lambda: sm.mx_quantize(n, sm.MX_FP8), lambda: sm.add_rmsnorm(n, fmt=sm.MX_FP8),
                 lambda: sm.add_rmsnorm(x, n, fmt=sm.MX_FP8), lambda: sm.mx_linear(q, r, bias),
                 lambda: sm.mx_linear(q, q, out=torch._neg_view(x[:, :4].contiguous())),
                 lambda: sm.pack_experts(w, torch._neg_view(w), d)):
        with pytest.raises(ValueError, match="negates"):
            call()
