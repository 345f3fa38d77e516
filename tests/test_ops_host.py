"""CPU: what the operators on quantised weights refuse, before anything reaches a GPU, and the 64-bit reference
forms of their tests against torch's own conversions."""
import ctypes as C

import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from device_checkpoint_dequantisation_amd import _lib
from tests import ops_reference as ref

KINDS = ("FP8_TENSOR", "FP8_BLOCK128", "NVFP4", "MXFP8", "MXFP4")
P = 0x10000     # a well-aligned address that is never followed


def _weight(kind="FP8_TENSOR", n=64, k=128):
    return ref.random_weight(st, kind, n, k, 1)


def _x(m=4, k=128, dtype=torch.bfloat16):
    return torch.zeros(m, k, dtype=dtype)


@pytest.mark.parametrize("kind", KINDS)
def test_linear_needs_a_gpu(kind):
    with pytest.raises(ValueError, match="GPU"):
        st.linear(_x(), _weight(kind))
    with pytest.raises(ValueError, match="GPU"):
        st.rms_norm(_x())
    with pytest.raises(ValueError, match="GPU"):
        st.quantize_activation(_x(), "MXFP8")


def test_linear_refuses_weights_that_are_not_what_they_say():
    for kind in KINDS:
        w = _weight(kind)
        for field in ("data", "scale"):
            good = getattr(w, field)
            if good.numel() > 1:
                setattr(w, field, good[:1])
                with pytest.raises(ValueError, match="holds|scale"):
                    st.linear(_x(), w)
            setattr(w, field, torch.zeros(good.shape, dtype=torch.int8))
            with pytest.raises(ValueError, match="holds|scale"):
                st.linear(_x(), w)
            setattr(w, field, good)
    w = _weight("NVFP4")
    w.scale2 = None
    with pytest.raises(ValueError, match="global scale"):
        st.linear(_x(), w)
    w = _weight()
    w.data = w.data.t().contiguous().t()
    with pytest.raises(ValueError, match="strides"):
        st.linear(_x(), w)
    w = _weight()
    w.shape, w.data = (64, 8, 16), w.data.view(64, 8, 16)
    with pytest.raises(ValueError, match="matrix"):
        st.linear(_x(), w)
    w = _weight()
    w.kind = "PASS_BF16"
    with pytest.raises(ValueError, match="not a quantised kind"):
        st.linear(_x(), w)


def test_linear_refuses_rows_that_do_not_fit():
    with pytest.raises(ValueError, match="against a weight"):
        st.linear(_x(k=127), _weight())
    with pytest.raises(ValueError, match="bf16, fp16"):
        st.linear(_x(dtype=torch.float32), _weight())
    for xk, wk in (("FP8_ROW", "NVFP4"), ("FP8_ROW", "FP8_BLOCK128"), ("MXFP8", "FP8_TENSOR"), ("FP8_GROUP128", "MXFP8"), ("MXFP8", "NVFP4")):
        with pytest.raises(ValueError, match="do not go with"):
            st.linear(ref.random_rows(st, xk, 4, 128, 2), _weight(wk))
    q = ref.random_rows(st, "FP8_GROUP128", 4, 128, 2)
    q.scale = q.scale[:3]
    with pytest.raises(ValueError, match="scales"):
        st.linear(q, _weight("FP8_BLOCK128"))


def test_linear_and_norm_refuse_grad():
    from device_checkpoint_dequantisation_amd import ops
    dev = type("Device", (), {"type": "cuda"})()      # stands in for a GPU: the check comes with the device check
    x2 = type("T", (), {"device": dev, "requires_grad": True})()
    with pytest.raises(RuntimeError, match="no backward"):
        ops._on_device(dev, (None, x2), "linear")
    with torch.no_grad():
        ops._on_device(dev, (None, x2), "linear")


def test_encode_and_norm_refusals():
    with pytest.raises(ValueError, match="unknown encoding"):
        st.quantize_activation(_x(), "FP8")
    with pytest.raises(ValueError, match="multiple of 32"):
        st.quantize_activation(_x(k=100), "MXFP8")
    with pytest.raises(ValueError, match="rows are needed"):
        st.quantize_activation(torch.zeros(4, 4, dtype=torch.int32), "FP8_ROW")
    with pytest.raises(ValueError):
        st.rms_norm(torch.tensor(1.0))


def _linear_args(**kw):
    base = dict(x=P, x_scale=None, w=P, w_scale=P, w_scale2=None, bias=None, residual=None, out=P, workspace=None,
                workspace_bytes=0, m=4, n=64, k=128, x_pitch=128, residual_pitch=0, out_pitch=64, x_type=0, w_kind=3,
                activation=0, bias_type=0, residual_type=0, out_type=0)
    base.update(kw)
    return _lib.LinearArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(x_type=5), -1), (dict(w_kind=2), -1), (dict(w_kind=8), -1), (dict(activation=5), -1), (dict(out_type=3), -1),
    (dict(bias_type=3), -1), (dict(x_type=2, w_kind=5), -1), (dict(x_type=4, w_kind=3), -1), (dict(m=1 << 31), -6),
    (dict(n=1 << 31), -6), (dict(k=1 << 31), -6), (dict(w_kind=5, k=24), -6), (dict(w_kind=6, k=48), -6), (dict(out=None), -1),
    (dict(out_pitch=63), -6), (dict(x_pitch=127), -6), (dict(x=None), -1), (dict(w=None), -1), (dict(w_scale=None), -1),
    (dict(w_kind=5), -1), (dict(x_type=2), -1), (dict(x=P + 1), -1), (dict(out=P + 1), -1), (dict(w_scale=P + 2), -1),
    (dict(residual=P + 1, residual_pitch=64), -1), (dict(residual=P, residual_pitch=60), -6), (dict(bias=P + 2, bias_type=2), -1)])
def test_linear_abi_refusals(kw, code):
    L = _lib.lib()
    a = _linear_args(**kw)
    assert L.st_linear(C.byref(a), None) == code and L.st_last_error()
    need = C.c_uint64(7)
    assert L.st_linear_workspace_bytes(C.byref(a), C.byref(need)) == code and need.value == 0


def test_linear_abi_workspace_and_empty():
    L = _lib.lib()
    need = C.c_uint64()
    assert L.st_linear(None, None) == -1 and L.st_linear_workspace_bytes(None, C.byref(need)) == -1
    assert L.st_linear_workspace_bytes(C.byref(_linear_args()), None) == -1
    for kw in (dict(m=0), dict(n=0)):
        assert L.st_linear(C.byref(_linear_args(out=None, x=None, w=None, **kw)), None) == 0
    # a long K over a small output is split: a workspace of fp32 partial results, refused where it is missing, short or misaligned
    a = _linear_args(m=100, n=128, k=1 << 20, x_pitch=1 << 20, out_pitch=128)
    assert L.st_linear_workspace_bytes(C.byref(a), C.byref(need)) == 0 and need.value % (100 * 128 * 4) == 0 and need.value
    assert L.st_linear(C.byref(a), None) == -1
    a.workspace, a.workspace_bytes = P, need.value - 1
    assert L.st_linear(C.byref(a), None) == -1
    a.workspace, a.workspace_bytes = P + 8, need.value
    assert L.st_linear(C.byref(a), None) == -1


@pytest.mark.parametrize("kw,code", [(dict(kind=0), -1), (dict(kind=5), -1), (dict(x_type=3), -1), (dict(x=None), -1), (dict(data=None), -1),
                                     (dict(scale=None), -1), (dict(x=P + 1), -1), (dict(gate=P + 1), -1), (dict(scale=P + 2), -1),
                                     (dict(x_pitch=100), -6), (dict(gate=P, gate_pitch=100), -6), (dict(kind=4, d=100), -6), (dict(m=1 << 31), -6),
                                     (dict(d=1 << 31), -6)])
def test_encode_abi_refusals(kw, code):
    base = dict(x=P, gate=None, data=P, scale=P, m=4, d=128, x_pitch=128, gate_pitch=0, x_type=0, kind=2)
    base.update(kw)
    assert _lib.lib().st_encode(C.byref(_lib.EncodeArgs(**base)), None) == code


@pytest.mark.parametrize("kw,code", [(dict(kind=1), -1), (dict(kind=5), -1), (dict(x_type=3), -1), (dict(weight_type=3), -1), (dict(out_type=3), -1),
                                     (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(x=None), -1), (dict(out=None), -1),
                                     (dict(kind=2, scale=None), -1), (dict(h_out=P + 1), -1), (dict(weight=P + 1), -1),
                                     (dict(residual=P, residual_pitch=1), -6), (dict(kind=4, d=100), -6), (dict(m=1 << 31), -6)])
def test_norm_abi_refusals(kw, code):
    base = dict(x=P, residual=None, weight=P, h_out=None, out=P, scale=P, m=4, d=128, x_pitch=128, residual_pitch=0, eps=1e-6,
                x_type=0, weight_type=0, out_type=0, kind=0)
    base.update(kw)
    assert _lib.lib().st_rms_norm(C.byref(_lib.RmsNormArgs(**base)), None) == code
    assert _lib.lib().st_rms_norm(None, None) == -1 and _lib.lib().st_encode(None, None) == -1


def test_reference_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = ref.e4m3(codes.view(torch.float8_e4m3fn))
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
    v = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 100
    assert torch.equal(ref.e4m3_codes(v.double()), v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) & 127)
    e = torch.arange(255, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    assert torch.equal(ref.e8m0(e), e.float().double())


@pytest.mark.parametrize("kw", [dict(m=1, n=1 << 26, k=4096), dict(m=16, n=1 << 27, k=4096), dict(m=16, n=1 << 29, k=4096, w_kind=7),
                                dict(m=20, n=1 << 30, k=128), dict(m=(1 << 31) - 1, n=1, k=128, out_pitch=1)])
def test_linear_refuses_more_threads_than_a_launch_holds(kw):
    """Sizes whose grid would hold 2^32 threads are refused before anything is launched."""
    L = _lib.lib()
    a = _linear_args(**{"x_pitch": kw["k"], "out_pitch": kw["n"], **kw})
    need = C.c_uint64(7)
    assert L.st_linear(C.byref(a), None) == -6 and b"threads" in L.st_last_error()
    assert L.st_linear_workspace_bytes(C.byref(a), C.byref(need)) == -6 and need.value == 0
    a.n = a.out_pitch = kw["n"] - 512 if kw["n"] > 512 else 1
    a.m = kw["m"] if kw["n"] > 512 else kw["m"] - 256
    assert L.st_linear_workspace_bytes(C.byref(a), C.byref(need)) == 0


def test_operators_refuse_forward_mode_tangents(monkeypatch):
    """A dual tensor does not require grad; its tangent would be lost without a word."""
    import torch.autograd.forward_ad as fwd
    from device_checkpoint_dequantisation_amd import ops
    check = ops._on_device                 # CPU tensors are refused for their device: let them pass as GPU ones
    gpu = type("Device", (), {"type": "cuda", "__eq__": lambda a, b: True, "__ne__": lambda a, b: False})()
    monkeypatch.setattr(ops, "_on_device", lambda device, tensors, who: check(gpu, tensors, who))

    def dual(*shape, dtype=torch.bfloat16):
        return fwd.make_dual(torch.zeros(shape, dtype=dtype), torch.ones(shape, dtype=dtype))
    with fwd.dual_level():
        x, w = _x(), _weight()
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                for call in (lambda: st.linear(dual(4, 128), w), lambda: st.linear(dual(4, 128)[:2], w),
                             lambda: st.linear(x, w, bias=dual(64)), lambda: st.linear(x, w, residual=dual(4, 64)),
                             lambda: st.rms_norm(dual(4, 128)), lambda: st.rms_norm(x, dual(128, dtype=torch.float32)),
                             lambda: st.rms_norm(x, residual=dual(4, 128)), lambda: st.quantize_activation(dual(4, 128), "MXFP8"),
                             lambda: st.quantize_activation(x, "MXFP8", gate=dual(4, 128))):
                    with pytest.raises(RuntimeError, match="tangent"):
                        call()
        ops._on_device(gpu, (None, x, w.data, w.scale, _weight("MXFP8").scale), "linear")


def test_rows_of_any_layout_are_made_adjacent_whatever_the_batch():
    """[..., K] inputs whose elements are not adjacent are copied for one image as for two; a matrix of such rows is refused."""
    from device_checkpoint_dequantisation_amd import ops
    for batch in (1, 2):
        image = torch.randn(batch, 6, 2, 5)                        # [B, K, H, W], the usual patch embedding
        t = image.flatten(2).transpose(1, 2)
        rows, pitch = ops._rows(t, 6, "x", "linear")
        assert rows.stride(1) == 1 and pitch == rows.stride(0) >= 6 and torch.equal(rows, t.reshape(-1, 6))
        windows = torch.arange(20.0).unfold(0, 6, 2)[None].expand(batch, 8, 6)      # rows that overlap
        rows, pitch = ops._rows(windows, 6, "x", "linear")
        assert pitch >= 6 and torch.equal(rows, windows.reshape(-1, 6))
        row = torch.randn(6)
        rows, pitch = ops._rows(row.expand(batch, 3, 6), 6, "residual", "linear")
        assert torch.equal(rows, row.expand(3 * batch, 6)) and pitch in (0, 6)
    rows, pitch = ops._rows(torch.arange(12.0)[::2], 6, "x", "linear")
    assert rows.shape == (1, 6) and rows.stride(1) == 1
    t = torch.randn(4, 3, 6)                                       # adjacent already: no copy
    assert ops._rows(t, 6, "x", "linear")[0].data_ptr() == t.data_ptr()
    with pytest.raises(ValueError, match="stride 1"):
        ops._rows(torch.randn(6, 4).t(), 6, "x", "linear")


def test_importing_the_package_leaves_torch_alone():
    """The header side of the package works without torch: neither an import nor a star import brings it in, and the
    operators are there on first use."""
    import subprocess
    import sys
    code = ("import sys\nimport device_checkpoint_dequantisation_amd as st\nfrom device_checkpoint_dequantisation_amd import *\n"
            "assert 'torch' not in sys.modules and SafeTensorIndex is st.SafeTensorIndex\n"
            "assert st.linear.__module__.endswith('.ops') and 'torch' in sys.modules\n"
            "from device_checkpoint_dequantisation_amd import QuantizedActivation, quantize_activation, rms_norm\n")
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr


def test_overlap_of_columns_of_one_buffer():
    """Columns of one buffer lie between each other without overlapping; what shares a byte does."""
    from device_checkpoint_dequantisation_amd import ops
    buf = torch.zeros(7, 40)
    cols = lambda a, b, rows=slice(None): buf[rows, a:b]   # noqa: E731
    for out, t, want in ((cols(0, 16), cols(16, 40), False), (cols(16, 40), cols(0, 16), False), (cols(0, 16), cols(15, 20), True),
                         (cols(0, 16), cols(0, 16), True), (cols(10, 20), cols(20, 30, slice(2, 5)), False),
                         (cols(10, 20, slice(0, 3)), cols(12, 14, slice(3, 7)), False), (cols(30, 40), cols(0, 1), False),
                         (cols(10, 20), cols(0, 40), True), (cols(0, 16), cols(16, 40).view(torch.int32), False),
                         (cols(0, 16), buf[3, 4:9], True), (cols(0, 16), buf[3, 20:29], True),      # (a row: by its span)
                         (cols(0, 16), torch.zeros(7, 16), False), (cols(0, 16), None, False), (cols(0, 16), buf[:0], False)):
        assert ops._overlaps(out, t) == want, (out.storage_offset(), None if t is None else (t.shape, t.storage_offset()))
    assert ops._overlaps(cols(0, 20), buf.view(torch.bfloat16)[:, 36:44]) and not ops._overlaps(cols(0, 20), buf.view(torch.bfloat16)[:, 40:44])
