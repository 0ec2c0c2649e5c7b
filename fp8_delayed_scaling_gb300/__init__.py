"""Python binding of libfp8dl — the GB300 (sm_103a) FP8 delayed-scaling linear layer.

Argument marshalling only: every function here forwards device pointers and
sizes to the C ABI declared in ``include/fp8dl.h`` (same names), and every step
of the computation runs in the library's CUDA kernels.  There is no CPU
fallback: if ``libfp8dl.so`` is missing the import fails, and on a machine
without an sm_103 GPU the calls return FP8DL_ERR_UNSUPPORTED_DEVICE.

PyTorch is used for device memory and streams only.  Pointer arguments accept a
``torch.Tensor`` (its ``data_ptr()``), a plain integer device address, or None.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8dl.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libfp8dl.so is not built (%s); run `python -c 'import __graft_entry__ as g; g.build()'`"
                      % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

# enums (include/fp8dl.h)
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED_DEVICE, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(8)
E4M3, E5M2 = 0, 1
F32, BF16 = 0, 1
FORMAT_E4M3, FORMAT_HYBRID = 0, 1
FP8_MAX = {E4M3: 448.0, E5M2: 57344.0}

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class fp8dl_recipe(ctypes.Structure):
    _fields_ = [("margin", _i32), ("interval", _i32), ("fp8_format", _i32), ("amax_history_len", _i32),
                ("amax_compute_algo", _i32)]


class fp8dl_cast_item(ctypes.Structure):
    """One tensor of fp8_cast_amax_transpose_multi (include/fp8dl.h)."""
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_t", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("scale_inv_out", ctypes.c_void_p)]


_SIGS = {
    "fp8dl_slot_stride": (_sz, [_i32]),
    "fp8dl_scaling_state_bytes": (_sz, [_i32, _i32]),
    "fp8_scaling_state_init": (_i32, [ctypes.POINTER(fp8dl_recipe), _i32, _vp, _vp, _vp]),
    "fp8_update_scale": (_i32, [ctypes.POINTER(fp8dl_recipe), _i32, _vp, _i64, _vp]),
    "fp8_seed_amax_history": (_i32, [ctypes.POINTER(fp8dl_recipe), _i32, _vp, _vp]),
    "fp8_cast_workspace_size": (_sz, [_i64, _i64]),
    "fp8_cast_amax_transpose": (_i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fp8_cast_amax_transpose_noalloc": (_i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fp8_cast_amax_transpose_multi": (_i32, [_i32, ctypes.POINTER(fp8dl_cast_item), _i32, _i32, _vp]),
    "fp8_gemm": (_i32, [_vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp]),
    "fp8_gemm_gelu_cast": (_i32, [_vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp]),
    "fp8_gemm_dgelu_workspace_size": (_sz, [_i64, _i64]),
    "fp8_gemm_dgelu_cast": (_i32, [_vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _sz, _vp, _vp, _vp]),
    "mxfp8_scale_bytes": (_sz, [_i64, _i64]),
    "mxfp8_quantize": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mxfp8_gemm": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp]),
    "fp8_block_padded_rows": (_i64, [_i64, _i32]),
    "fp8_block_quantize": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fp8_block_quantize_weight": (_i32, [_vp, _i32, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp]),
    "fp8_block_gemm": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _vp,
                              _vp]),
    "fp8_block_gemm_plan": (_i32, [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "fp8_block_gemm_grouped": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp,
                                      _vp]),
    "fp8_block_gemm_grouped_wgrad": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32,
                                            _vp, _vp]),
    "fp8_layernorm_cast": (_i32, [_vp, _i64, _i64, _vp, _vp, ctypes.c_float, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp]),
    "fp8_gelu_cast": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fp8_dgelu_cast": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "fp8_layernorm_bwd_workspace_size": (_sz, [_i64, _i64]),
    "fp8_layernorm_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fp8dl_wait_selftest": (_i32, [_i64, _i32, _vp, _vp]),
    "fp8dl_device_supported": (_i32, [_i32]),
    "fp8dl_clock_probe": (_i32, [_vp, _i32, _vp]),
    "fp8dl_last_error": (ctypes.c_char_p, []),
    "fp8dl_version": (_i32, []),
    "fp8dl_kernel_launches": (ctypes.c_uint64, []),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class FP8DLError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed with status %d: %s" % (where, status, fp8dl_last_error()))


def _check(status: int, where: str) -> None:
    if status != OK:
        raise FP8DLError(status, where)


def _p(x):
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _hp(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


# --------------------------------------------------------------------------
# library state
# --------------------------------------------------------------------------
def fp8dl_last_error() -> str:
    return _lib.fp8dl_last_error().decode()


def fp8dl_version() -> int:
    return _lib.fp8dl_version()


def fp8dl_kernel_launches() -> int:
    """Kernels the library has enqueued in this process (graph replays not included)."""
    return _lib.fp8dl_kernel_launches()


def fp8dl_device_supported(device: int = 0) -> bool:
    return bool(_lib.fp8dl_device_supported(device))


def fp8dl_clock_probe(out, n_ctas: int, stream=None) -> None:
    """out: uint64 device tensor of 3 * n_ctas entries (SM id, cycle counter, ns timer per CTA)."""
    _check(_lib.fp8dl_clock_probe(_p(out), int(n_ctas), _stream(stream)), "fp8dl_clock_probe")


def fp8dl_wait_selftest(budget_cycles: int, arrive_first: bool, dev_status, stream=None) -> None:
    """Run the bounded-wait self-test; the outcome is written to dev_status (device int32)."""
    _check(_lib.fp8dl_wait_selftest(int(budget_cycles), 1 if arrive_first else 0, _p(dev_status), _stream(stream)),
           "fp8dl_wait_selftest")


def fp8dl_slot_stride(amax_history_len: int) -> int:
    return _lib.fp8dl_slot_stride(amax_history_len)


def fp8dl_scaling_state_bytes(amax_history_len: int, n_slots: int) -> int:
    return _lib.fp8dl_scaling_state_bytes(amax_history_len, n_slots)


def fp8_cast_workspace_size(rows: int, cols: int) -> int:
    return _lib.fp8_cast_workspace_size(rows, cols)


# --------------------------------------------------------------------------
# recipe + scaling state
# --------------------------------------------------------------------------
@dataclass
class Recipe:
    """DelayedScaling recipe: margin, interval, fp8_format, amax_history_len, "max"."""
    margin: int = 0
    interval: int = 1
    fp8_format: int = FORMAT_HYBRID
    amax_history_len: int = 16
    amax_compute_algo: int = 0

    def c(self) -> fp8dl_recipe:
        return fp8dl_recipe(self.margin, self.interval, self.fp8_format, self.amax_history_len,
                            self.amax_compute_algo)

    def fwd_dtype(self) -> int:
        return E4M3

    def bwd_dtype(self) -> int:
        return E5M2 if self.fp8_format == FORMAT_HYBRID else E4M3


def fp8_scaling_state_init(recipe: Recipe, slot_fp8_dtype, state, stream=None) -> None:
    n = len(slot_fp8_dtype)
    arr = (ctypes.c_int32 * n)(*[int(d) for d in slot_fp8_dtype])
    r = recipe.c()
    _check(_lib.fp8_scaling_state_init(ctypes.byref(r), n, ctypes.cast(arr, _vp), _p(state), _stream(stream)),
           "fp8_scaling_state_init")


def fp8_update_scale(recipe: Recipe, n_slots: int, state, step: int, stream=None) -> None:
    r = recipe.c()
    _check(_lib.fp8_update_scale(ctypes.byref(r), n_slots, _p(state), int(step), _stream(stream)),
           "fp8_update_scale")


def fp8_seed_amax_history(recipe: Recipe, n_slots: int, state, stream=None) -> None:
    r = recipe.c()
    _check(_lib.fp8_seed_amax_history(ctypes.byref(r), n_slots, _p(state), _stream(stream)),
           "fp8_seed_amax_history")


class ScalingState:
    """Device block holding the delayed-scaling state of `len(slot_fp8_dtype)` tensors."""

    def __init__(self, recipe: Recipe, slot_fp8_dtype, device="cuda", stream=None):
        self.recipe = recipe
        self.slot_fp8_dtype = [int(d) for d in slot_fp8_dtype]
        self.n_slots = len(self.slot_fp8_dtype)
        self.stride = fp8dl_slot_stride(recipe.amax_history_len)
        self.buf = torch.empty(fp8dl_scaling_state_bytes(recipe.amax_history_len, self.n_slots),
                               dtype=torch.uint8, device=device)
        fp8_scaling_state_init(recipe, self.slot_fp8_dtype, self.buf, stream)

    def _addr(self, slot: int, off: int) -> int:
        assert 0 <= slot < self.n_slots
        return self.buf.data_ptr() + slot * self.stride + off

    def scale(self, slot: int) -> int:
        return self._addr(slot, 0)

    def scale_inv(self, slot: int) -> int:
        return self._addr(slot, 4)

    def amax(self, slot: int) -> int:
        return self._addr(slot, 8)

    def update(self, step: int, stream=None) -> None:
        fp8_update_scale(self.recipe, self.n_slots, self.buf, step, stream)

    def seed(self, stream=None) -> None:
        fp8_seed_amax_history(self.recipe, self.n_slots, self.buf, stream)

    def read(self) -> dict:
        """Host copy of every slot's fields (synchronises)."""
        raw = self.buf.cpu()
        L = self.recipe.amax_history_len
        rows = raw.view(self.n_slots, self.stride)
        hdr = rows[:, :32].contiguous()
        f = hdr.view(torch.float32)
        i = hdr.view(torch.int32)
        hist = rows[:, 32:32 + 4 * L].contiguous().view(torch.float32)
        return {"scale": f[:, 0].numpy().copy(), "scale_inv": f[:, 1].numpy().copy(),
                "amax": f[:, 2].numpy().copy(), "pos": i[:, 3].numpy().copy(),
                "fp8_dtype": i[:, 4].numpy().copy(), "hist": hist.numpy().copy()}


# --------------------------------------------------------------------------
# kernels
# --------------------------------------------------------------------------
def fp8_cast_amax_transpose(x: torch.Tensor, out_dtype: int, scale, out=None, out_t=None, amax=None, dbias=None,
                            workspace=None, scale_inv_out=None, stream=None) -> None:
    assert x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    ws_bytes = workspace.numel() * workspace.element_size() if isinstance(workspace, torch.Tensor) else 0
    _check(_lib.fp8_cast_amax_transpose(_p(x), _hp(x), rows, cols, out_dtype, _p(scale), _p(out), _p(out_t),
                                        _p(amax), _p(scale_inv_out), _p(dbias), _p(workspace), ws_bytes,
                                        _stream(stream)),
           "fp8_cast_amax_transpose")


def fp8_cast_amax_transpose_multi(items, out_dtype: int, stream=None) -> None:
    """Grouped cast: items is a list of dicts with keys x, scale, and any of out, out_t, amax,
    scale_inv_out (as for fp8_cast_amax_transpose, without dbias); one launch for all."""
    n = len(items)
    arr = (fp8dl_cast_item * n)()
    x_dtype = None
    for k, it in enumerate(items):
        x = it["x"]
        assert x.dim() == 2 and x.is_contiguous()
        if x_dtype is None:
            x_dtype = _hp(x)
        assert _hp(x) == x_dtype, "all items share one input dtype"
        arr[k] = fp8dl_cast_item(_p(x), x.shape[0], x.shape[1], _p(it.get("scale")), _p(it.get("out")),
                                 _p(it.get("out_t")), _p(it.get("amax")), _p(it.get("scale_inv_out")))
    _check(_lib.fp8_cast_amax_transpose_multi(n, arr, x_dtype if x_dtype is not None else BF16, out_dtype,
                                              _stream(stream)), "fp8_cast_amax_transpose_multi")


def fp8_cast_amax_transpose_noalloc(x: torch.Tensor, out_dtype: int, scale, out=None, out_t=None, amax=None,
                                    dbias=None, stream=None) -> None:
    """fp8_cast_amax_transpose for callers that cannot allocate device memory:
    the bias-gradient scratch is the library's own 4 MiB static device array
    (ceil(rows/128) * cols * 4 bytes must fit).  Calls on one device share
    that array, so concurrent calls must be ordered on one stream."""
    assert x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    _check(_lib.fp8_cast_amax_transpose_noalloc(_p(x), _hp(x), rows, cols, out_dtype, _p(scale), _p(out),
                                                _p(out_t), _p(amax), _p(dbias), _stream(stream)),
           "fp8_cast_amax_transpose_noalloc")


def fp8_gemm(A: torch.Tensor, a_dtype: int, B: torch.Tensor, b_dtype: int, a_scale_inv, b_scale_inv, D: torch.Tensor,
             bias: torch.Tensor | None = None, dev_status=None, stream=None) -> None:
    """D[M,N] = (A[M,K] * B[N,K]^T) * a_scale_inv * b_scale_inv + bias."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and tuple(D.shape) == (M, N)
    _check(_lib.fp8_gemm(_p(A), a_dtype, _p(B), b_dtype, M, N, K, _p(a_scale_inv), _p(b_scale_inv), _p(bias),
                         _hp(bias) if bias is not None else BF16, _p(D), _hp(D), _p(dev_status), _stream(stream)),
           "fp8_gemm")


def fp8_gemm_gelu_cast(A: torch.Tensor, a_dtype: int, B: torch.Tensor, b_dtype: int, a_scale_inv, b_scale_inv,
                       H: torch.Tensor, q_dtype: int, q_scale, q: torch.Tensor, q_t: torch.Tensor, q_amax=None,
                       bias: torch.Tensor | None = None, g=None, dev_status=None, stream=None) -> None:
    """H = A*B^T*sa_inv*sb_inv + bias (bf16); q, q^T = FP8 codes of GELU(H) at q_scale; amax of GELU(H)."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and tuple(H.shape) == (M, N) and H.dtype == torch.bfloat16
    _check(_lib.fp8_gemm_gelu_cast(_p(A), a_dtype, _p(B), b_dtype, M, N, K, _p(a_scale_inv), _p(b_scale_inv), _p(bias),
                                   _hp(bias) if bias is not None else BF16, _p(H), q_dtype, _p(q_scale), _p(q), _p(q_t),
                                   _p(q_amax), _p(g), _p(dev_status), _stream(stream)), "fp8_gemm_gelu_cast")


def fp8_gemm_dgelu_workspace_size(M: int, N: int) -> int:
    return _lib.fp8_gemm_dgelu_workspace_size(M, N)


def fp8_gemm_dgelu_cast(A: torch.Tensor, a_dtype: int, B: torch.Tensor, b_dtype: int, a_scale_inv, b_scale_inv,
                        h: torch.Tensor, q_dtype: int, q_scale, q: torch.Tensor, q_t: torch.Tensor, q_amax=None,
                        dbias=None, workspace=None, dg=None, dh=None, dev_status=None, stream=None) -> None:
    """dg = A*B^T*sa_inv*sb_inv (bf16, not stored unless dg is given); q, q^T = FP8 codes of
    dh = bf16(dg * GELU'(h)) at q_scale; amax |dh|; dbias = column sums of dh."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and tuple(h.shape) == (M, N) and h.dtype == torch.bfloat16
    ws_bytes = workspace.numel() * workspace.element_size() if isinstance(workspace, torch.Tensor) else 0
    _check(_lib.fp8_gemm_dgelu_cast(_p(A), a_dtype, _p(B), b_dtype, M, N, K, _p(a_scale_inv), _p(b_scale_inv), _p(h),
                                    _p(dg), q_dtype, _p(q_scale), _p(q), _p(q_t), _p(q_amax), _p(dbias),
                                    _p(workspace), ws_bytes, _p(dh), _p(dev_status), _stream(stream)),
           "fp8_gemm_dgelu_cast")


def mxfp8_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the tiled E8M0 scale buffer of an MXFP8 [rows x cols] matrix (blocks along cols)."""
    return _lib.mxfp8_scale_bytes(rows, cols)


def mxfp8_quantize(x: torch.Tensor, row_q=None, row_s=None, col_q=None, col_s=None, dbias=None, workspace=None,
                   stream=None) -> None:
    """Row- and/or column-wise MXFP8 codes and tiled E8M0 scales of x; dbias (fp32 [cols])
    receives the column sums of x in the same pass (workspace: fp8_cast_workspace_size bytes)."""
    assert x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.mxfp8_quantize(_p(x), _hp(x), rows, cols, _p(row_q), _p(row_s), _p(col_q), _p(col_s), _p(dbias),
                               _p(workspace), ws_bytes, _stream(stream)), "mxfp8_quantize")


def mxfp8_gemm(A, A_s, B, B_s, D: torch.Tensor, bias: torch.Tensor | None = None, dev_status=None,
               stream=None) -> None:
    """D[M,N] = sum over 32-blocks of 2^(ea+eb) * (A_blk * B_blk^T) + bias."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and tuple(D.shape) == (M, N)
    _check(_lib.mxfp8_gemm(_p(A), _p(A_s), _p(B), _p(B_s), M, N, K, _p(bias),
                           _hp(bias) if bias is not None else BF16, _p(D), _hp(D), _p(dev_status), _stream(stream)),
           "mxfp8_gemm")


# --------------------------------------------------------------------------
# block-scaled FP8: one fp32 scale per 128 values (include/fp8dl.h has the layouts)
# --------------------------------------------------------------------------
def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _tensor(t, dtype, shape, dev: int, name: str):
    """Address of t, a contiguous tensor of this dtype and shape on device `dev` (or None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the device of the others, got %s %s on %s%s" % (
            name, dtype, tuple(shape), t.dtype, tuple(t.shape), t.device, "" if t.is_contiguous() else ", strided"))
    return t.data_ptr()


def _launch(dev: int, stream):
    """The stream to launch on; the tensors must be on the current CUDA device, where the kernels run."""
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device, got %s" % ("cuda:%d" % dev if dev >= 0 else "CPU tensors"))
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def fp8_block_padded_rows(rows: int, n_groups: int = 0) -> int:
    """Columns of the transposed codes of fp8_block_quantize (every group padded to a multiple of 128)."""
    return _lib.fp8_block_padded_rows(int(rows), int(n_groups))


def fp8_block_quantize(x: torch.Tensor, out_dtype: int, row_q=None, row_s=None, col_q=None, col_s=None, offsets=None,
                       dbias=None, workspace=None, stream=None) -> None:
    """Codes and factors of x [R x C] in blocks of 128: along the rows (row_q [R x C], row_s [C/128 x R]) and
    transposed, along the columns (col_q [C x T], col_s [T/128 x C], T = fp8_block_padded_rows(R, groups)).
    offsets (int32 [groups + 1]): ragged groups of rows, each padded to a multiple of 128 in col_q; dbias (fp32 [C],
    without offsets): column sums of x (workspace: fp8_cast_workspace_size bytes)."""
    _need(x.dim() == 2 and x.is_contiguous(), "x must be a contiguous matrix")
    rows, cols = x.shape
    groups = 0 if offsets is None else offsets.numel() - 1
    _need(groups >= 1 or offsets is None, "offsets must hold n_groups + 1 entries")
    dev, T = x.get_device(), (rows + 127 * min(max(groups, 1), rows)) // 128 * 128  # fp8_block_padded_rows
    _need(workspace is None or workspace.get_device() == dev, "workspace must be on the device of x")
    args = (x.data_ptr(), _hp(x), rows, cols, _tensor(offsets, torch.int32, (groups + 1,), dev, "offsets"), groups,
            out_dtype, _tensor(row_q, torch.uint8, (rows, cols), dev, "row_q"),
            _tensor(row_s, torch.float32, (_blocks(cols), rows), dev, "row_s"),
            _tensor(col_q, torch.uint8, (cols, T), dev, "col_q"),
            _tensor(col_s, torch.float32, (T // 128, cols), dev, "col_s"),
            _tensor(dbias, torch.float32, (cols,), dev, "dbias"), _p(workspace), _nbytes(workspace))
    _check(_lib.fp8_block_quantize(*args, _launch(dev, stream)), "fp8_block_quantize")


def fp8_block_quantize_weight(w: torch.Tensor, out_dtype: int, q=None, s=None, q_t=None, s_t=None,
                              stream=None) -> None:
    """Codes and factors of weights w [R x C] or [E x R x C] in 128 x 128 blocks: q like w with s [(E x) C/128 x R/128]
    (the B operand of the forward product), and transposed, q_t [(E x) C x R] with s_t [(E x) R/128 x C/128] (dgrad)."""
    _need(w.dim() in (2, 3) and w.is_contiguous(), "w must be a contiguous [R x C] or [E x R x C] tensor")
    lead, (rows, cols) = tuple(w.shape[:-2]), w.shape[-2:]
    dev = w.get_device()
    args = (w.data_ptr(), _hp(w), lead[0] if lead else 1, rows, cols, out_dtype,
            _tensor(q, torch.uint8, lead + (rows, cols), dev, "q"),
            _tensor(s, torch.float32, lead + (_blocks(cols), _blocks(rows)), dev, "s"),
            _tensor(q_t, torch.uint8, lead + (cols, rows), dev, "q_t"),
            _tensor(s_t, torch.float32, lead + (_blocks(rows), _blocks(cols)), dev, "s_t"))
    _check(_lib.fp8_block_quantize_weight(*args, _launch(dev, stream)), "fp8_block_quantize_weight")


def _status(dev_status, dev: int):
    return None if dev_status is None else _tensor(dev_status, torch.int32, dev_status.shape, dev, "dev_status")


def fp8_block_gemm(A: torch.Tensor, a_dtype: int, a_s: torch.Tensor, B: torch.Tensor, b_dtype: int, b_s: torch.Tensor,
                   D: torch.Tensor, bias: torch.Tensor | None = None, dev_status=None, stream=None) -> None:
    """D[M,N] = sum over blocks of 128 of (A_blk * B_blk^T) * a_s * b_s, + bias.  A [M x K], a_s [K/128 x M];
    B [N x K], b_s [K/128 x N/128] (a weight) or [K/128 x N] (an activation or gradient)."""
    _need(A.dim() == 2 and B.dim() == 2 and A.shape[1] == B.shape[1], "A [M x K] and B [N x K] must share K")
    (M, K), N, dev = A.shape, B.shape[0], A.get_device()
    b_rows = 1 if b_s.shape[-1:] == (N,) else 128
    args = (_tensor(A, torch.uint8, (M, K), dev, "A"), a_dtype, _tensor(a_s, torch.float32, (_blocks(K), M), dev, "a_s"),
            _tensor(B, torch.uint8, (N, K), dev, "B"), b_dtype,
            _tensor(b_s, torch.float32, (_blocks(K), N if b_rows == 1 else _blocks(N)), dev, "b_s"), b_rows, M, N, K,
            None if bias is None else _tensor(bias, bias.dtype, (N,), dev, "bias"),
            BF16 if bias is None else _hp(bias), _tensor(D, D.dtype, (M, N), dev, "D"), _hp(D), _status(dev_status, dev))
    _check(_lib.fp8_block_gemm(*args, _launch(dev, stream)), "fp8_block_gemm")


def fp8_block_gemm_plan(M: int, N: int, K: int, n_groups: int = 0, b_rows: int = 128) -> tuple[int, int, int, int]:
    """What fp8_block_gemm (or, with groups, fp8_block_gemm_grouped) runs a product as on the current device: rows of A
    a tile (16, 32, 64 or 256), CTAs (256: CTA pairs) that share each of the shared tiles, tiles computed alone, shared
    tiles.  Launches nothing."""
    rows, shares, whole, shared = _i32(), _i32(), _i64(), _i64()
    _check(_lib.fp8_block_gemm_plan(b_rows, n_groups, M, N, K, ctypes.byref(rows), ctypes.byref(shares), ctypes.byref(whole),
                                    ctypes.byref(shared)), "fp8_block_gemm_plan")
    return rows.value, shares.value, whole.value, shared.value


def fp8_block_gemm_grouped(A: torch.Tensor, a_dtype: int, a_s: torch.Tensor, B: torch.Tensor, b_dtype: int,
                           b_s: torch.Tensor, offsets: torch.Tensor, D: torch.Tensor, dev_status=None,
                           stream=None) -> None:
    """D[m] = A[m] * B[g]^T for the rows m of group g: A [M x K], a_s [K/128 x M]; B [G x N x K],
    b_s [G x K/128 x N/128]; offsets int32 [G + 1]; D [M x N].  Rows outside the groups keep their values."""
    _need(A.dim() == 2 and B.dim() == 3 and A.shape[1] == B.shape[2], "A [M x K] and B [G x N x K] must share K")
    (M, K), (G, N, _), dev = A.shape, B.shape, A.get_device()
    args = (_tensor(A, torch.uint8, (M, K), dev, "A"), a_dtype, _tensor(a_s, torch.float32, (_blocks(K), M), dev, "a_s"),
            _tensor(B, torch.uint8, (G, N, K), dev, "B"), b_dtype,
            _tensor(b_s, torch.float32, (G, _blocks(K), _blocks(N)), dev, "b_s"),
            _tensor(offsets, torch.int32, (G + 1,), dev, "offsets"), G, M, N, K, _tensor(D, D.dtype, (M, N), dev, "D"),
            _hp(D), _status(dev_status, dev))
    _check(_lib.fp8_block_gemm_grouped(*args, _launch(dev, stream)), "fp8_block_gemm_grouped")


def fp8_block_gemm_grouped_wgrad(A: torch.Tensor, a_dtype: int, a_s: torch.Tensor, B: torch.Tensor, b_dtype: int,
                                 b_s: torch.Tensor, offsets: torch.Tensor, D: torch.Tensor, dev_status=None,
                                 stream=None) -> None:
    """D[g] = A_g * B_g^T over group g's tokens: A [M x T], a_s [T/128 x M] and B [N x T], b_s [T/128 x N] are col_q and
    col_s of fp8_block_quantize with these offsets (int32 [G + 1]); D [G x M x N], zeros for a group without rows."""
    _need(A.dim() == 2 and B.dim() == 2 and A.shape[1] == B.shape[1], "A [M x T] and B [N x T] must share T")
    (M, T), N, G, dev = A.shape, B.shape[0], offsets.numel() - 1, A.get_device()
    args = (_tensor(A, torch.uint8, (M, T), dev, "A"), a_dtype, _tensor(a_s, torch.float32, (_blocks(T), M), dev, "a_s"),
            _tensor(B, torch.uint8, (N, T), dev, "B"), b_dtype, _tensor(b_s, torch.float32, (_blocks(T), N), dev, "b_s"),
            _tensor(offsets, torch.int32, (G + 1,), dev, "offsets"), G, M, N, T,
            _tensor(D, D.dtype, (G, M, N), dev, "D"), _hp(D), _status(dev_status, dev))
    _check(_lib.fp8_block_gemm_grouped_wgrad(*args, _launch(dev, stream)), "fp8_block_gemm_grouped_wgrad")


# --------------------------------------------------------------------------
# LayerNormMLP pieces (bf16 tensors)
# --------------------------------------------------------------------------
def _nbytes(t):
    return t.numel() * t.element_size() if isinstance(t, torch.Tensor) else 0


def fp8_layernorm_cast(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float, out_dtype: int, scale,
                       mu: torch.Tensor, rsigma: torch.Tensor, out=None, out_t=None, amax=None, y=None,
                       stream=None) -> None:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    _check(_lib.fp8_layernorm_cast(_p(x), rows, cols, _p(gamma), _p(beta), float(eps), out_dtype, _p(scale),
                                   _p(out), _p(out_t), _p(amax), _p(mu), _p(rsigma), _p(y), _stream(stream)),
           "fp8_layernorm_cast")


def fp8_gelu_cast(h: torch.Tensor, out_dtype: int, scale, out=None, out_t=None, amax=None, g=None,
                  stream=None) -> None:
    assert h.dtype == torch.bfloat16 and h.dim() == 2 and h.is_contiguous()
    rows, cols = h.shape
    _check(_lib.fp8_gelu_cast(_p(h), rows, cols, out_dtype, _p(scale), _p(out), _p(out_t), _p(amax), _p(g),
                              _stream(stream)), "fp8_gelu_cast")


def fp8_dgelu_cast(dg: torch.Tensor, h: torch.Tensor, out_dtype: int, scale, out=None, out_t=None, amax=None,
                   dbias=None, workspace=None, dh=None, stream=None) -> None:
    assert dg.dtype == torch.bfloat16 and h.dtype == torch.bfloat16 and dg.shape == h.shape
    rows, cols = h.shape
    _check(_lib.fp8_dgelu_cast(_p(dg), _p(h), rows, cols, out_dtype, _p(scale), _p(out), _p(out_t), _p(amax),
                               _p(dbias), _p(workspace), _nbytes(workspace), _p(dh), _stream(stream)),
           "fp8_dgelu_cast")


def fp8_layernorm_bwd_workspace_size(rows: int, cols: int) -> int:
    return _lib.fp8_layernorm_bwd_workspace_size(rows, cols)


def fp8_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mu, rsigma, dx: torch.Tensor,
                      dgamma: torch.Tensor, dbeta: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    rows, cols = x.shape
    _check(_lib.fp8_layernorm_bwd(_p(dy), _p(x), _p(gamma), _p(mu), _p(rsigma), rows, cols, _p(dx), _p(dgamma),
                                  _p(dbeta), _p(workspace), _nbytes(workspace), _stream(stream)),
           "fp8_layernorm_bwd")


from .autocast import fp8_autocast  # noqa: E402  (the step region; see autocast.py)
