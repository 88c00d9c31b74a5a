"""Python binding of libamsim (LUT-simulated approximate multipliers on GB300).

Argument marshalling only: every function forwards to the C ABI declared in
``include/amsim.h`` with the same name.  Device buffers are torch CUDA tensors
(or raw integer device pointers); the stream defaults to torch's current
stream.  All arithmetic runs in the library's CUDA kernels; there is no CPU
fallback -- importing works without a GPU, but calls fail loudly when the
library is not built or no GPU is present.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "amsim.h")
LIB_PATH = os.path.join(HERE, "_build", "libamsim.so")

AMSIM_EXACT = 0
AMSIM_MITCHELL = 1
KINDS = {"exact": AMSIM_EXACT, "mitchell": AMSIM_MITCHELL}

AMSIM_OK = 0
AMSIM_EINVAL = 1
AMSIM_EUNSUPPORTED = 2
AMSIM_ENOMEM = 3
AMSIM_ECUDA = 4
AMSIM_ETIMEOUT = 5
AMSIM_WAIT_COPY = 1
AMSIM_WAIT_PARTIAL = 2
AMSIM_WAIT_PHASE = 4

_lib = None


class AmsimError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({status_string(status)})")


class ConvDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("N", "H", "W", "C", "K", "R", "S", "stride_h", "stride_w", "pad_h", "pad_w", "dil_h", "dil_w")]

    @classmethod
    def make(cls, N, H, W, C, K, R, S, stride=(1, 1), pad=(0, 0), dil=(1, 1)):
        return cls(N, H, W, C, K, R, S, stride[0], stride[1], pad[0], pad[1], dil[0], dil[1])


APPROX_MUL_FN = ctypes.CFUNCTYPE(ctypes.c_float, ctypes.c_float, ctypes.c_float)


class GemmProblem(ctypes.Structure):
    """amsim_gemm_problem: one GEMM of a grouped launch."""
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("strideA", ctypes.c_int64), ("strideB", ctypes.c_int64), ("strideC", ctypes.c_int64),
                ("m", ctypes.c_int), ("n", ctypes.c_int), ("k", ctypes.c_int), ("lda", ctypes.c_int),
                ("ldb", ctypes.c_int), ("ldc", ctypes.c_int), ("batch", ctypes.c_int),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("transA", ctypes.c_char), ("transB", ctypes.c_char)]

    @classmethod
    def make(cls, transA, transB, m, n, k, alpha, A, lda, B, ldb, beta, C, ldc, strideA=0, strideB=0, strideC=0,
             batch=1):
        return cls(_ptr(A), _ptr(B), _ptr(C), strideA, strideB, strideC, m, n, k, lda, ldb, ldc, batch,
                   float(alpha), float(beta), transA.encode(), transB.encode())


AMSIM_F32 = 0
AMSIM_BF16 = 1
AMSIM_REDUCE_MEAN = 0
AMSIM_REDUCE_SUM = 1
REDUCTIONS = {"mean": AMSIM_REDUCE_MEAN, "sum": AMSIM_REDUCE_SUM}
AMSIM_ADAMW_BLOCK = 256
AMSIM_BLOCK_NORM_MAX_COLS = 16384
AMSIM_MAX_DISTANCE = 1024
AMSIM_ACT_NONE = 0
AMSIM_ACT_RELU = 1
AMSIM_ACT_SILU = 2
ACTIVATIONS = {"none": AMSIM_ACT_NONE, "relu": AMSIM_ACT_RELU, "silu": AMSIM_ACT_SILU}


class BlockNormDesc(ctypes.Structure):
    """amsim_block_norm_desc (row strides of 0 mean dense rows)."""
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "gate_rows", "ldx", "ldy", "ldr", "ldn", "lddx", "lddy", "lddr",
                                               "lddn")] +
                [(n, ctypes.c_int) for n in ("cols", "x_type", "y_type", "n_type")] +
                [("alpha", ctypes.c_float), ("eps", ctypes.c_float)])


class VocabLossDesc(ctypes.Structure):
    """amsim_vocab_loss_desc (row strides of 0 mean dense rows)."""
    _fields_ = ([(n, ctypes.c_int64) for n in ("tokens", "ignore_index", "ld_h", "ld_w", "ld_dh", "ld_dw")] +
                [(n, ctypes.c_int) for n in ("vocab", "dim", "reduction")])


class AdamwTensor(ctypes.Structure):
    """amsim_adamw_tensor: one tensor of a step."""
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("g_type", ctypes.c_int), ("reserved", ctypes.c_int)]

    @classmethod
    def make(cls, p, g, m, v, m_scale=None, v_scale=None, copy=None, weight_decay=0.0, lr_scale=1.0):
        """From contiguous CUDA tensors: p fp32; g fp32 or bf16; m, v fp32, or int8 and uint8 codes with their
        block scales; copy bf16 or None.  The tensors must outlive the table."""
        import torch
        n, eight, here = p.numel(), m_scale is not None, _current_device()
        want = [("p", p, torch.float32, n), ("m", m, torch.int8 if eight else torch.float32, n),
                ("v", v, torch.uint8 if eight else torch.float32, n), ("g", g, g.dtype, n)]
        blocks = -(-n // AMSIM_ADAMW_BLOCK)
        if eight:
            want += [("m_scale", m_scale, torch.float32, blocks), ("v_scale", v_scale, torch.float32, blocks)]
        if copy is not None:
            want.append(("copy", copy, torch.bfloat16, n))
        for name, t, dtype, size in want:
            if t is None or t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.numel() != size:
                raise TypeError(f"AdamwTensor: {name} must be a contiguous CUDA tensor of {size} {dtype} values")
            if t.get_device() != here:
                raise _elsewhere(name, t, here)
        entry = cls(_ptr(p), _ptr(g), _ptr(m), _ptr(v), _ptr(m_scale), _ptr(v_scale), _ptr(copy), n, float(lr_scale),
                    float(weight_decay), _dtype(g), 0)
        entry.device = here
        return entry


class AdamwHyper(ctypes.Structure):
    """amsim_adamw_hyper."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("grad_scale", ctypes.c_void_p)]


class DropoutDesc(ctypes.Structure):
    """amsim_dropout_desc."""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("call", ctypes.c_uint64), ("step", ctypes.c_void_p)]


class AttentionSoftmaxDesc(ctypes.Structure):
    """amsim_attention_softmax_desc (row strides of 0 mean dense rows)."""
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "heads", "queries", "keys", "ld_scores", "ld_probs",
                                               "ld_dprobs", "ld_dscores", "offset")] +
                [("lengths", ctypes.c_void_p), ("offsets", ctypes.c_void_p)] +
                [(n, ctypes.c_int) for n in ("causal", "num_buckets", "max_distance", "reserved")] +
                [("dropout", DropoutDesc)])


class GroupNormDesc(ctypes.Structure):
    """amsim_group_norm_desc (pixel strides of 0 mean dense channels)."""
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "pixels", "ldx", "ldy", "lddx")] +
                [(n, ctypes.c_int) for n in ("channels", "groups", "x_type", "y_type", "activation")] +
                [("eps", ctypes.c_float)])


def build():
    from . import build_ext
    return build_ext.build()


def lib():
    """Load libamsim.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libamsim.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz, ch = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t, ctypes.c_char)
    sig = {
        "amsim_status_string": ([i32], ctypes.c_char_p),
        "amsim_kernel_launches": ([], ctypes.c_ulonglong),
        "amsim_last_path": ([], i32),
        "amsim_device_errors": ([ctypes.POINTER(ctypes.c_uint), i32], i32),
        "amsim_set_flag_wait_limit": ([ctypes.c_longlong], i32),
        "amsim_set_cooperative_launches": ([i32], i32),
        "amsim_lut_generate": ([i32, i32, vp], i32),
        "amsim_lut_generate_from_fn": ([APPROX_MUL_FN, i32, vp], i32),
        "amsim_lut_build": ([i32, i32, ctypes.POINTER(vp)], i32),
        "amsim_lut_build_from_entries": ([vp, i32, ctypes.POINTER(vp)], i32),
        "amsim_lut_build_from_fn": ([APPROX_MUL_FN, i32, ctypes.POINTER(vp)], i32),
        "amsim_lut_entries": ([vp, vp], i32),
        "amsim_lut_info": ([vp, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
        "amsim_lut_set_closed_form": ([vp, i32], i32),
        "amsim_lut_set_exponent_bits": ([vp, i32], i32),
        "amsim_lut_destroy": ([vp], None),
        "amsim_mul": ([vp, vp, vp, i64, vp, vp], i32),
        "amsim_gemm": ([ch, ch, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp, vp, sz, vp], i32),
        "amsim_gemm_strided_batched": ([ch, ch, i32, i32, i32, f32, vp, i32, i64, vp, i32, i64, f32, vp, i32,
                                        i64, i32, vp, vp, sz, vp], i32),
        "amsim_gemm_workspace_size": ([ch, ch, i32, i32, i32, i32, vp], sz),
        "amsim_gemm_grouped": ([i32, ctypes.POINTER(GemmProblem), vp, vp, sz, vp], i32),
        "amsim_gemm_noalloc": ([ch, ch, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp, vp], i32),
        "amsim_gemm_grouped_workspace_size": ([i32, ctypes.POINTER(GemmProblem), vp], sz),
        "amsim_gemm_phased": ([i32, ctypes.POINTER(GemmProblem), i32, ctypes.POINTER(i32), ctypes.POINTER(i32), vp,
                               vp, sz, vp], i32),
        "amsim_gemm_phased_workspace_size": ([i32, ctypes.POINTER(GemmProblem), i32, ctypes.POINTER(i32),
                                              ctypes.POINTER(i32), vp], sz),
        "amsim_conv2d_out_hw": ([ctypes.POINTER(ConvDesc), ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
        "amsim_conv2d_fwd": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_conv2d_bwd_data": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_conv2d_bwd_filter": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_conv2d_workspace_size": ([ctypes.POINTER(ConvDesc), i32, vp], sz),
        "amsim_dwconv2d_fwd": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_dwconv2d_bwd_data": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_dwconv2d_bwd_filter": ([ctypes.POINTER(ConvDesc), vp, vp, vp, vp, vp, sz, vp], i32),
        "amsim_dwconv2d_workspace_size": ([ctypes.POINTER(ConvDesc), i32, vp], sz),
        "amsim_softmax_rows": ([vp, vp, i64, i32, vp], i32),
        "amsim_softmax_rows_backward": ([vp, vp, vp, i64, i32, vp], i32),
        "amsim_block_norm_fwd": ([ctypes.POINTER(BlockNormDesc)] + [vp] * 10, i32),
        "amsim_block_norm_bwd": ([ctypes.POINTER(BlockNormDesc)] + [vp] * 15 + [sz, vp], i32),
        "amsim_block_norm_workspace_size": ([ctypes.POINTER(BlockNormDesc)], sz),
        "amsim_vocab_loss": ([ctypes.POINTER(VocabLossDesc)] + [vp] * 8 + [sz, vp], i32),
        "amsim_vocab_loss_grad": ([ctypes.POINTER(VocabLossDesc)] + [vp] * 10 + [sz, vp], i32),
        "amsim_vocab_loss_workspace_size": ([ctypes.POINTER(VocabLossDesc), i32], sz),
        "amsim_vocab_loss_workspace_size_at": ([ctypes.POINTER(VocabLossDesc), i32, vp, vp], sz),
        "amsim_vocab_loss_workspace_min": ([ctypes.POINTER(VocabLossDesc), i32], sz),
        "amsim_adamw_step": ([i32, ctypes.POINTER(AdamwTensor), ctypes.POINTER(AdamwHyper), vp], i32),
        "amsim_adamw_moment_values": ([vp, vp, i32, i64, vp, vp], i32),
        "amsim_dropout": ([ctypes.POINTER(DropoutDesc), i32, i64, vp, vp, vp, vp], i32),
        "amsim_attention_softmax_fwd": ([ctypes.POINTER(AttentionSoftmaxDesc)] + [vp] * 6, i32),
        "amsim_attention_softmax_bwd": ([ctypes.POINTER(AttentionSoftmaxDesc)] + [vp] * 9 + [sz, vp], i32),
        "amsim_attention_softmax_workspace_size": ([ctypes.POINTER(AttentionSoftmaxDesc)], sz),
        "amsim_group_norm_fwd": ([ctypes.POINTER(GroupNormDesc)] + [vp] * 7 + [sz, vp], i32),
        "amsim_group_norm_bwd": ([ctypes.POINTER(GroupNormDesc)] + [vp] * 10 + [sz, vp], i32),
        "amsim_group_norm_workspace_size": ([ctypes.POINTER(GroupNormDesc), i32], sz),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions that include/amsim.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"\b(amsim_[a-z0-9_]+)\s*\(", text)
    return sorted(set(names))


AMSIM_PATH_PLANES = 1
AMSIM_PATH_INKERNEL_DECODE = 4
AMSIM_PATH_SINGLE_ROLE = 8
AMSIM_PATH_STREAMK = 16
AMSIM_PATH_FIXUP = 32
AMSIM_PATH_CONV_BOXES = 64
AMSIM_PATH_RAW_TILES = 128
AMSIM_PATH_PHASED = 256
AMSIM_PATH_CLOSED_FORM = 512
AMSIM_PATH_DW_TILES = 1024
AMSIM_PATH_DW_DIRECT = 2048
AMSIM_PATH_WIDE_TILES = 4096


def amsim_last_path() -> int:
    """Kernel-path bits (AMSIM_PATH_*) of this thread's most recent GEMM or convolution call."""
    return int(lib().amsim_last_path())


def amsim_kernel_launches() -> int:
    """Kernels the library has enqueued so far in this process."""
    return int(lib().amsim_kernel_launches())


def amsim_device_errors(clear: bool = True) -> tuple[int, int]:
    """(status, AMSIM_WAIT_* bits) of the device-side waits that gave up on the
    current device since the last clear (synchronises the device)."""
    bits = ctypes.c_uint(0)
    rc = lib().amsim_device_errors(ctypes.byref(bits), 1 if clear else 0)
    if rc not in (AMSIM_OK, AMSIM_ETIMEOUT):
        raise AmsimError("amsim_device_errors", rc)
    return rc, int(bits.value)


def amsim_set_flag_wait_limit(ns: int) -> None:
    _check("amsim_set_flag_wait_limit", lib().amsim_set_flag_wait_limit(int(ns)))


def amsim_set_cooperative_launches(on: bool) -> None:
    _check("amsim_set_cooperative_launches", lib().amsim_set_cooperative_launches(1 if on else 0))


def status_string(status: int) -> str:
    return lib().amsim_status_string(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != AMSIM_OK:
        raise AmsimError(fn, rc)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if hasattr(t, "ctypes"):
        return t.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(t)}")


def _at(t) -> int | None:
    """_ptr of a checked tensor or None, in half the time (a small call's time is the host's)."""
    return None if t is None else t.data_ptr()


_device_index = None


def _current_device() -> int:
    """torch's current CUDA device, on which a call's tensors must be: its stream and its kernels are that one's.  Less
    than any tensor's device without one."""
    global _device_index
    try:
        if _device_index is None:
            import torch
            _device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        return _device_index()
    except (RuntimeError, AssertionError):
        return -2


def _elsewhere(name, t, here):
    """The error of a tensor that is not on device `here`."""
    if not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")


_raw_stream = None


def _current_stream() -> int:
    """torch's current stream on the current device, as a raw handle."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if get is not None and device is not None:
            _raw_stream = lambda: get(device())     # without building a Stream object: a tenth of the time
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _raw_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    if t is None:
        return 0
    return t.numel() * t.element_size()


def _kind(kind) -> int:
    return KINDS[kind] if isinstance(kind, str) else int(kind)


# ------------------------------------------------------------------ LUT
class Lut:
    """Owner of an amsim_lut_t handle (device LUT on the current device).  There is one owner of a handle: a copy, or a
    copied layer's, is the same object."""

    def __init__(self, handle: int, M: int):
        self.handle = handle
        self.M = M

    @classmethod
    def build(cls, kind, M: int) -> "Lut":
        return cls(amsim_lut_build(kind, M), M)

    @classmethod
    def from_entries(cls, entries, M: int) -> "Lut":
        return cls(amsim_lut_build_from_entries(entries, M), M)

    @classmethod
    def from_fn(cls, approx_mul, M: int) -> "Lut":
        return cls(amsim_lut_build_from_fn(approx_mul, M), M)

    def info(self):
        return amsim_lut_info(self.handle)

    def entries(self):
        return amsim_lut_entries(self.handle, self.M)

    def set_closed_form(self, on: bool = True) -> "Lut":
        amsim_lut_set_closed_form(self.handle, on)
        return self

    def set_exponent_bits(self, E: int) -> "Lut":
        amsim_lut_set_exponent_bits(self.handle, E)
        return self

    def close(self):
        if self.handle:
            lib().amsim_lut_destroy(self.handle)
            self.handle = None

    def __copy__(self):
        return self

    def __deepcopy__(self, memo):
        return self

    def __reduce__(self):
        raise TypeError("a Lut holds device memory and cannot be pickled: save a layer's state dict, and build the table "
                        "again")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _h(lut) -> int:
    return lut.handle if isinstance(lut, Lut) else lut


def amsim_lut_generate(kind, M: int):
    import numpy as np
    out = np.zeros(1 << (2 * M) if 1 <= M <= 11 else 1, dtype=np.uint32)
    _check("amsim_lut_generate", lib().amsim_lut_generate(_kind(kind), M, out.ctypes.data))
    return out


def amsim_lut_generate_from_fn(approx_mul, M: int):
    import numpy as np
    out = np.zeros(1 << (2 * M) if 1 <= M <= 11 else 1, dtype=np.uint32)
    cb = APPROX_MUL_FN(approx_mul)
    _check("amsim_lut_generate_from_fn", lib().amsim_lut_generate_from_fn(cb, M, out.ctypes.data))
    return out


def amsim_lut_build(kind, M: int) -> int:
    h = ctypes.c_void_p(0)
    _check("amsim_lut_build", lib().amsim_lut_build(_kind(kind), M, ctypes.byref(h)))
    return h.value


def amsim_lut_build_from_entries(entries, M: int) -> int:
    import numpy as np
    e = np.ascontiguousarray(entries, dtype=np.uint32)
    h = ctypes.c_void_p(0)
    _check("amsim_lut_build_from_entries", lib().amsim_lut_build_from_entries(e.ctypes.data, M, ctypes.byref(h)))
    return h.value


def amsim_lut_build_from_fn(approx_mul, M: int) -> int:
    """approx_mul: a Python callable (float, float) -> float, called through a C
    function pointer during the call."""
    cb = APPROX_MUL_FN(approx_mul)
    h = ctypes.c_void_p(0)
    _check("amsim_lut_build_from_fn", lib().amsim_lut_build_from_fn(cb, M, ctypes.byref(h)))
    return h.value


def amsim_lut_entries(lut, M: int):
    import numpy as np
    out = np.zeros(1 << (2 * M), dtype=np.uint32)
    _check("amsim_lut_entries", lib().amsim_lut_entries(_h(lut), out.ctypes.data))
    return out


def amsim_lut_set_closed_form(lut, on: bool = True) -> None:
    _check("amsim_lut_set_closed_form", lib().amsim_lut_set_closed_form(_h(lut), 1 if on else 0))


def amsim_lut_set_exponent_bits(lut, E: int) -> None:
    """Exponent width E (1..8) of the simulated (1, E, M) multiplier."""
    _check("amsim_lut_set_exponent_bits", lib().amsim_lut_set_exponent_bits(_h(lut), int(E)))


def amsim_lut_info(lut):
    M, w, s = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check("amsim_lut_info", lib().amsim_lut_info(_h(lut), ctypes.byref(M), ctypes.byref(w), ctypes.byref(s)))
    return {"M": M.value, "width_bits": w.value, "shift": s.value}


def amsim_lut_destroy(lut):
    if isinstance(lut, Lut):
        lut.close()
    else:
        lib().amsim_lut_destroy(lut)


# ------------------------------------------------------------------ compute calls
def amsim_mul(a, b, c, n: int, lut, stream=None):
    _check("amsim_mul", lib().amsim_mul(_ptr(a), _ptr(b), _ptr(c), int(n), _h(lut), _stream(stream)))


def amsim_gemm(transA, transB, m, n, k, alpha, A, lda, B, ldb, beta, C, ldc, lut, ws=None, ws_bytes=None,
               stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_gemm", lib().amsim_gemm(transA.encode(), transB.encode(), m, n, k, float(alpha), _ptr(A), lda,
                                          _ptr(B), ldb, float(beta), _ptr(C), ldc, _h(lut), _ptr(ws), ws_bytes,
                                          _stream(stream)))


def amsim_gemm_strided_batched(transA, transB, m, n, k, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                               strideC, batch, lut, ws=None, ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_gemm_strided_batched",
           lib().amsim_gemm_strided_batched(transA.encode(), transB.encode(), m, n, k, float(alpha), _ptr(A), lda,
                                            strideA, _ptr(B), ldb, strideB, float(beta), _ptr(C), ldc, strideC,
                                            batch, _h(lut), _ptr(ws), ws_bytes, _stream(stream)))


def amsim_gemm_noalloc(transA, transB, m, n, k, alpha, A, lda, B, ldb, beta, C, ldc, lut, stream=None):
    """amsim_gemm with its scratch inside the library (no workspace, no allocation)."""
    _check("amsim_gemm_noalloc", lib().amsim_gemm_noalloc(transA.encode(), transB.encode(), m, n, k, float(alpha),
                                                          _ptr(A), lda, _ptr(B), ldb, float(beta), _ptr(C), ldc,
                                                          _h(lut), _stream(stream)))


def amsim_gemm_workspace_size(transA, transB, m, n, k, batch, lut) -> int:
    return int(lib().amsim_gemm_workspace_size(transA.encode(), transB.encode(), m, n, k, batch, _h(lut)))


def _problem_array(problems):
    if isinstance(problems, ctypes.Array):
        return problems
    arr = (GemmProblem * len(problems))()
    for i, p in enumerate(problems):
        arr[i] = p
    return arr


def amsim_gemm_grouped(problems, lut, ws=None, ws_bytes=None, stream=None):
    """problems: a sequence of GemmProblem (or a ctypes array of them)."""
    arr = _problem_array(problems)
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_gemm_grouped", lib().amsim_gemm_grouped(len(arr), arr, _h(lut), _ptr(ws), ws_bytes,
                                                          _stream(stream)))


def _phase_arrays(phase_first, phase_after):
    n = len(phase_first)
    if len(phase_after) != n:
        raise ValueError("phase_first and phase_after differ in length")
    return n, (ctypes.c_int32 * n)(*phase_first), (ctypes.c_int32 * n)(*phase_after)


def amsim_gemm_phased(problems, phase_first, phase_after, lut, ws=None, ws_bytes=None, stream=None):
    """Ordered phases of GEMMs (sequences of GemmProblem): phase ph is
    problems[phase_first[ph]:phase_first[ph + 1]] and reads outputs of phases
    before phase_after[ph] only."""
    arr = _problem_array(problems)
    nph, first, after = _phase_arrays(phase_first, phase_after)
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_gemm_phased", lib().amsim_gemm_phased(len(arr), arr, nph, first, after, _h(lut), _ptr(ws),
                                                        ws_bytes, _stream(stream)))


def amsim_gemm_phased_workspace_size(problems, phase_first, phase_after, lut) -> int:
    arr = _problem_array(problems)
    nph, first, after = _phase_arrays(phase_first, phase_after)
    return int(lib().amsim_gemm_phased_workspace_size(len(arr), arr, nph, first, after, _h(lut)))


def amsim_gemm_grouped_workspace_size(problems, lut) -> int:
    arr = _problem_array(problems)
    return int(lib().amsim_gemm_grouped_workspace_size(len(arr), arr, _h(lut)))


def amsim_conv2d_out_hw(desc: ConvDesc):
    P, Q = ctypes.c_int(0), ctypes.c_int(0)
    _check("amsim_conv2d_out_hw", lib().amsim_conv2d_out_hw(ctypes.byref(desc), ctypes.byref(P), ctypes.byref(Q)))
    return P.value, Q.value


def _conv(name, desc, t0, t1, out, lut, ws, ws_bytes, stream):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check(name, getattr(lib(), name)(ctypes.byref(desc), _ptr(t0), _ptr(t1), _ptr(out), _h(lut), _ptr(ws),
                                      ws_bytes, _stream(stream)))


def amsim_conv2d_fwd(desc, x, w, y, lut, ws=None, ws_bytes=None, stream=None):
    _conv("amsim_conv2d_fwd", desc, x, w, y, lut, ws, ws_bytes, stream)


def amsim_conv2d_bwd_data(desc, dy, w, dx, lut, ws=None, ws_bytes=None, stream=None):
    _conv("amsim_conv2d_bwd_data", desc, dy, w, dx, lut, ws, ws_bytes, stream)


def amsim_conv2d_bwd_filter(desc, x, dy, dw, lut, ws=None, ws_bytes=None, stream=None):
    _conv("amsim_conv2d_bwd_filter", desc, x, dy, dw, lut, ws, ws_bytes, stream)


def amsim_conv2d_workspace_size(desc, which: int, lut) -> int:
    return int(lib().amsim_conv2d_workspace_size(ctypes.byref(desc), int(which), _h(lut)))


def amsim_dwconv2d_fwd(desc, x, w, y, lut, ws=None, ws_bytes=None, stream=None):
    """Depthwise forward; desc.K = C * D, w is R x S x C x D."""
    _conv("amsim_dwconv2d_fwd", desc, x, w, y, lut, ws, ws_bytes, stream)


def amsim_dwconv2d_bwd_data(desc, dy, w, dx, lut, ws=None, ws_bytes=None, stream=None):
    _conv("amsim_dwconv2d_bwd_data", desc, dy, w, dx, lut, ws, ws_bytes, stream)


def amsim_dwconv2d_bwd_filter(desc, x, dy, dw, lut, ws=None, ws_bytes=None, stream=None):
    _conv("amsim_dwconv2d_bwd_filter", desc, x, dy, dw, lut, ws, ws_bytes, stream)


def amsim_dwconv2d_workspace_size(desc, which: int, lut) -> int:
    return int(lib().amsim_dwconv2d_workspace_size(ctypes.byref(desc), int(which), _h(lut)))


def amsim_softmax_rows_backward(P, dP, dS, rows, cols, stream=None):
    _check("amsim_softmax_rows_backward",
           lib().amsim_softmax_rows_backward(_ptr(P), _ptr(dP), _ptr(dS), int(rows), int(cols), _stream(stream)))


def amsim_softmax_rows(S, P, rows, cols, stream=None):
    _check("amsim_softmax_rows", lib().amsim_softmax_rows(_ptr(S), _ptr(P), int(rows), int(cols),
                                                          _stream(stream)))


def amsim_block_norm_fwd(desc: BlockNormDesc, x, y, gate, w_post, w_pre, r, n, rstd_post, rstd_pre, stream=None):
    _check("amsim_block_norm_fwd",
           lib().amsim_block_norm_fwd(ctypes.byref(desc), _ptr(x), _ptr(y), _ptr(gate), _ptr(w_post), _ptr(w_pre),
                                      _ptr(r), _ptr(n), _ptr(rstd_post), _ptr(rstd_pre), _stream(stream)))


def amsim_block_norm_bwd(desc: BlockNormDesc, dr, dn, r, y, gate, w_post, w_pre, rstd_post, rstd_pre, dx, dy, dgate,
                         dw_post, dw_pre, ws=None, ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_block_norm_bwd",
           lib().amsim_block_norm_bwd(ctypes.byref(desc), _ptr(dr), _ptr(dn), _ptr(r), _ptr(y), _ptr(gate),
                                      _ptr(w_post), _ptr(w_pre), _ptr(rstd_post), _ptr(rstd_pre), _ptr(dx), _ptr(dy),
                                      _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), _ptr(ws), ws_bytes,
                                      _stream(stream)))


def amsim_block_norm_workspace_size(desc: BlockNormDesc) -> int:
    return int(lib().amsim_block_norm_workspace_size(ctypes.byref(desc)))


def amsim_vocab_loss(desc: VocabLossDesc, h, w, targets, row_weight, loss, row_loss, lse, ws=None, ws_bytes=None,
                     stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_vocab_loss",
           lib().amsim_vocab_loss(ctypes.byref(desc), _ptr(h), _ptr(w), _ptr(targets), _ptr(row_weight), _ptr(loss),
                                  _ptr(row_loss), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream)))


def amsim_vocab_loss_grad(desc: VocabLossDesc, h, w, targets, row_weight, loss, row_loss, lse, dh, dw, ws=None,
                          ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_vocab_loss_grad",
           lib().amsim_vocab_loss_grad(ctypes.byref(desc), _ptr(h), _ptr(w), _ptr(targets), _ptr(row_weight),
                                       _ptr(loss), _ptr(row_loss), _ptr(lse), _ptr(dh), _ptr(dw), _ptr(ws), ws_bytes,
                                       _stream(stream)))


def amsim_vocab_loss_workspace_size(desc: VocabLossDesc, which: int) -> int:
    return int(lib().amsim_vocab_loss_workspace_size(ctypes.byref(desc), int(which)))


def amsim_vocab_loss_workspace_size_at(desc: VocabLossDesc, which: int, h, w) -> int:
    return int(lib().amsim_vocab_loss_workspace_size_at(ctypes.byref(desc), int(which), _ptr(h), _ptr(w)))


def amsim_vocab_loss_workspace_min(desc: VocabLossDesc, which: int) -> int:
    return int(lib().amsim_vocab_loss_workspace_min(ctypes.byref(desc), int(which)))


def amsim_adamw_step(tensors, hyper: AdamwHyper, stream=None):
    """tensors: a ctypes array of AdamwTensor (adamw_table)."""
    _check("amsim_adamw_step", lib().amsim_adamw_step(len(tensors), tensors, ctypes.byref(hyper), _stream(stream)))


def amsim_adamw_moment_values(codes, scales, second: bool, n: int, out, stream=None):
    _check("amsim_adamw_moment_values",
           lib().amsim_adamw_moment_values(_ptr(codes), _ptr(scales), 1 if second else 0, int(n), _ptr(out),
                                           _stream(stream)))


def amsim_dropout(desc: DropoutDesc, type: int, n: int, x, residual, y, stream=None):
    _check("amsim_dropout", lib().amsim_dropout(ctypes.byref(desc), int(type), int(n), _ptr(x), _ptr(residual), _ptr(y),
                                                _stream(stream)))


def amsim_attention_softmax_fwd(desc: AttentionSoftmaxDesc, scores, table, buckets, probs, stats, stream=None):
    _check("amsim_attention_softmax_fwd",
           lib().amsim_attention_softmax_fwd(ctypes.byref(desc), _ptr(scores), _ptr(table), _ptr(buckets), _ptr(probs),
                                             _ptr(stats), _stream(stream)))


def amsim_attention_softmax_bwd(desc: AttentionSoftmaxDesc, dprobs, scores, stats, probs, table, buckets, dscores,
                                dtable, ws=None, ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_attention_softmax_bwd",
           lib().amsim_attention_softmax_bwd(ctypes.byref(desc), _ptr(dprobs), _ptr(scores), _ptr(stats), _ptr(probs),
                                             _ptr(table), _ptr(buckets), _ptr(dscores), _ptr(dtable), _ptr(ws),
                                             ws_bytes, _stream(stream)))


def amsim_attention_softmax_workspace_size(desc: AttentionSoftmaxDesc) -> int:
    return int(lib().amsim_attention_softmax_workspace_size(ctypes.byref(desc)))


def amsim_group_norm_fwd(desc: GroupNormDesc, x, w, b, y, mean, rstd, ws=None, ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_group_norm_fwd",
           lib().amsim_group_norm_fwd(ctypes.byref(desc), _ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd),
                                      _ptr(ws), ws_bytes, _stream(stream)))


def amsim_group_norm_bwd(desc: GroupNormDesc, dy, x, w, b, mean, rstd, dx, dw, db, ws=None, ws_bytes=None, stream=None):
    ws_bytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("amsim_group_norm_bwd",
           lib().amsim_group_norm_bwd(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(w), _ptr(b), _ptr(mean), _ptr(rstd),
                                      _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), ws_bytes, _stream(stream)))


def amsim_group_norm_workspace_size(desc: GroupNormDesc, which: int) -> int:
    return int(lib().amsim_group_norm_workspace_size(ctypes.byref(desc), int(which)))


# ------------------------------------------------------------------ conveniences (still marshalling only)
def workspace(nbytes: int, device=None):
    """A caller-owned scratch buffer (uint8 torch tensor, 256-byte aligned by the caching allocator)."""
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device or "cuda")


def gemm(A, B, lut, *, transA=False, transB=False, alpha=1.0, beta=0.0, C=None, ws=None, stream=None):
    """C = alpha op(A) op(B) + beta C for contiguous row-major fp32 CUDA tensors."""
    import torch
    m = A.shape[1] if transA else A.shape[0]
    k = A.shape[0] if transA else A.shape[1]
    n = B.shape[0] if transB else B.shape[1]
    if C is None:
        C = torch.empty((m, n), dtype=torch.float32, device=A.device)
    if ws is None:
        ws = workspace(amsim_gemm_workspace_size("T" if transA else "N", "T" if transB else "N", m, n, k, 1, lut),
                       A.device)
    amsim_gemm("T" if transA else "N", "T" if transB else "N", m, n, k, alpha, A, max(1, A.shape[1]), B,
               max(1, B.shape[1]), beta, C, max(1, n), lut, ws=ws, stream=stream)
    return C


_dtypes = {}


def _dtype(t) -> int:
    """amsim_dtype of a tensor (or of a torch dtype)."""
    dtype = getattr(t, "dtype", t)
    if dtype in _dtypes:
        return _dtypes[dtype]
    import torch
    if dtype in (torch.float32, torch.bfloat16):
        _dtypes.update({torch.float32: AMSIM_F32, torch.bfloat16: AMSIM_BF16})
        return _dtypes[dtype]
    raise TypeError(f"exact operators take fp32 or bf16 tensors, not {dtype}")


def _rows(name, t, rows, cols, here, dtype=None) -> int:
    """Row stride of a matrix of `rows` x `cols` on device `here` whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {rows} x {cols}, not {tuple(t.shape)}")
    if t.get_device() != here:
        raise _elsewhere(name, t, here)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.is_contiguous():
        return cols
    outer, inner = t.stride()
    if cols > 1 and inner != 1 or rows > 1 and outer < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return outer if rows > 1 else cols


def _vector(name, t, n, dtype, here):
    if t.get_device() != here:
        raise _elsewhere(name, t, here)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values")


# Descriptors and scratch sizes by the sizes and types of a call: a small call's
# time is the host's, and building them costs more than its launch.
@functools.lru_cache(maxsize=1024)
def _block_norm_plan(rows, cols, gate_rows, x, y, n, r, dr, dn, alpha, eps, backward):
    """(descriptor by reference, scratch bytes); x, y, n: (type, row stride)."""
    d = BlockNormDesc(rows=rows, cols=cols, gate_rows=gate_rows, alpha=alpha, eps=eps, x_type=x[0], ldx=x[1],
                      y_type=y[0], ldy=y[1], n_type=n[0], ldr=r, lddr=dr, lddn=dn)
    return ctypes.byref(d), amsim_block_norm_workspace_size(d) if backward else 0


@functools.lru_cache(maxsize=1024)
def _vocab_plan(tokens, vocab, dim, ld_h, ld_w, ignore_index, reduction, h, w):
    """(descriptor by reference, scratch bytes of the loss, of the gradients); h, w: addresses alike in their last bits."""
    d = VocabLossDesc(tokens=tokens, vocab=vocab, dim=dim, ld_h=ld_h, ld_w=ld_w, ignore_index=ignore_index,
                      reduction=REDUCTIONS[reduction])
    return ctypes.byref(d), *(amsim_vocab_loss_workspace_size_at(d, which, h, w) for which in (0, 1))


def _gate_rows(first, gate, w_post, w_pre, here):
    """Rows per row of the gate (0 without one), the vectors of a block norm over rows like `first`'s checked."""
    import torch
    if first.ndim != 2:
        raise ValueError("block norms take matrices of rows x channels")
    rows, cols = first.shape
    if w_post is not None:
        _vector("w_post", w_post, cols, torch.float32, here)
    if w_pre is not None:
        _vector("w_pre", w_pre, cols, torch.float32, here)
    if gate is None:
        return 0
    groups = gate.shape[0] if gate.ndim == 2 else 1
    if gate.ndim not in (1, 2) or gate.shape[-1] != cols or groups < 1 or rows % groups:
        raise ValueError(f"gate must have one row of {cols} values for every so many of the {rows} rows")
    _vector("gate", gate, groups * cols, torch.float32, here)
    return rows // groups


def block_norm(x, y=None, w_post=None, w_pre=None, *, gate=None, alpha=1.0, eps=1e-6, n_dtype=None):
    """r = x + alpha gate rms_norm(y) w_post and n = rms_norm(r) w_pre: (r, n, rstd_post, rstd_pre).

    x: rows x channels, fp32 or bf16; y the same shape (or None: r is x itself); w_post None: y enters as it is;
    gate: [groups, channels], one row for each rows / groups consecutive rows, or None.  n has type `n_dtype` (y's,
    or x's).  rstd_post is None without w_post."""
    import torch
    here = _current_device()
    gate_rows = _gate_rows(x, gate, w_post, w_pre, here)
    rows, cols = x.shape
    xs = (_dtype(x), _rows("x", x, rows, cols, here))
    ys = (AMSIM_F32, 0) if y is None else (_dtype(y), _rows("y", y, rows, cols, here))
    empty, device = torch.empty, x.device
    n = empty((rows, cols), dtype=n_dtype or (x if y is None else y).dtype, device=device)
    desc, _ = _block_norm_plan(rows, cols, gate_rows, xs, ys, (_dtype(n), 0), 0, 0, 0, alpha, eps, False)
    r = x if y is None else empty((rows, cols), dtype=x.dtype, device=device)
    rstd_pre = empty(rows, dtype=torch.float32, device=device)
    rstd_post = None if w_post is None else empty(rows, dtype=torch.float32, device=device)
    _check("amsim_block_norm_fwd",
           lib().amsim_block_norm_fwd(desc, x.data_ptr(), _at(y), _at(gate), _at(w_post), _at(w_pre),
                                      None if y is None else r.data_ptr(), n.data_ptr(), _at(rstd_post),
                                      rstd_pre.data_ptr(), _current_stream()))
    return r, n, rstd_post, rstd_pre


def block_norm_backward(dr, dn, r, y, w_post, w_pre, rstd_post, rstd_pre, *, gate=None, alpha=1.0):
    """Gradients of block_norm: (dx, dy, dgate, dw_post, dw_pre), None where there was no such input.  dr or dn may
    be None (zeros); r, rstd_post and rstd_pre are block_norm's."""
    import torch
    here = _current_device()
    gate_rows = _gate_rows(r, gate, w_post, w_pre, here)
    rows, cols = r.shape
    f32, empty, device = torch.float32, torch.empty, r.device
    ys, ns, lddr, lddn = (AMSIM_F32, 0), (AMSIM_F32, 0), 0, 0
    ldr = _rows("r", r, rows, cols, here)
    if dr is not None:
        lddr = _rows("dr", dr, rows, cols, here, r.dtype)
    if dn is not None:
        ns, lddn = (_dtype(dn), 0), _rows("dn", dn, rows, cols, here)
        _vector("rstd_pre", rstd_pre, rows, f32, here)
    dx = empty((rows, cols), dtype=r.dtype, device=device)
    dy = dgate = dw_post = dw_pre = None
    if y is not None:
        ys = (_dtype(y), _rows("y", y, rows, cols, here))
        dy = empty((rows, cols), dtype=y.dtype, device=device)
    if gate is not None:
        dgate = torch.empty_like(gate) if rows else torch.zeros_like(gate)
    if w_post is not None:
        _vector("rstd_post", rstd_post, rows, f32, here)
        dw_post = torch.empty_like(w_post)
    if w_pre is not None:
        dw_pre = torch.empty_like(w_pre) if dn is not None else torch.zeros_like(w_pre)
    desc, nb = _block_norm_plan(rows, cols, gate_rows, (_dtype(r), 0), ys, ns, ldr, lddr, lddn, alpha, 0.0, True)
    ws = empty(nb, dtype=torch.uint8, device=device) if nb else None
    _check("amsim_block_norm_bwd",
           lib().amsim_block_norm_bwd(desc, _at(dr), _at(dn), r.data_ptr(), _at(y), _at(gate), _at(w_post),
                                      _at(w_pre), _at(rstd_post), _at(rstd_pre), dx.data_ptr(), _at(dy),
                                      _at(dgate), _at(dw_post), _at(dw_pre) if dn is not None else None, _at(ws),
                                      nb, _current_stream()))
    return dx, dy, dgate, dw_post, dw_pre


def _vocab_call(h, w, targets, row_weight, ignore_index, reduction):
    import torch
    if h.dim() != 2 or w.dim() != 2:
        raise ValueError("the vocabulary loss takes h [tokens, dim] and w [vocab, dim]")
    tokens, dim = h.shape
    vocab = w.shape[0]
    bf16, here = torch.bfloat16, _current_device()
    plan = _vocab_plan(tokens, vocab, dim, _rows("h", h, tokens, dim, here, bf16), _rows("w", w, vocab, dim, here, bf16),
                       ignore_index, reduction, 128 + h.data_ptr() % 128, 128 + w.data_ptr() % 128)
    _vector("targets", targets, tokens, torch.int64, here)
    if row_weight is not None:
        _vector("row_weight", row_weight, tokens, torch.float32, here)
    empty, device = torch.empty, h.device
    row = empty(tokens, dtype=torch.float32, device=device)
    return plan, empty(1, dtype=torch.float32, device=device), row, torch.empty_like(row)


def vocab_loss(h, w, targets, *, row_weight=None, ignore_index=-100, reduction="mean"):
    """Cross entropy of softmax(h w^T) against the targets, without the logits: (loss [1], row_loss, lse).
    h [tokens, dim] and w [vocab, dim] bf16, targets int64; reduction "mean" (over the tokens' weights) or "sum"."""
    import torch
    (desc, nb, _), loss, row, lse = _vocab_call(h, w, targets, row_weight, ignore_index, reduction)
    ws = torch.empty(nb, dtype=torch.uint8, device=h.device)
    _check("amsim_vocab_loss",
           lib().amsim_vocab_loss(desc, h.data_ptr(), w.data_ptr(), targets.data_ptr(), _at(row_weight),
                                  loss.data_ptr(), row.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb,
                                  _current_stream()))
    return loss, row, lse


def vocab_loss_grad(h, w, targets, *, row_weight=None, ignore_index=-100, reduction="mean"):
    """vocab_loss and the loss's gradients: (loss, row_loss, lse, dh, dw), dh and dw bf16."""
    import torch
    (desc, _, nb), loss, row, lse = _vocab_call(h, w, targets, row_weight, ignore_index, reduction)
    empty, bf16, device = torch.empty, torch.bfloat16, h.device
    dh, dw = empty(h.shape, dtype=bf16, device=device), empty(w.shape, dtype=bf16, device=device)
    ws = empty(nb, dtype=torch.uint8, device=device)
    _check("amsim_vocab_loss_grad",
           lib().amsim_vocab_loss_grad(desc, h.data_ptr(), w.data_ptr(), targets.data_ptr(), _at(row_weight),
                                       loss.data_ptr(), row.data_ptr(), lse.data_ptr(), dh.data_ptr(), dw.data_ptr(),
                                       ws.data_ptr(), nb, _current_stream()))
    return loss, row, lse, dh, dw


def adamw_table(tensors):
    """The table adamw_step takes, from AdamwTensor entries; it holds their addresses only, and their device."""
    tensors = list(tensors)
    devices = {t.device for t in tensors if hasattr(t, "device")}
    if len(devices) > 1:
        raise ValueError("the tensors of a table must be on one device")
    table = (AdamwTensor * len(tensors))(*tensors)
    table.device = devices.pop() if devices else None
    return table


def adamw_step(table, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, step, grad_scale=None):
    """One AdamW step over a table of tensors on the current device; `step` counts from 1, grad_scale is one fp32 CUDA
    value or None."""
    device, here = getattr(table, "device", None), _current_device()
    if grad_scale is not None:
        import torch
        _vector("grad_scale", grad_scale, 1, torch.float32, here)
    if device is not None and device != here:
        raise ValueError(f"the table's tensors are on cuda:{device}, the current device is cuda:{here}")
    amsim_adamw_step(table, AdamwHyper(lr, beta1, beta2, eps, step, _ptr(grad_scale)))


def adamw_moment_values(codes, scales):
    """fp32 values of an 8-bit moment's codes (int8: first moment, uint8: second), in the codes' shape."""
    import torch
    n, second = codes.numel(), codes.dtype == torch.uint8
    if not second and codes.dtype != torch.int8:
        raise TypeError("moment codes are int8 (first moment) or uint8 (second)")
    here = _current_device()
    _vector("codes", codes, n, codes.dtype, here)
    _vector("scales", scales, -(-n // AMSIM_ADAMW_BLOCK), torch.float32, here)
    out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
    _check("amsim_adamw_moment_values",
           lib().amsim_adamw_moment_values(codes.data_ptr(), scales.data_ptr(), 1 if second else 0, n, out.data_ptr(),
                                           _current_stream()))
    return out


# ------------------------------------------------------------------ between two contractions
def _drop(p, seed, call, step, here) -> DropoutDesc:
    if step is not None:
        import torch
        _vector("step", step, 1, torch.int64, here)
    return DropoutDesc(p, seed & 0xFFFFFFFFFFFFFFFF, call & 0xFFFFFFFFFFFFFFFF, _at(step))


def dropout(x, p, *, seed, call=0, step=None, residual=None):
    """residual + (x / (1 - p) where x stays, else 0), elements dropped with probability p.

    x: contiguous, fp32 or bf16, any shape; residual: alike, or None.  The mask is a function of (seed, call + step)
    and the element's place: the same numbers give the same mask, so dropout(dy, p, ...) is the gradient of x.  step: one
    int64 CUDA value or None, read when the kernel runs, so that a captured graph can draw another mask each time."""
    import torch
    here, n = _current_device(), x.numel()
    _vector("x", x, n, x.dtype, here)
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError(f"residual must be of x's shape {tuple(x.shape)}, not {tuple(residual.shape)}")
        _vector("residual", residual, n, x.dtype, here)
    y = torch.empty_like(x)
    _check("amsim_dropout",
           lib().amsim_dropout(ctypes.byref(_drop(p, seed, call, step, here)), _dtype(x), n, x.data_ptr(), _at(residual),
                               y.data_ptr(), _current_stream()))
    return y


def relative_buckets(buckets: int, max_distance: int, bidirectional: bool = True):
    """Bucket numbers of the distances -max_distance .. max_distance (key's position minus query's), an int32 CPU tensor.

    In both directions the first half of the buckets is for keys up to the query's place and the second for later ones;
    else all are for keys up to its place, and later ones share the first.  Half of a direction's buckets hold one
    distance each; the others' sizes grow by a constant factor up to max_distance, from which on all share the last."""
    import torch
    count = buckets // 2 if bidirectional else buckets
    near = count // 2
    if near < 1 or max_distance <= near or max_distance > AMSIM_MAX_DISTANCE:
        raise ValueError(f"relative_buckets: {buckets} buckets need a max_distance above {near} (and at least one near "
                         f"bucket each way), at most {AMSIM_MAX_DISTANCE}")
    steps = count - near

    def bucket(far):
        if far < near:
            return far
        k = 0                            # the last k with near (max_distance / near)^(k / steps) <= far, in whole numbers
        while k + 1 < steps and max_distance ** (k + 1) * near ** steps <= far ** steps * near ** (k + 1):
            k += 1
        return near + k
    up_to = [bucket(d) for d in range(max_distance, -1, -1)]
    later = [count + bucket(d) if bidirectional else 0 for d in range(1, max_distance + 1)]
    return torch.tensor(up_to + later, dtype=torch.int32)


def _score_rows(name, t, shape, here) -> int:
    """Row stride of a [batch, heads, queries, keys] tensor whose rows are evenly spaced and contiguous."""
    import torch
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != here:
        raise _elsewhere(name, t, here)
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be a CUDA tensor of torch.float32")
    if t.is_contiguous():
        return shape[3]
    b, h, q, k = shape
    outer, inner = t.stride()[:3], t.stride(3)
    ld = outer[2] if q > 1 else outer[1] if h > 1 else outer[0] if b > 1 else k
    want = (h * q * ld, q * ld, ld)
    if k > 1 and inner != 1 or ld < k or any(n > 1 and s != w for n, s, w in zip((b, h, q), outer, want)):
        raise ValueError(f"{name} must have contiguous rows, evenly spaced")
    return ld


def _softmax_call(shape, table, buckets, lengths, causal, offset, p, seed, call, step, here):
    """The descriptor of an attention softmax over checked arguments (without row strides)."""
    import torch
    b, h, q, k = shape
    d = AttentionSoftmaxDesc(batch=b, heads=h, queries=q, keys=k, causal=1 if causal else 0,
                             dropout=_drop(p, seed, call, step, here))
    if table is not None:
        if buckets is None:
            raise ValueError("a table of biases needs the buckets of its distances")
        if table.dim() != 2 or table.shape[1] != h or table.shape[0] < 1:
            raise ValueError(f"table must be buckets x {h} heads, not {tuple(table.shape)}")
        _vector("table", table, table.numel(), torch.float32, here)
        d.num_buckets = table.shape[0]
    if buckets is not None:
        if buckets.numel() % 2 != 1:
            raise ValueError("buckets must hold an odd number of values, from distance -D to D")
        _vector("buckets", buckets, buckets.numel(), torch.int32, here)
        d.max_distance = buckets.numel() // 2
    if lengths is not None:
        _vector("lengths", lengths, b, torch.int32, here)
        d.lengths = lengths.data_ptr()
    if hasattr(offset, "data_ptr"):
        _vector("offset", offset, b, torch.int32, here)
        d.offsets = offset.data_ptr()
    else:
        d.offset = operator.index(offset)
        if abs(offset) > 1 << 40:                # a field of 64 bits would keep some of it
            raise ValueError(f"offset must be within 2^40, not {offset}")
    return d


def attention_softmax(scores, *, table=None, buckets=None, lengths=None, causal=False, offset=0, p=0.0, seed=0, call=0,
                      step=None, out=None):
    """Softmax over the keys of scores [batch, heads, queries, keys] fp32: (probs, stats).

    table [num_buckets, heads] fp32 and buckets (int32, 2 D + 1 values, see relative_buckets): a bias by the distance
    between key and query, added to the scores.  lengths (int32 [batch]): keys from there on are not seen.  causal: keys
    after the query's position are not seen.  offset: the position of the first query, an int or an int32 tensor
    [batch] (a single token's place in its cache).  A row that sees no key is zeros.  p, seed, call, step: dropout of
    the probabilities, as in dropout().  out: the tensor to write, which may be scores.
    stats [batch, heads, queries, 2] is what attention_softmax_backward needs where p > 0."""
    import torch
    here = _current_device()
    if scores.dim() != 4:
        raise ValueError("scores must be [batch, heads, queries, keys]")
    shape = scores.shape
    ld = _score_rows("scores", scores, shape, here)
    if (table is None) != (buckets is None):
        raise ValueError("a bias needs both its table and the buckets of its distances")
    d = _softmax_call(shape, table, buckets, lengths, causal, offset, p, seed, call, step, here)
    d.ld_scores = ld
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=scores.device)
    else:
        d.ld_probs = _score_rows("out", out, shape, here)
    stats = torch.empty((*shape[:3], 2), dtype=torch.float32, device=scores.device)
    _check("amsim_attention_softmax_fwd",
           lib().amsim_attention_softmax_fwd(ctypes.byref(d), scores.data_ptr(), _at(table), _at(buckets),
                                             out.data_ptr(), stats.data_ptr(), _current_stream()))
    if stats.numel() and not shape[3]:       # rows without keys
        stats[..., 0], stats[..., 1] = -float("inf"), 0.0
    return out, stats


def attention_softmax_backward(dprobs, *, probs=None, scores=None, stats=None, table=None, buckets=None, lengths=None,
                               causal=False, offset=0, p=0.0, seed=0, call=0, step=None, table_grad=True, out=None):
    """Gradients of attention_softmax: (dscores, dtable), dtable None without a table or with table_grad false.

    Without dropout from probs, the forward pass's output; with dropout from the scores and stats it was given and
    left.  The other arguments are the forward pass's.  out: the tensor to write, which may be dprobs, probs or scores."""
    import torch
    here = _current_device()
    if dprobs.dim() != 4:
        raise ValueError("dprobs must be [batch, heads, queries, keys]")
    shape = dprobs.shape
    ld = _score_rows("dprobs", dprobs, shape, here)
    if (probs is None) == (scores is None) or (scores is None) != (stats is None):
        raise ValueError("the gradient is taken from probs, or from scores with their stats")
    if probs is not None and p > 0.0:
        raise ValueError("with dropout the gradient needs the scores and stats: dropped probabilities are gone")
    d = _softmax_call(shape, table, buckets, lengths, causal, offset, p, seed, call, step, here)
    d.ld_dprobs = ld
    if probs is not None:
        d.ld_probs = _score_rows("probs", probs, shape, here)
    else:
        d.ld_scores = _score_rows("scores", scores, shape, here)
        _vector("stats", stats, 2 * shape[0] * shape[1] * shape[2], torch.float32, here)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dprobs.device)
    else:
        d.ld_dscores = _score_rows("out", out, shape, here)
    dtable = torch.empty_like(table) if table is not None and table_grad else None
    nb = amsim_attention_softmax_workspace_size(d) if dtable is not None else 0
    ws = torch.empty(nb, dtype=torch.uint8, device=dprobs.device) if nb else None
    _check("amsim_attention_softmax_bwd",
           lib().amsim_attention_softmax_bwd(ctypes.byref(d), dprobs.data_ptr(), _at(scores), _at(stats), _at(probs),
                                             None if probs is not None else _at(table), _at(buckets), out.data_ptr(),
                                             _at(dtable), _at(ws), nb, _current_stream()))
    return out, dtable


def _pixels(name, t, here, shape=None) -> int:
    """Pixel stride of a [batch, ..., channels] tensor whose pixels are evenly spaced and their channels contiguous."""
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be of shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != here:
        raise _elsewhere(name, t, here)
    c = t.shape[-1]
    if t.is_contiguous():
        return c
    strides = t.stride()
    ld, at = None, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(strides[:-1])):
        if n > 1:
            ld = s // at if ld is None else ld
            if s != ld * at:
                ld = -1
        at *= n
    ld = c if ld is None else ld
    if c > 1 and strides[-1] != 1 or ld < c:
        raise ValueError(f"{name} must have contiguous channels and evenly spaced pixels")
    return ld


@functools.lru_cache(maxsize=1024)
def _group_norm_plan(batch, pixels, channels, groups, x, y, activation, eps, lddx, which):
    """(descriptor by reference, scratch bytes); x, y: (type, pixel stride)."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, not {activation!r}")
    d = GroupNormDesc(batch=batch, pixels=pixels, channels=channels, groups=groups, x_type=x[0], ldx=x[1], y_type=y[0],
                      ldy=y[1], lddx=lddx, activation=ACTIVATIONS[activation], eps=eps)
    return ctypes.byref(d), amsim_group_norm_workspace_size(d, which)


def _norm_shape(x, groups, w, b, here):
    import torch
    if x.dim() < 2:
        raise ValueError("group norms take [batch, ..., channels]")
    batch, channels = x.shape[0], x.shape[-1]
    if groups < 1 or channels < 1 or channels % groups:
        raise ValueError(f"{groups} groups do not divide {channels} channels")
    if w is not None:
        _vector("w", w, channels, torch.float32, here)
    if b is not None:
        _vector("b", b, channels, torch.float32, here)
    pixels = 1
    for n in x.shape[1:-1]:
        pixels *= n
    return batch, pixels, channels


def group_norm(x, groups, w=None, b=None, *, eps=1e-5, activation="none", y_dtype=None):
    """y = act(xh w + b), xh = x normalised over each group of a sample's channels and all its pixels: (y, mean, rstd).

    x: [batch, ..., channels] fp32 or bf16, channels last; w, b: [channels] fp32, or None (ones, zeros); activation:
    "none", "relu" or "silu"; y has x's shape and type `y_dtype` (x's).  mean, rstd: [batch, groups] fp32."""
    import torch
    here = _current_device()
    batch, pixels, channels = _norm_shape(x, groups, w, b, here)
    empty, device = torch.empty, x.device
    xs = (_dtype(x), _pixels("x", x, here))
    y = empty(x.shape, dtype=y_dtype or x.dtype, device=device)
    desc, nb = _group_norm_plan(batch, pixels, channels, groups, xs, (_dtype(y), 0), activation, eps, 0, 0)
    mean, rstd = (empty((batch, groups), dtype=torch.float32, device=device) for _ in range(2))
    ws = empty(nb, dtype=torch.uint8, device=device) if nb else None
    _check("amsim_group_norm_fwd",
           lib().amsim_group_norm_fwd(desc, x.data_ptr(), _at(w), _at(b), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                      _at(ws), nb, _current_stream()))
    return y, mean, rstd


def group_norm_backward(dy, x, w, b, mean, rstd, *, activation="none"):
    """Gradients of group_norm: (dx, dw, db), None where there was no such input.  mean and rstd are group_norm's."""
    import torch
    here = _current_device()
    if mean.dim() != 2:
        raise ValueError("mean must be [batch, groups]")
    groups = mean.shape[1]
    batch, pixels, channels = _norm_shape(x, groups, w, b, here)
    _vector("mean", mean, batch * groups, torch.float32, here)
    _vector("rstd", rstd, batch * groups, torch.float32, here)
    xs, ys = (_dtype(x), _pixels("x", x, here)), (_dtype(dy), _pixels("dy", dy, here, x.shape))
    empty, device = torch.empty, x.device
    desc, nb = _group_norm_plan(batch, pixels, channels, groups, xs, ys, activation, 0.0, 0, 1)
    dx = empty(x.shape, dtype=x.dtype, device=device)
    dw = None if w is None else torch.empty_like(w)
    db = None if b is None else torch.empty_like(b)
    ws = empty(nb, dtype=torch.uint8, device=device) if nb else None
    _check("amsim_group_norm_bwd",
           lib().amsim_group_norm_bwd(desc, dy.data_ptr(), x.data_ptr(), _at(w), _at(b), mean.data_ptr(),
                                      rstd.data_ptr(), dx.data_ptr(), _at(dw), _at(db), _at(ws), nb, _current_stream()))
    return dx, dw, db
