"""INT8 ConvRot linear layer for NVIDIA B200 (sm_100a).

Python binding of libconvrot (include/convrot.h). Each function has the name
of the C entry point it calls and only marshals arguments: torch tensors are
passed as device pointers, the current CUDA stream as the stream. Outputs and
workspaces that the caller does not pass are allocated with torch (the
library itself never allocates). Every computation runs in the library's
CUDA kernels; there is no CPU path.

    Wq, s_w = convrot_prepare_weight(W, g=256)         # once per layer
    Y = convrot_linear(X, Wq, s_w, g=256, bias=b)     # per call
"""

from __future__ import annotations

import functools

from . import _lib

__all__ = [
    "ConvRotError",
    "convrot_abi_version",
    "convrot_status_string",
    "convrot_prepare_weight",
    "convrot_quant_act",
    "convrot_linear_workspace_bytes",
    "convrot_linear",
    "convrot_linear_one_launch",
    "convrot_prepare_weight_ex",
    "convrot_quant_act_ex",
    "convrot_linear_ex",
    "DTYPE_BF16",
    "DTYPE_F16",
    "WSCALE_TENSOR",
    "WSCALE_CHANNEL",
    "ACT_NONE",
    "ACT_GELU_ERF",
    "convrot_gemm_dequant",
    "convrot_gemm_s32",
    "convrot_read_device_status",
    "convrot_test_wait_timeout",
    "convrot_probe_i8_peak",
    "convrot_attention_workspace_bytes",
    "convrot_attention_int8",
    "convrot_rope_tables",
    "convrot_rope",
    "convrot_cache_append",
    "convrot_cache_read",
    "convrot_cache_attention_workspace_bytes",
    "convrot_cache_attention",
    "ConvRotCache",
    "ConvRotLinear",
    "lib",
]

# convrot_dtype, convrot_wscale_mode, convrot_activation, convrot_pos_dtype (include/convrot.h)
DTYPE_BF16, DTYPE_F16 = 0, 1
WSCALE_TENSOR, WSCALE_CHANNEL = 0, 1
ACT_NONE, ACT_GELU_ERF = 0, 1
POS_I32, POS_F32 = 0, 1

STATUS_NAMES = {0: "CONVROT_OK", 1: "CONVROT_ERR_INVALID_ARG", 2: "CONVROT_ERR_UNSUPPORTED",
                3: "CONVROT_ERR_WORKSPACE", 4: "CONVROT_ERR_CUDA", 5: "CONVROT_ERR_DEVICE_TIMEOUT"}


class ConvRotError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({convrot_status_string(status)})")


def lib():
    """The loaded ctypes library (raises ImportError if it is not built)."""
    return _lib.load()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise ConvRotError(status, where)


def _stream_ptr(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(t, dtype, shape, name):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def convrot_abi_version() -> int:
    return int(lib().convrot_abi_version())


def convrot_status_string(status: int) -> str:
    return lib().convrot_status_string(int(status)).decode()


def convrot_prepare_weight(W, g: int = 256, Wq=None, w_scale=None, ws=None, stream=None):
    """Rotate and quantise a bf16 weight [N,K]: returns (Wq int8 [N,K], w_scale float32 [1])."""
    import torch

    _require(W, torch.bfloat16, None, "W")
    N, K = W.shape
    if Wq is None:
        Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if w_scale is None:
        w_scale = torch.empty((1,), dtype=torch.float32, device=W.device)
    L = lib()
    if ws is None:
        ws = torch.empty((L.convrot_prepare_weight_workspace_bytes(),), dtype=torch.uint8, device=W.device)
    _require(Wq, torch.int8, (N, K), "Wq")
    _require(w_scale, torch.float32, (1,), "w_scale")
    _check(L.convrot_prepare_weight(_ptr(W), N, K, g, _ptr(Wq), _ptr(w_scale), _ptr(ws), ws.numel(),
                                    _stream_ptr(stream)), "convrot_prepare_weight")
    return Wq, w_scale


def convrot_quant_act(X, g: int = 256, Xq=None, x_scale=None, stream=None):
    """Rotate + per-token quantise bf16 X [M,K]: returns (Xq int8 [M,K], x_scale float32 [M])."""
    import torch

    _require(X, torch.bfloat16, None, "X")
    M, K = X.shape
    if Xq is None:
        Xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if x_scale is None:
        x_scale = torch.empty((M,), dtype=torch.float32, device=X.device)
    _require(Xq, torch.int8, (M, K), "Xq")
    _require(x_scale, torch.float32, (M,), "x_scale")
    _check(lib().convrot_quant_act(_ptr(X), M, K, g, _ptr(Xq), _ptr(x_scale), _stream_ptr(stream)),
           "convrot_quant_act")
    return Xq, x_scale


def convrot_linear_workspace_bytes(M: int, N: int, K: int, g: int) -> int:
    return int(lib().convrot_linear_workspace_bytes(M, N, K, g))


def convrot_linear(X, Wq, w_scale, g: int = 256, bias=None, Y=None, ws=None, stream=None):
    """Y [M,N] bf16 = ConvRot linear of bf16 X [M,K] with the prepared weight (Wq, w_scale)."""
    import torch

    _require(X, torch.bfloat16, None, "X")
    M, K = X.shape
    _require(Wq, torch.int8, None, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Wq must be [N, K] with the K of X")
    _require(w_scale, torch.float32, (1,), "w_scale")
    if bias is not None:
        _require(bias, torch.bfloat16, (N,), "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    need = convrot_linear_workspace_bytes(M, N, K, g)
    if ws is None:
        ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=X.device)
    _check(lib().convrot_linear(_ptr(X), M, K, g, _ptr(Wq), _ptr(w_scale), N, _ptr(bias), _ptr(Y), _ptr(ws),
                                ws.numel(), _stream_ptr(stream)), "convrot_linear")
    return Y


def convrot_linear_one_launch(X, Wq, w_scale, g: int = 256, bias=None, Y=None, ws=None, stream=None):
    """convrot_linear as one kernel launch (rotate+quantise workers inside the GEMM kernel; K <= 20480)."""
    import torch

    _require(X, torch.bfloat16, None, "X")
    M, K = X.shape
    _require(Wq, torch.int8, None, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Wq must be [N, K] with the K of X")
    _require(w_scale, torch.float32, (1,), "w_scale")
    if bias is not None:
        _require(bias, torch.bfloat16, (N,), "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    need = convrot_linear_workspace_bytes(M, N, K, g)
    if ws is None:
        ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=X.device)
    _check(lib().convrot_linear_one_launch(_ptr(X), M, K, g, _ptr(Wq), _ptr(w_scale), N, _ptr(bias), _ptr(Y),
                                           _ptr(ws), ws.numel(), _stream_ptr(stream)), "convrot_linear_one_launch")
    return Y


def _dtype_code(t, name):
    import torch

    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float16:
        return DTYPE_F16
    raise TypeError(f"{name}: expected bfloat16 or float16, got {t.dtype}")


def convrot_prepare_weight_ex(W, g: int = 256, wscale_mode: int = WSCALE_TENSOR, Wq=None, w_scale=None, ws=None,
                              stream=None):
    """Rotate and quantise a bf16 or fp16 weight [N,K]: returns (Wq int8 [N,K], w_scale float32 [1] or [N])."""
    import torch

    dtype = _dtype_code(W, "W")
    _require(W, W.dtype, None, "W")
    N, K = W.shape
    ns = N if wscale_mode == WSCALE_CHANNEL else 1
    if Wq is None:
        Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if w_scale is None:
        w_scale = torch.empty((ns,), dtype=torch.float32, device=W.device)
    L = lib()
    if ws is None and wscale_mode != WSCALE_CHANNEL:
        ws = torch.empty((L.convrot_prepare_weight_workspace_bytes(),), dtype=torch.uint8, device=W.device)
    _require(Wq, torch.int8, (N, K), "Wq")
    _require(w_scale, torch.float32, (ns,), "w_scale")
    _check(L.convrot_prepare_weight_ex(_ptr(W), dtype, N, K, g, int(wscale_mode), _ptr(Wq), _ptr(w_scale), _ptr(ws),
                                       0 if ws is None else ws.numel(), _stream_ptr(stream)),
           "convrot_prepare_weight_ex")
    return Wq, w_scale


def _rows_view(t, name):
    """(rows, cols, row stride in elements) of a 2-D tensor whose rows may be strided."""
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    return t.shape[0], t.shape[1], t.stride(0)


def convrot_quant_act_ex(X, g: int = 256, Xq=None, x_scale=None, stream=None):
    """convrot_quant_act for a bf16 or fp16 X [M,K] whose rows may be strided."""
    import torch

    dtype = _dtype_code(X, "X")
    M, K, ldx = _rows_view(X, "X")
    if Xq is None:
        Xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if x_scale is None:
        x_scale = torch.empty((M,), dtype=torch.float32, device=X.device)
    _require(Xq, torch.int8, (M, K), "Xq")
    _require(x_scale, torch.float32, (M,), "x_scale")
    _check(lib().convrot_quant_act_ex(_ptr(X), dtype, M, K, ldx, g, _ptr(Xq), _ptr(x_scale), _stream_ptr(stream)),
           "convrot_quant_act_ex")
    return Xq, x_scale


def convrot_linear_ex(X, Wq, w_scale, g: int = 256, bias=None, activation: int = ACT_NONE, Y=None, ws=None,
                      stream=None, addend=None):
    """ConvRot linear in the dtype of X (bf16 or fp16; bias, addend and Y the same), with a
    tensor (w_scale [1]) or per-output-channel (w_scale [N]) weight scale, an optional
    addend [M,N] (a term computed beside the int8 layer, e.g. a LoRA's output) and an
    optional exact-erf GELU. X, Y and addend may have strided rows (Y and addend share
    one row stride)."""
    import torch

    dtype = _dtype_code(X, "X")
    M, K, ldx = _rows_view(X, "X")
    _require(Wq, torch.int8, None, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Wq must be [N, K] with the K of X")
    if w_scale.numel() == N and N != 1:
        mode = WSCALE_CHANNEL
    elif w_scale.numel() == 1:
        mode = WSCALE_TENSOR
    else:
        raise ValueError("w_scale must hold 1 or N floats")
    _require(w_scale, torch.float32, (w_scale.numel(),), "w_scale")
    if bias is not None:
        _require(bias, X.dtype, (N,), "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if Y.dtype != X.dtype or tuple(Y.shape) != (M, N):
        raise ValueError(f"Y must be [{M}, {N}] {X.dtype}")
    _, _, ldy = _rows_view(Y, "Y")
    if addend is not None:
        if addend.dtype != X.dtype or tuple(addend.shape) != (M, N) or _rows_view(addend, "addend")[2] != ldy:
            raise ValueError("addend must be [M, N] in the dtype of X, with the row stride of Y")
    need = convrot_linear_workspace_bytes(M, N, K, g)
    if ws is None:
        ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=X.device)
    _check(lib().convrot_linear_ex(_ptr(X), dtype, M, K, ldx, g, _ptr(Wq), _ptr(w_scale), mode, N, _ptr(bias),
                                   _ptr(addend), int(activation), _ptr(Y), ldy, _ptr(ws), ws.numel(),
                                   _stream_ptr(stream)), "convrot_linear_ex")
    return Y


def convrot_gemm_dequant(Xq, x_scale, Wq, w_scale, bias=None, Y=None, ws=None, stream=None):
    """GEMM + epilogue on already-quantised codes: Y [M,N] bf16."""
    import torch

    _require(Xq, torch.int8, None, "Xq")
    M, K = Xq.shape
    _require(Wq, torch.int8, None, "Wq")
    N = Wq.shape[0]
    _require(x_scale, torch.float32, (M,), "x_scale")
    _require(w_scale, torch.float32, (1,), "w_scale")
    if bias is not None:
        _require(bias, torch.bfloat16, (N,), "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    L = lib()
    if ws is None:
        ws = torch.empty((L.convrot_gemm_workspace_bytes(),), dtype=torch.uint8, device=Xq.device)
    _check(L.convrot_gemm_dequant(_ptr(Xq), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, K, _ptr(bias), _ptr(Y),
                                  _ptr(ws), ws.numel(), _stream_ptr(stream)), "convrot_gemm_dequant")
    return Y


def convrot_gemm_s32(Xq, Wq, acc=None, ws=None, stream=None):
    """Raw int32 accumulators acc [M,N] = Xq Wq^T from the tcgen05 GEMM."""
    import torch

    _require(Xq, torch.int8, None, "Xq")
    M, K = Xq.shape
    _require(Wq, torch.int8, None, "Wq")
    N = Wq.shape[0]
    if acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=Xq.device)
    _require(acc, torch.int32, (M, N), "acc")
    L = lib()
    if ws is None:
        ws = torch.empty((L.convrot_gemm_workspace_bytes(),), dtype=torch.uint8, device=Xq.device)
    _check(L.convrot_gemm_s32(_ptr(Xq), _ptr(Wq), M, N, K, _ptr(acc), _ptr(ws), ws.numel(), _stream_ptr(stream)),
           "convrot_gemm_s32")
    return acc


def convrot_read_device_status(ws, stream=None) -> int:
    """Status word of a workspace (synchronises the stream): 0 or CONVROT_ERR_DEVICE_TIMEOUT (5)."""
    return int(lib().convrot_read_device_status(_ptr(ws), _stream_ptr(stream)))


def convrot_test_wait_timeout(ws, timeout_ns: int, stream=None) -> None:
    _check(lib().convrot_test_wait_timeout(_ptr(ws), ws.numel(), int(timeout_ns), _stream_ptr(stream)),
           "convrot_test_wait_timeout")


def convrot_probe_i8_peak(iters: int, operands=None, ws=None, stream=None) -> int:
    """Enqueue the int8 tensor-pipe peak probe (one CTA pair per two SMs, `iters` x 4
    tcgen05.mma.cta_group::2.kind::i8 of 256x256x32 each, no global traffic in the loop);
    returns the number of CTAs launched. `operands`: None (zero operands) or a contiguous
    device tensor whose bytes fill the CTAs' operand tiles. The caller times it with
    events on `stream`."""
    import torch

    L = lib()
    if ws is None:
        ws = torch.empty((256,), dtype=torch.uint8, device=torch.cuda.current_device())
    op_ptr, op_bytes = None, 0
    if operands is not None:
        if not operands.is_contiguous():
            raise ValueError("operands must be contiguous")
        op_ptr, op_bytes = _ptr(operands), operands.numel() * operands.element_size()
    _check(L.convrot_probe_i8_peak(int(iters), op_ptr, op_bytes, _ptr(ws), ws.numel(), _stream_ptr(stream)),
           "convrot_probe_i8_peak")
    return int(L.convrot_probe_i8_peak_ctas())


def convrot_attention_workspace_bytes(BH: int, Sq: int, Skv: int, D: int = 128) -> int:
    return int(lib().convrot_attention_workspace_bytes(BH, Sq, Skv, D))


def convrot_attention_int8(Q, K, V, softmax_scale=None, O=None, ws=None, stream=None):
    """INT8 attention of bf16 Q [..., Sq, 128] with K, V [..., Skv, 128] (same leading
    dims, flattened to batch*heads): O [..., Sq, 128] bf16 (see include/convrot.h)."""
    import math

    import torch

    for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
        _require(t, torch.bfloat16, None, name)
        if t.dim() < 2 or t.shape[-1] != 128:
            raise ValueError(f"{name} must be [..., S, 128]")
    lead = tuple(Q.shape[:-2])
    if tuple(K.shape[:-2]) != lead or tuple(V.shape) != tuple(K.shape):
        raise ValueError("Q, K and V must share their leading dimensions, and K and V their shape")
    Sq, Skv, D = Q.shape[-2], K.shape[-2], Q.shape[-1]
    BH = int(math.prod(lead)) if lead else 1
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16, device=Q.device)
    _require(O, torch.bfloat16, tuple(Q.shape), "O")
    need = convrot_attention_workspace_bytes(BH, Sq, Skv, D)
    if ws is None:
        ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=Q.device)
    _check(lib().convrot_attention_int8(_ptr(Q), _ptr(K), _ptr(V), BH, Sq, Skv, D, float(softmax_scale), _ptr(O),
                                        _ptr(ws), ws.numel(), _stream_ptr(stream)), "convrot_attention_int8")
    return O


class _Torch:
    """What the calls below use of torch, bound at the first of them: a call of a few microseconds
    notices every import statement and attribute on its way."""

    def __getattr__(self, name):
        import torch

        self.module = torch
        self.code = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
        self.int8, self.int32, self.int64, self.uint8 = torch.int8, torch.int32, torch.int64, torch.uint8
        self.float32, self.float64 = torch.float32, torch.float64
        self.dense = torch.contiguous_format
        self.empty_like, self.empty = torch.empty_like, torch.empty
        self.grad = torch.is_grad_enabled
        self.device = torch._C._cuda_getDevice
        self.stream = torch._C._cuda_getCurrentRawStream  # a Stream object costs ten times as much
        # the native forms of the calls; they return None where the Python form has to see to a call
        native = _lib.binding()
        self.rope, self.append, self.read, self.attention = (
            (native.rope, native.append, native.read, native.attention) if native else (lambda *a: None,) * 4)
        return object.__getattribute__(self, name)


_T = _Torch()


def _elsewhere(index: int, stream):
    """None if a call on tensors of device `index` runs where torch is: that device current, its
    current stream. Otherwise a context that makes it so, within which buffers are allocated
    for the stream that uses them."""
    here = _T.device() == index
    torch = _T.module
    if stream is None:
        return None if here else torch.cuda.device(index)
    ptr = _stream_ptr(stream)
    if here and ptr == _T.stream(index):
        return None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(ptr, device=index) if ptr else torch.cuda.default_stream(index)
    elif stream.device_index != index:
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


def _beside(t, name, index, dtype, shape):
    """Checks a contiguous tensor argument of the given type and shape on device `index`; its address."""
    if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _head_vectors(t, name, dims=(3,)):
    """(type code, device, shape, strides) of bf16 or fp16 head vectors [..., heads, D] on a GPU whose
    channels are contiguous."""
    code = _T.code.get(t.dtype)
    index, shape, strides = t.get_device(), t.shape, t.stride()
    if code is not None and index >= 0 and len(shape) in dims and (strides[-1] == 1 or shape[-1] <= 1):
        return code, index, shape, strides
    if code is None:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {t.dtype}")
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    if len(shape) not in dims:
        raise ValueError(f"{name}: expected {' or '.join(str(d) for d in dims)} dimensions, got {len(shape)}")
    raise ValueError(f"{name}: the channels of a head must be contiguous")


def _output(t, name, code, index, shape):
    """The strides of an output that must be head vectors of this type, device and shape, each
    element at an address of its own."""
    code_t, index_t, shape_t, strides = _head_vectors(t, name, (len(shape),))
    if code_t != code or index_t != index or shape_t != shape:
        raise ValueError(f"{name} must be {tuple(shape)} in the dtype and on the device of the other tensors")
    if 0 in strides and any(n > 1 and st == 0 for n, st in zip(shape, strides)):
        raise ValueError(f"{name} must not be an expanded tensor")
    return strides


def _written(t):
    """Tells autograd that a tensor of the caller's has been written, as torch's own operations do."""
    if not t.is_inference():
        _T.module.autograd.graph.increment_version(t)


def _refused(status, where, **vectors):
    """The error of a call on head vectors, with the one that the kernels cannot take, if it is that."""
    for name, t in vectors.items():
        if status == 1 and (t.data_ptr() % 16 or any(st % 8 for n, st in zip(t.shape[:-1], t.stride()) if n > 1)):
            where = f"{where}: {name} must start on 16 bytes, with strides that are multiples of 8 elements"
    return ConvRotError(status, where)


def convrot_rope_tables(sections, theta: float = 10000.0, shared: bool = False, device="cuda"):
    """The tables of convrot_rope for axes with sections[a] pairs of channels each, in order:
    (freq float64, axis int32), both [sum(sections)]. Each axis has its own ladder
    theta^(-i / sections[a]), or, `shared`, pair i of all n takes theta^(-i / n)."""
    import torch

    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0 or not theta > 0:
        raise ValueError("sections must be non-negative counts of pairs, theta positive")
    n = sum(sections)
    power = [i / n for i in range(n)] if shared else [i / m for m in sections for i in range(m)]
    axis = [a for a, m in enumerate(sections) for _ in range(m)]
    freq = torch.tensor([float(theta) ** -p for p in power], dtype=torch.float64, device=device)
    return freq, torch.tensor(axis, dtype=torch.int32, device=device)


def convrot_rope(X, positions, freq, axis, interleaved: bool = False, inverse: bool = False, Y=None, stream=None):
    """Rotary positions with several axes: X [B, S, H, D] or [S, H, D] (bf16 or fp16, any
    strides, channels contiguous) with the pairs of its first 2 * len(freq) channels turned by
    positions[axis[i]] * freq[i]. positions [axes, S] or [axes, B, S], int32 or float32;
    freq float64 (radians), axis int32. `inverse` turns back, which is also the gradient.
    Y: an output of X's shape and any strides (X itself works in place); with
    Y = buf.transpose(-3, -2) the heads come out as convrot_attention_int8 takes them.
    Recorded by autograd for X, in place and into Y too; positions and freq take no gradient."""
    if stream is None:
        done = _T.rope(X, positions, freq, axis, interleaved, inverse, Y)
        if done is not None:
            return done
    code, index, shape, xs = _head_vectors(X, "X", (3, 4))
    if stream is not None or _T.device() != index:
        where = _elsewhere(index, stream)
        if where is not None:
            with where:
                return convrot_rope(X, positions, freq, axis, interleaved, inverse, Y)
    if _T.grad() and (X.requires_grad or positions.requires_grad or freq.requires_grad
                      or (Y is not None and Y.requires_grad)):
        return _recorded_rope(X, positions, freq, axis, interleaved, inverse, Y)
    if len(shape) == 4:
        B, S, H, D = shape
    else:
        (S, H, D), B, xs = shape, 1, (0, *xs)
    pairs = freq.numel()
    if 2 * pairs > D:
        raise ValueError(f"freq holds {pairs} pairs, a head vector {D} channels")
    freq_ptr = _beside(freq, "freq", index, _T.float64, (pairs,))
    axis_ptr = _beside(axis, "axis", index, _T.int32, (pairs,))
    ptype, pshape, ps = positions.dtype, positions.shape, positions.stride()
    if ptype is _T.int32:
        pos_code = POS_I32
    elif ptype is _T.float32:
        pos_code = POS_F32
    else:
        raise TypeError(f"positions: expected int32 or float32, got {ptype}")
    if positions.get_device() != index:
        raise ValueError("positions must be on the device of the other tensors")
    if len(pshape) == 2:
        pb = 0
    elif len(pshape) == 3 and pshape[1] == B:
        pb = ps[1]
    else:
        pb = None
    if pb is None or pshape[0] < 1 or pshape[-1] != S:
        raise ValueError(f"positions: expected [axes, {S}] or [axes, {B}, {S}], got {tuple(pshape)}")
    given = Y is not None
    if not given:
        Y = _T.empty_like(X, memory_format=_T.dense)
        yb, ys, yh = S * H * D, H * D, D
    else:
        yt = _output(Y, "Y", code, index, shape)
        yb, ys, yh = yt[:3] if len(yt) == 4 else (0, yt[0], yt[1])
    args = _lib.ROPE_ARGS.pack(X.data_ptr(), Y.data_ptr(), positions.data_ptr(), freq_ptr, axis_ptr, B, S, H, D,
                               2 * pairs, xs[0], xs[1], xs[2], yb, ys, yh, pshape[0], ps[0], pb, ps[-1], code, pos_code,
                               interleaved, inverse)
    status = (_lib._lib or lib()).convrot_rope(args, _T.stream(index))
    if status != 0:
        raise ConvRotError(status, "convrot_rope")
    if given:
        _written(Y)
    return Y


@functools.lru_cache(maxsize=1)
def _rope_function():
    import torch

    class Rope(torch.autograd.Function):
        # Y, the tensor written in place, comes first, as autograd has it of views; X is None where Y is turned itself
        @staticmethod
        def forward(ctx, Y, X, positions, freq, axis, interleaved, inverse):
            ctx.save_for_backward(positions, freq, axis)
            ctx.turn = interleaved, inverse
            ctx.in_place = X is None
            out = convrot_rope(Y if X is None else X, positions, freq, axis, interleaved, inverse, Y)
            if Y is not None:
                ctx.mark_dirty(out)
            return out

        @staticmethod
        def backward(ctx, dY):
            interleaved, inverse = ctx.turn
            dX = old = None
            if ctx.needs_input_grad[0 if ctx.in_place else 1]:
                rows = dY if dY.stride(-1) == 1 else dY.contiguous()
                dX = convrot_rope(rows, *ctx.saved_tensors, interleaved, not inverse)
            if ctx.in_place:
                old, dX = dX, None
            elif ctx.needs_input_grad[0]:
                old = torch.zeros_like(dY)  # what Y held before is gone
            return (old, dX) + (None,) * 5

    return Rope


def _recorded_rope(X, positions, freq, axis, interleaved, inverse, Y):
    """convrot_rope where autograd follows X, or a Y that it has followed so far."""
    if positions.requires_grad or freq.requires_grad:
        raise ValueError("positions and freq take no gradient: detach them")
    if Y is not None and Y.requires_grad and (Y.is_leaf or (Y._is_view() and Y._base.is_leaf)):
        raise RuntimeError("Y is a leaf that requires grad, or a view of one: it cannot be written to in place")
    return _rope_function().apply(Y, None if Y is X else X, positions, freq, axis, interleaved, inverse)


def _cells(index, k_codes, v_codes, k_scale, v_scale):
    """The fields of convrot_cells for the four cache tensors on device `index`."""
    shape = k_codes.shape
    if len(shape) != 4 or shape[3] != 128:
        raise ValueError("k_codes must be [pages, heads, page size, 128]")
    pages, heads, page, _ = shape
    cells = (pages, heads, page)
    return (_beside(k_codes, "k_codes", index, _T.int8, shape), _beside(v_codes, "v_codes", index, _T.int8, shape),
            _beside(k_scale, "k_scale", index, _T.float32, cells), _beside(v_scale, "v_scale", index, _T.float32, cells),
            pages, heads, page, 128)


def convrot_cache_append(K, V, slots, k_codes, v_codes, k_scale, v_scale, status=None, stream=None):
    """Write keys and values K, V [T, H, 128] (bf16 or fp16, strided tokens and heads) into the
    rotated int8 cache: token t to slot slots[t] (int32; page * page size + place; negative: skipped;
    the others must differ). Cache: codes int8 [pages, H, page size, 128], scales float32 [pages, H,
    page size]. Head vectors here and below start on 16 bytes, their strides are multiples of 8. status: an int32 [1] tensor that a slot past the cache sets to 1, or None."""
    if stream is None and _T.append(K, V, slots, k_codes, v_codes, k_scale, v_scale, status):
        return
    code, index, shape, ks = _head_vectors(K, "K")
    if stream is not None or _T.device() != index:
        where = _elsewhere(index, stream)
        if where is not None:
            with where:
                return convrot_cache_append(K, V, slots, k_codes, v_codes, k_scale, v_scale, status)
    code_v, index_v, shape_v, vs = _head_vectors(V, "V")
    if code_v != code or index_v != index or shape_v != shape:
        raise ValueError("V must have the shape, dtype and device of K")
    T, H, D = shape
    cells = _cells(index, k_codes, v_codes, k_scale, v_scale)
    if cells[5] != H or D != 128:
        raise ValueError(f"K has {H} heads of {D} channels, the cache {cells[5]} of 128")
    slots_ptr = _beside(slots, "slots", index, _T.int32, (T,))
    status_ptr = 0 if status is None else _beside(status, "status", index, _T.int32, (1,))
    args = _lib.CACHE_ARGS.pack(*cells, K.data_ptr(), V.data_ptr(), slots_ptr, status_ptr, T, ks[0], ks[1], vs[0],
                                vs[1], code)
    status = (_lib._lib or lib()).convrot_cache_append(args, _T.stream(index))
    if status != 0:
        raise _refused(status, "convrot_cache_append", K=K, V=V)


def convrot_cache_read(slots, k_codes, v_codes, k_scale, v_scale, dtype=None, K=None, V=None, status=None,
                       stream=None):
    """Read the keys and values of slots [T] back: (K, V) [T, H, 128] in `dtype` (bf16 by default, or
    fp16); a negative slot reads as zeros. K, V: outputs with strided tokens and heads, or None."""
    if stream is None:
        want = dtype if dtype is not None else K.dtype if K is not None else V.dtype if V is not None else None
        code = DTYPE_BF16 if want is None else _T.code.get(want, -1)
        done = _T.read(slots, k_codes, v_codes, k_scale, v_scale, code, K, V, status)
        if done is not None:
            return done
    index = slots.get_device()
    if index < 0:
        raise ValueError("slots must be on a CUDA device")
    if stream is not None or _T.device() != index:
        where = _elsewhere(index, stream)
        if where is not None:
            with where:
                return convrot_cache_read(slots, k_codes, v_codes, k_scale, v_scale, dtype, K, V, status)
    T = slots.numel()
    slots_ptr = _beside(slots, "slots", index, _T.int32, (T,))
    cells = _cells(index, k_codes, v_codes, k_scale, v_scale)
    H = cells[5]
    if dtype is None:
        dtype = K.dtype if K is not None else V.dtype if V is not None else _T.module.bfloat16
    code = _T.code.get(dtype)
    if code is None:
        raise TypeError(f"dtype: expected bfloat16 or float16, got {dtype}")
    shape = (T, H, 128)
    ks = vs = (H * 128, 128)
    given = [t for t in (K, V) if t is not None]
    if K is not None:
        ks = _output(K, "K", code, index, shape)
    else:
        K = slots.new_empty(shape, dtype=dtype)
    if V is not None:
        vs = _output(V, "V", code, index, shape)
    else:
        V = _T.empty_like(K, memory_format=_T.dense)
    status_ptr = 0 if status is None else _beside(status, "status", index, _T.int32, (1,))
    args = _lib.CACHE_ARGS.pack(*cells, K.data_ptr(), V.data_ptr(), slots_ptr, status_ptr, T, ks[0], ks[1], vs[0],
                                vs[1], code)
    status = (_lib._lib or lib()).convrot_cache_read(args, _T.stream(index))
    if status != 0:
        raise _refused(status, "convrot_cache_read", K=K, V=V)
    for t in given:
        _written(t)
    return K, V


@functools.lru_cache(maxsize=1024)
def convrot_cache_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, D: int = 128) -> int:
    return int(lib().convrot_cache_attention_workspace_bytes(T, B, Hq, Hkv, D))


def convrot_cache_attention(Q, k_codes, v_codes, k_scale, v_scale, pages, lengths, starts=None, tree=None,
                            softmax_scale=None, O=None, ws=None, stream=None, status=None):
    """Attention of the newest tokens over the rotated int8 cache: Q [T, Hq, 128] (bf16 or fp16,
    strided tokens and heads) -> O [T, Hq, 128]. pages [B, n] int32: the cache pages of each sequence;
    lengths [B] int32: its keys, the new tokens' included; starts [B + 1] int32: its tokens in Q
    (None: token b belongs to sequence b). Among its new tokens a query sees the earlier ones and
    itself, or, with tree [T] int64, those whose bit is set in its mask (at most 64 a sequence).
    status: an int32 [1] tensor into which the call's status is ORed (1: a length, page or start was
    out of range; 5: a wait ran out and the rows it cost are NaN), or None. Nothing here is recorded
    by autograd. See include/convrot.h."""
    if stream is None:
        done = _T.attention(Q, k_codes, v_codes, k_scale, v_scale, pages, lengths, starts, tree, softmax_scale, O, ws,
                            status)
        if done is not None:
            return done
    code, index, shape, qs = _head_vectors(Q, "Q")
    if stream is not None or _T.device() != index:
        where = _elsewhere(index, stream)
        if where is not None:
            with where:
                return convrot_cache_attention(Q, k_codes, v_codes, k_scale, v_scale, pages, lengths, starts, tree,
                                               softmax_scale, O, ws, status=status)
    T, Hq, D = shape
    cells = _cells(index, k_codes, v_codes, k_scale, v_scale)
    Hkv = cells[5]
    if Hkv == 0 or Hq == 0 or Hq % Hkv != 0 or D != 128:
        raise ValueError(f"{Hq} query heads of {D} channels do not divide among {Hkv} key heads of 128")
    B = lengths.numel()
    lengths_ptr = _beside(lengths, "lengths", index, _T.int32, (B,))
    if pages.dtype is not _T.int32:
        raise TypeError(f"pages: expected torch.int32, got {pages.dtype}")
    pshape, ps = pages.shape, pages.stride()
    if len(pshape) != 2 or pshape[0] != B or (ps[1] != 1 and pshape[1] > 1) or pages.get_device() != index:
        raise ValueError(f"pages must be [{B}, n] with contiguous rows on the device of the other tensors")
    starts_ptr = tree_ptr = 0
    if starts is not None:
        starts_ptr = _beside(starts, "starts", index, _T.int32, (B + 1,))
    elif T != B:
        raise ValueError("without starts Q must hold one token per sequence")
    if tree is not None:
        tree_ptr = _beside(tree, "tree", index, _T.int64, (T,))
    if softmax_scale is None:
        softmax_scale = 0.08838834764831845  # 1 / sqrt(128)
    ot, oh = Hq * D, D
    given = O is not None
    if given:
        ot, oh, _ = _output(O, "O", code, index, shape)
    else:
        O = _T.empty_like(Q, memory_format=_T.dense)
    if ws is None:
        room = convrot_cache_attention_workspace_bytes(T, B, Hq, Hkv, D)
        ws = Q.new_empty(room if room > 256 else 256, dtype=_T.uint8)
    else:
        if ws.get_device() != index or not ws.is_contiguous():
            raise ValueError("ws must be contiguous on the device of the other tensors")
        room = ws.numel() * ws.element_size()
    status_ptr = 0 if status is None else _beside(status, "status", index, _T.int32, (1,))
    args = _lib.CACHE_ATTENTION_ARGS.pack(
        *cells, Q.data_ptr(), O.data_ptr(), pages.data_ptr(), lengths_ptr, starts_ptr, tree_ptr, ws.data_ptr(), room,
        T, Hq, B, pshape[1], ps[0], qs[0], qs[1], ot, oh, softmax_scale, code)
    status = (_lib._lib or lib()).convrot_cache_attention_ex(args, status_ptr, 0, _T.stream(index))
    if status != 0:
        raise _refused(status, "convrot_cache_attention", Q=Q, O=O)
    if given:
        _written(O)
    return O


class ConvRotCache:
    """A paged cache of rotated int8 keys and values for `heads` key/value heads of 128 channels.

    ``cache.append(K, V, slots)``, ``cache.read(slots)`` and ``cache.attention(Q, pages, lengths)`` are
    the entry points of the same names on its tensors; ``cache.slots(pages, sequence, position)`` finds
    the slots of tokens. ``check()`` synchronises and raises if a slot was past the cache, or an attention
    met a length, page or start out of range or a wait that ran out (``status.zero_()`` forgets it).
    """

    def __init__(self, num_pages: int, heads: int, page_size: int = 64, device="cuda"):
        import torch

        shape = (num_pages, heads, page_size)
        self.page_size = page_size
        self.k_codes = torch.zeros((*shape, 128), dtype=torch.int8, device=device)
        self.v_codes = torch.zeros((*shape, 128), dtype=torch.int8, device=device)
        self.k_scale = torch.zeros(shape, dtype=torch.float32, device=device)
        self.v_scale = torch.zeros(shape, dtype=torch.float32, device=device)
        self.status = torch.zeros((1,), dtype=torch.int32, device=device)

    @property
    def cells(self):
        return self.k_codes, self.v_codes, self.k_scale, self.v_scale

    def slots(self, pages, sequence, position):
        """Slots (int32) of the tokens at `position` of the sequences whose rows of `pages` are
        `sequence`; -1 where `pages` has no such place or no page for it. A page past the cache gives a
        slot past it, which the append reports."""
        import torch

        sequence, position = sequence.long(), position.long()
        if pages.numel() == 0:
            return torch.full(position.shape, -1, dtype=torch.int32, device=position.device)
        column = position // self.page_size
        page = pages[sequence.clamp(0, pages.shape[0] - 1), column.clamp(0, pages.shape[1] - 1)].long()
        there = ((sequence >= 0) & (sequence < pages.shape[0]) & (position >= 0) & (column < pages.shape[1])
                 & (page >= 0))
        slot = (page * self.page_size + position % self.page_size).clamp(max=2**31 - 1)
        return torch.where(there, slot, -1).to(torch.int32)

    def append(self, K, V, slots, stream=None):
        convrot_cache_append(K, V, slots, *self.cells, status=self.status, stream=stream)

    def read(self, slots, dtype=None, K=None, V=None, stream=None):
        return convrot_cache_read(slots, *self.cells, dtype=dtype, K=K, V=V, status=self.status, stream=stream)

    def attention(self, Q, pages, lengths, starts=None, tree=None, softmax_scale=None, O=None, ws=None, stream=None):
        return convrot_cache_attention(Q, *self.cells, pages, lengths, starts, tree, softmax_scale, O, ws, stream,
                                       self.status)

    def check(self):
        if int(self.status.item()) != 0:
            raise ConvRotError(int(self.status.item()), "ConvRotCache")


class ConvRotLinear:
    """A ConvRot linear layer: prepared int8 weight + optional bias, reusable workspace.

    ``layer = ConvRotLinear(W, bias, g=256)`` rotates and quantises W once;
    ``layer(X)`` runs convrot_linear on the current stream. With a float16 W,
    ``wscale_mode=WSCALE_CHANNEL`` or ``activation=ACT_GELU_ERF`` the layer
    runs convrot_linear_ex instead (X, bias and Y then share W's dtype), and
    ``layer(X, addend=Z)`` adds Z [M,N] before the activation.
    """

    def __init__(self, W, bias=None, g: int = 256, wscale_mode: int = WSCALE_TENSOR, activation: int = ACT_NONE):
        import torch

        self.g = g
        self.N, self.K = W.shape
        self.activation = int(activation)
        self.general = W.dtype != torch.bfloat16 or wscale_mode != WSCALE_TENSOR or self.activation != ACT_NONE
        if self.general:
            self.Wq, self.w_scale = convrot_prepare_weight_ex(W, g, wscale_mode)
        else:
            self.Wq, self.w_scale = convrot_prepare_weight(W, g)
        self.bias = bias
        self._ws = None

    def workspace(self, M: int):
        import torch

        need = convrot_linear_workspace_bytes(M, self.N, self.K, self.g)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty((need,), dtype=torch.uint8, device=self.Wq.device)
        return self._ws

    def __call__(self, X, Y=None, stream=None, addend=None):
        ws = self.workspace(X.shape[0])
        if self.general or addend is not None:
            return convrot_linear_ex(X, self.Wq, self.w_scale, self.g, self.bias, self.activation, Y, ws, stream,
                                     addend)
        return convrot_linear(X, self.Wq, self.w_scale, self.g, self.bias, Y, ws, stream)
