"""Python binding of the C ABI in include/mfp8.h.

The ``mfp8_*`` functions here have the C names and arguments (integer device
pointers, sizes, a cudaStream_t as an integer) and only marshal arguments.
The torch helpers below them allocate outputs with torch and pass pointers;
every step of the computation runs in the CUDA kernels of libmfp8.so.  There
is no CPU fallback: without the built library every call raises.
"""
import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmfp8.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_MISALIGNED = 2
ERR_UNSUPPORTED_SHAPE = 3
ERR_WORKSPACE = 4
ERR_CUDA = 5
ERR_TIMEOUT = 6
ERR_DEVICE = 7
ERR_INDEX = 8

PATH_AUTO = 0
PATH_TILED = 1
PATH_SPLITK = 2
PATH_PAIR = 3
PATH_FUSED = 4

FLAG_STATIC_WEIGHTS = 1

ROPE_HALF = 0
ROPE_INTERLEAVED = 1

ATTEND_AUTO = 0
ATTEND_ROWS = 1
ATTEND_TALL = 2

ROPE_SCALE_NONE = 0
ROPE_SCALE_LINEAR = 1
ROPE_SCALE_NTK = 2
ROPE_SCALE_YARN = 3


class Mfp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {mfp8_status_string(status)} (status {status})")


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(python -m fp8_w8a8_dynamic_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        f32, f64 = ctypes.c_float, ctypes.c_double
        sig = {
            "mfp8_quantize_weight": (i32, [P, i64, i64, P, P, P]),
            "mfp8_quantize_act": (i32, [P, i64, i64, P, P, P]),
            "mfp8_linear_workspace_bytes": (sz, [i64, i64, i64]),
            "mfp8_linear": (i32, [P, i64, i64, P, P, i64, P, P, sz, P]),
            "mfp8_linear_ex": (i32, [P, i64, i64, P, P, i64, P, P, sz, i32, i32, P, P, P]),
            "mfp8_linear_noalloc": (i32, [P, i64, i64, P, P, i64, P, P]),
            "mfp8_choose_path": (i32, [i64, i64, i64]),
            "mfp8_gemm_workspace_bytes": (sz, [i64, i64, i64]),
            "mfp8_gemm": (i32, [P, P, i64, i64, P, P, i64, P, P, sz, i32, P]),
            "mfp8_rmsnorm_quantize": (i32, [P, P, ctypes.c_float, i64, i64, P, P, P, P]),
            "mfp8_silu_mul_quantize": (i32, [P, i64, i64, P, P, P, P]),
            "mfp8_kv_quantize": (i32, [P, i64, i64, i64, P, P, P]),
            "mfp8_kv_dequantize": (i32, [P, P, i64, i64, i64, P, P]),
            "mfp8_kv8_quantize": (i32, [P, i64, i64, i64, P, P, P, P]),
            "mfp8_kv8_read": (i32, [P, P, P, i64, P, i64, i64, i64, P, P]),
            "mfp8_kv8_history_tokens": (i64, [i64]),
            "mfp8_rope_frequencies": (i32, [i64, f64, i32, f64, i64, f64, f64, P, P]),
            "mfp8_rope": (i32, [P, i64, i64, i64, i64, P, i32, P, P, i64, i32, f64, P, i64, P]),
            "mfp8_kv_page_store": (i32, [P, i64, P, i64, i64, i64, P, P, i64, i64, P]),
            "mfp8_kv_page_read": (i32, [P, P, i64, i64, P, i64, i64, i64, P, P]),
            "mfp8_rope_kv_store": (i32, [P, i64, i64, i64, i64, i64, P, i32, P, P, i64, i32, f64, P, P, P, P, P, P,
                                         i64, i64, P]),
            "mfp8_prefix_attention_workspace_bytes": (sz, [i64] * 9),
            "mfp8_prefix_attention": (i32, [P, i64, i64, i64, i64, i64, P, P, i64, i64, P, P, P, P, i64, i64, P, i64,
                                            P, i64, i64, f32, P, P, P, sz, i32, P]),
            "mfp8_debug_kv8_code_check": (i32, [P, i64, ctypes.c_uint32, P]),
            "mfp8_e4m3_encode_f32": (i32, [P, i64, P, P]),
            "mfp8_debug_quantize_check": (i32, [P, P]),
            "mfp8_debug_bounded_wait": (i32, [i64, P]),
            "mfp8_get_device_status": (i32, [P]),
            "mfp8_status_string": (ctypes.c_char_p, [i32]),
            "mfp8_version": (i32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# ---------------------------------------------------------------- C names --

def mfp8_quantize_weight(W_bf16, N, K, W_fp8, w_scale, stream=0):
    return lib().mfp8_quantize_weight(W_bf16, N, K, W_fp8, w_scale, stream)


def mfp8_quantize_act(X_bf16, M, K, X_fp8, x_scale, stream=0):
    return lib().mfp8_quantize_act(X_bf16, M, K, X_fp8, x_scale, stream)


def mfp8_linear_workspace_bytes(M, N, K):
    return lib().mfp8_linear_workspace_bytes(M, N, K)


def mfp8_linear(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes, stream=0):
    return lib().mfp8_linear(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes, stream)


def mfp8_linear_ex(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes, path, flags,
                   X_fp8_out, x_scale_out, stream=0):
    return lib().mfp8_linear_ex(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes,
                                path, flags, X_fp8_out, x_scale_out, stream)


def mfp8_linear_noalloc(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, stream=0):
    return lib().mfp8_linear_noalloc(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, stream)


STATIC_WORKSPACE_BYTES = 16 << 20  # MFP8_STATIC_WORKSPACE_BYTES


def mfp8_choose_path(M, N, K):
    return lib().mfp8_choose_path(M, N, K)


KERNEL_OF_PATH = {PATH_TILED: "gemm_tiled_kernel", PATH_SPLITK: "gemm_cluster_kernel",
                  PATH_PAIR: "gemm_pair_kernel", PATH_FUSED: "gemm_stream_kernel"}


def mfp8_gemm_workspace_bytes(M, N, K):
    return lib().mfp8_gemm_workspace_bytes(M, N, K)


def mfp8_gemm(X_fp8, x_scale, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes, path=PATH_AUTO,
              stream=0):
    return lib().mfp8_gemm(X_fp8, x_scale, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes, path,
                           stream)


def mfp8_rmsnorm_quantize(X_bf16, gamma_bf16, eps, M, K, Y_bf16, X_fp8, x_scale, stream=0):
    return lib().mfp8_rmsnorm_quantize(X_bf16, gamma_bf16, eps, M, K, Y_bf16, X_fp8, x_scale, stream)


def mfp8_silu_mul_quantize(GU_bf16, M, I, Y_bf16, X_fp8, x_scale, stream=0):
    return lib().mfp8_silu_mul_quantize(GU_bf16, M, I, Y_bf16, X_fp8, x_scale, stream)


def mfp8_kv_quantize(KV_bf16, T, H, D, KV_fp8, kv_scale, stream=0):
    return lib().mfp8_kv_quantize(KV_bf16, T, H, D, KV_fp8, kv_scale, stream)


def mfp8_kv_dequantize(KV_fp8, kv_scale, T, H, D, KV_bf16, stream=0):
    return lib().mfp8_kv_dequantize(KV_fp8, kv_scale, T, H, D, KV_bf16, stream)


def mfp8_kv8_quantize(KV_bf16, T, H, D, KV_u8, kv_scale, kv_zero, stream=0):
    return lib().mfp8_kv8_quantize(KV_bf16, T, H, D, KV_u8, kv_scale, kv_zero, stream)


def mfp8_kv8_read(KV_u8, kv_scale, kv_zero, Tq, tail_bf16, Tr, H, D, out_bf16, stream=0):
    return lib().mfp8_kv8_read(KV_u8, kv_scale, kv_zero, Tq, tail_bf16, Tr, H, D, out_bf16, stream)


def mfp8_kv8_history_tokens(T):
    return lib().mfp8_kv8_history_tokens(T)


def mfp8_rope_frequencies(rot, theta, scaling, factor, trained_len, beta_fast, beta_slow, inv_freq_host, mscale_host):
    return lib().mfp8_rope_frequencies(rot, theta, scaling, factor, trained_len, beta_fast, beta_slow, inv_freq_host,
                                       mscale_host)


def mfp8_rope(X_bf16, ldx, T, H, D, pos, n_axes, axis, inv_freq, rot, layout, mscale, Y_bf16, ldy, stream=0):
    return lib().mfp8_rope(X_bf16, ldx, T, H, D, pos, n_axes, axis, inv_freq, rot, layout, mscale, Y_bf16, ldy, stream)


def mfp8_kv_page_store(KV_bf16, ldkv, slot, T, H, D, pages, scale, n_pages, page_size, stream=0):
    return lib().mfp8_kv_page_store(KV_bf16, ldkv, slot, T, H, D, pages, scale, n_pages, page_size, stream)


def mfp8_kv_page_read(pages, scale, n_pages, page_size, slot, T, H, D, out_bf16, stream=0):
    return lib().mfp8_kv_page_read(pages, scale, n_pages, page_size, slot, T, H, D, out_bf16, stream)


def mfp8_rope_kv_store(QKV_bf16, ldqkv, T, Hq, Hkv, D, pos, n_axes, axis, inv_freq, rot, layout, mscale, slot, Q_bf16,
                       k_pages, k_scale, v_pages, v_scale, n_pages, page_size, stream=0):
    return lib().mfp8_rope_kv_store(QKV_bf16, ldqkv, T, Hq, Hkv, D, pos, n_axes, axis, inv_freq, rot, layout, mscale,
                                    slot, Q_bf16, k_pages, k_scale, v_pages, v_scale, n_pages, page_size, stream)


def mfp8_prefix_attention_workspace_bytes(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size):
    return lib().mfp8_prefix_attention_workspace_bytes(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size)


def mfp8_prefix_attention(Q_bf16, ldq, T, Hq, Hkv, D, q_start, kv_len, B, max_q, k_pages, k_scale, v_pages, v_scale,
                          n_pages, page_size, prefix_pages, prefix_len, page_table, ld_table, max_pages,
                          softmax_scale, O_bf16, lse, workspace, workspace_bytes, path=0, stream=0):
    return lib().mfp8_prefix_attention(Q_bf16, ldq, T, Hq, Hkv, D, q_start, kv_len, B, max_q, k_pages, k_scale,
                                       v_pages, v_scale, n_pages, page_size, prefix_pages, prefix_len, page_table,
                                       ld_table, max_pages, softmax_scale, O_bf16, lse, workspace, workspace_bytes,
                                       path, stream)


def mfp8_debug_kv8_code_check(out, n_scale_pairs, seed, stream=0):
    return lib().mfp8_debug_kv8_code_check(out, n_scale_pairs, seed, stream)


def mfp8_e4m3_encode_f32(inp, n, out, stream=0):
    return lib().mfp8_e4m3_encode_f32(inp, n, out, stream)


def mfp8_debug_quantize_check(out, stream=0):
    return lib().mfp8_debug_quantize_check(out, stream)


def mfp8_debug_bounded_wait(timeout_us, stream=0):
    return lib().mfp8_debug_bounded_wait(timeout_us, stream)


def mfp8_get_device_status(stream=0):
    return lib().mfp8_get_device_status(stream)


def mfp8_status_string(status):
    return lib().mfp8_status_string(int(status)).decode()


def mfp8_version():
    return lib().mfp8_version()


# ---------------------------------------------------------- torch helpers --

def _check(status, where):
    if status != OK:
        raise Mfp8Error(status, where)


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t):
    return t.data_ptr() if t is not None else None


def quantize_weight(W, stream=None):
    """W: bf16 [N, K] CUDA tensor -> (W_fp8 uint8 [N, K], w_scale fp32 [N])."""
    import torch
    N, K = W.shape
    W8 = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    sw = torch.empty((N,), dtype=torch.float32, device=W.device)
    _check(mfp8_quantize_weight(_ptr(W), N, K, _ptr(W8), _ptr(sw), _stream_handle(stream)),
           "mfp8_quantize_weight")
    return W8, sw


def quantize_act(X, stream=None):
    """X: bf16 [M, K] CUDA tensor -> (X_fp8 uint8 [M, K], x_scale fp32 [M])."""
    import torch
    M, K = X.shape
    X8 = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    sa = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(mfp8_quantize_act(_ptr(X), M, K, _ptr(X8), _ptr(sa), _stream_handle(stream)),
           "mfp8_quantize_act")
    return X8, sa


def workspace_for(M, N, K, device):
    """A workspace for mfp8_linear at these sizes: room for the activation
    codes and scales of the quantize pass (none below 17 tokens, where one
    kernel quantizes on chip).  The kernels need no particular contents; it
    is zero-filled only so that a fresh buffer is deterministic."""
    import torch
    nbytes = mfp8_linear_workspace_bytes(M, N, K)
    return torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=device)


def linear(X, W8, w_scale, out=None, workspace=None, path=PATH_AUTO, x8_out=None, xs_out=None,
           flags=0, stream=None):
    """Y = FP8_DYNAMIC Linear(X) with pre-quantized weights.  X bf16 [M, K]."""
    import torch
    M, K = X.shape
    N = W8.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if workspace is None:
        workspace = workspace_for(M, N, K, X.device)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(mfp8_linear_ex(_ptr(X), M, K, _ptr(W8), _ptr(w_scale), N, _ptr(out), _ptr(workspace),
                          ws_bytes, path, flags, _ptr(x8_out), _ptr(xs_out), _stream_handle(stream)),
           "mfp8_linear_ex")
    return out


def gemm(X8, x_scale, W8, w_scale, out=None, path=PATH_AUTO, workspace=None, stream=None):
    """The contraction alone on pre-quantized activations."""
    import torch
    M, K = X8.shape
    N = W8.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X8.device)
    if workspace is None:
        workspace = torch.zeros((max(mfp8_gemm_workspace_bytes(M, N, K), 16),), dtype=torch.uint8,
                                device=X8.device)
    _check(mfp8_gemm(_ptr(X8), _ptr(x_scale), M, K, _ptr(W8), _ptr(w_scale), N, _ptr(out), _ptr(workspace),
                     workspace.numel(), path, _stream_handle(stream)), "mfp8_gemm")
    return out


def rmsnorm_quantize(X, gamma, eps, want_y=True, stream=None):
    """X bf16 [M, K], gamma bf16 [K] -> (y bf16 [M, K] or None, codes uint8 [M, K], scales fp32 [M])."""
    import torch
    M, K = X.shape
    y = torch.empty((M, K), dtype=torch.bfloat16, device=X.device) if want_y else None
    codes = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    scales = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(mfp8_rmsnorm_quantize(_ptr(X), _ptr(gamma), float(eps), M, K, _ptr(y), _ptr(codes), _ptr(scales),
                                 _stream_handle(stream)), "mfp8_rmsnorm_quantize")
    return y, codes, scales


def silu_mul_quantize(GU, want_y=True, stream=None):
    """GU bf16 [M, 2I] (gate | up) -> (y bf16 [M, I] or None, codes uint8 [M, I], scales fp32 [M])."""
    import torch
    M, I2 = GU.shape
    I = I2 // 2
    y = torch.empty((M, I), dtype=torch.bfloat16, device=GU.device) if want_y else None
    codes = torch.empty((M, I), dtype=torch.uint8, device=GU.device)
    scales = torch.empty((M,), dtype=torch.float32, device=GU.device)
    _check(mfp8_silu_mul_quantize(_ptr(GU), M, I, _ptr(y), _ptr(codes), _ptr(scales), _stream_handle(stream)),
           "mfp8_silu_mul_quantize")
    return y, codes, scales


def kv_quantize(KV, stream=None):
    """KV: bf16 [T, H, D] CUDA tensor -> (codes uint8 [T, H, D], scales fp32 [T, H])."""
    import torch
    T, H, D = KV.shape
    codes = torch.empty((T, H, D), dtype=torch.uint8, device=KV.device)
    scales = torch.empty((T, H), dtype=torch.float32, device=KV.device)
    _check(mfp8_kv_quantize(_ptr(KV), T, H, D, _ptr(codes), _ptr(scales), _stream_handle(stream)),
           "mfp8_kv_quantize")
    return codes, scales


def kv_dequantize(codes, scales, stream=None):
    """codes uint8 [T, H, D], scales fp32 [T, H] -> bf16 [T, H, D]."""
    import torch
    T, H, D = codes.shape
    out = torch.empty((T, H, D), dtype=torch.bfloat16, device=codes.device)
    _check(mfp8_kv_dequantize(_ptr(codes), _ptr(scales), T, H, D, _ptr(out), _stream_handle(stream)),
           "mfp8_kv_dequantize")
    return out


def kv8_quantize(KV, stream=None):
    """KV: bf16 [T, H, D] CUDA tensor, T % 64 == 0 -> (codes uint8 [T, H, D],
    scale fp32 [T/64, H, D], zero fp32 [T/64, H, D])."""
    import torch
    T, H, D = KV.shape
    codes = torch.empty((T, H, D), dtype=torch.uint8, device=KV.device)
    scale = torch.empty((T // 64, H, D), dtype=torch.float32, device=KV.device)
    zero = torch.empty((T // 64, H, D), dtype=torch.float32, device=KV.device)
    _check(mfp8_kv8_quantize(_ptr(KV), T, H, D, _ptr(codes), _ptr(scale), _ptr(zero), _stream_handle(stream)),
           "mfp8_kv8_quantize")
    return codes, scale, zero


def kv8_read(codes, scale, zero, tail, out=None, stream=None):
    """History (codes [Tq, H, D], scale and zero [Tq/64, H, D]) and bf16 tail
    [Tr, H, D] -> bf16 [Tq + Tr, H, D]: the history dequantized, then the
    tail."""
    import torch
    Tq, H, D = codes.shape
    Tr = tail.shape[0]
    if out is None:
        out = torch.empty((Tq + Tr, H, D), dtype=torch.bfloat16, device=codes.device)
    _check(mfp8_kv8_read(_ptr(codes), _ptr(scale), _ptr(zero), Tq, _ptr(tail), Tr, H, D, _ptr(out),
                         _stream_handle(stream)), "mfp8_kv8_read")
    return out


class Kv8Cache:
    """One K or V tensor of a layer held as the INT8 cache: a history of
    whole 64-token groups (codes, scale, zero) and the bf16 tail of the
    latest positions.  Buffers are allocated once for `capacity` positions.
    ``append`` stages the old tail and the new positions in one bf16 buffer,
    quantizes the positions that mfp8_kv8_history_tokens moves into the
    history (mfp8_kv8_quantize, written in place after the existing groups)
    and keeps the rest as the tail; ``read`` returns every position as bf16
    (mfp8_kv8_read).  Work is queued on the current torch stream."""

    def __init__(self, capacity, H, D, device):
        import torch
        groups = (capacity + 63) // 64
        self.capacity, self.H, self.D = capacity, H, D
        self.codes = torch.empty((groups * 64, H, D), dtype=torch.uint8, device=device)
        self.scale = torch.empty((groups, H, D), dtype=torch.float32, device=device)
        self.zero = torch.empty((groups, H, D), dtype=torch.float32, device=device)
        self.tail = torch.empty((0, H, D), dtype=torch.bfloat16, device=device)
        self.T = 0

    @property
    def Tq(self):
        return mfp8_kv8_history_tokens(self.T)

    def append(self, kv):
        import torch
        n = kv.shape[0]
        if kv.shape[1:] != (self.H, self.D) or kv.dtype != torch.bfloat16:
            raise ValueError("Kv8Cache.append: expected bf16 [n, H, D]")
        if self.T + n > self.capacity:
            raise ValueError("Kv8Cache.append: capacity exceeded")
        tq, tq2 = self.Tq, mfp8_kv8_history_tokens(self.T + n)
        staged = torch.cat([self.tail, kv]) if self.tail.shape[0] else kv.contiguous()
        f = tq2 - tq
        if f:
            g = tq // 64
            _check(mfp8_kv8_quantize(_ptr(staged), f, self.H, self.D, _ptr(self.codes[tq]), _ptr(self.scale[g]),
                                     _ptr(self.zero[g]), _stream_handle(None)), "mfp8_kv8_quantize")
        self.tail = staged[f:].clone()
        self.T += n

    def read(self, out=None):
        tq = self.Tq
        return kv8_read(self.codes[:tq], self.scale[:tq // 64], self.zero[:tq // 64], self.tail, out=out)


def _on(where, stream, tensors):
    """The stream handle that a helper's kernels run on: `stream`, or torch's
    current one, of the current device, which must hold every tensor (a
    tensor elsewhere answers another device number, or -1)."""
    import torch
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensors must be on the current CUDA device ({dev})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"{where}: the stream belongs to another device")
    if stream.cuda_stream != torch._C._cuda_getCurrentRawStream(dev):
        # torch's allocator must not hand these on before the kernels are done with them
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return stream.cuda_stream


def _new(like, shape, dtype, stream):
    """An uninitialised tensor on like's device, allocated on the stream that writes it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _need(ok, where, what):
    if not ok:
        raise ValueError(f"{where}: {what}")


def _rows(where, x, name="x"):
    """bf16 [T, H, D] with whole head rows one after the other: T, H, D, elements between tokens."""
    import torch
    if x.dtype is not torch.bfloat16 or x.dim() != 3:
        raise ValueError(f"{where}: {name} must be bf16 [T, H, D]")
    T, H, D = x.shape
    if x.is_contiguous():
        return T, H, D, H * D
    ld, sh, sd = x.stride()
    if T and ((D > 1 and sd != 1) or (H > 1 and sh != D)):
        raise ValueError(f"{where}: the head rows of a token in {name} must be contiguous")
    return T, H, D, ld if T > 1 else H * D


def _rope_args(where, T, pos, inv_freq, axis):
    """(n_axes, rot) of position and frequency tensors that fit."""
    import torch
    if pos.dtype is not torch.int32 or pos.dim() not in (1, 2) or pos.shape[-1] != T or not pos.is_contiguous():
        raise ValueError(f"{where}: pos must be contiguous int32 [T] or [axes, T]")
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"{where}: inv_freq must be contiguous fp32 [rot / 2]")
    n_axes = pos.shape[0] if pos.dim() == 2 else 1
    if axis is None:
        _need(n_axes == 1, where, "several position axes need `axis`")
    else:
        _need(axis.dtype is torch.uint8 and axis.shape == inv_freq.shape and axis.is_contiguous(), where,
              "axis must be contiguous uint8 [rot / 2]")
    return n_axes, 2 * inv_freq.shape[0]


def _pool(where, pages, scale):
    """(n_pages, H, page_size, D) of a paged cache tensor with its scales."""
    import torch
    shape = pages.shape
    if pages.dtype is not torch.uint8 or len(shape) != 4 or not pages.is_contiguous():
        raise ValueError(f"{where}: pages must be contiguous uint8 [n_pages, H, page_size, D]")
    if scale.dtype is not torch.float32 or scale.shape != shape[:3] or not scale.is_contiguous():
        raise ValueError(f"{where}: scale must be contiguous fp32 [n_pages, H, page_size]")
    return shape


def _slots(where, slot):
    import torch
    if slot.dtype is not torch.int64 or slot.dim() != 1 or not slot.is_contiguous():
        raise ValueError(f"{where}: slot must be contiguous int64 [T]")
    return slot.shape[0]


def rope_frequencies(rot, theta, scaling=ROPE_SCALE_NONE, factor=1.0, trained_len=0, beta_fast=32.0, beta_slow=1.0,
                     device="cuda"):
    """The frequency table of ``rope``: (fp32 [rot / 2] on `device`, mscale)."""
    import torch
    host = torch.empty((max(int(rot), 0) // 2,), dtype=torch.float32)
    mscale = ctypes.c_double(1.0)
    _check(mfp8_rope_frequencies(rot, theta, scaling, factor, trained_len, beta_fast, beta_slow, host.data_ptr(),
                                 ctypes.addressof(mscale)), "mfp8_rope_frequencies")
    return host.to(device), mscale.value


def rope(x, pos, inv_freq, axis=None, layout=ROPE_HALF, mscale=1.0, out=None, stream=None):
    """Rotary positions: x bf16 [T, H, D] (tokens may be strided, as the query
    columns of a packed projection) -> rotated bf16 [T, H, D].  pos int32 [T]
    or [axes, T]; inv_freq fp32 [rot / 2]; axis uint8 [rot / 2].  `out` may
    be x itself."""
    T, H, D, ldx = _rows("rope", x)
    n_axes, rot = _rope_args("rope", T, pos, inv_freq, axis)
    handle = _on("rope", stream, (x, pos, inv_freq, axis, out))
    if out is None:
        out, ldy = _new(x, (T, H, D), x.dtype, stream), H * D
    else:
        _need(out.shape == x.shape, "rope", "out must have x's shape")
        ldy = _rows("rope", out, "out")[3]
    _check(lib().mfp8_rope(x.data_ptr(), ldx, T, H, D, pos.data_ptr(), n_axes, _ptr(axis), inv_freq.data_ptr(), rot,
                           layout, mscale, out.data_ptr(), ldy, handle), "mfp8_rope")
    return out


def kv_page_store(kv, slot, pages, scale, stream=None):
    """Quantize kv bf16 [T, H, D] (tokens may be strided) into the slots (int64
    [T], negative: skipped) of pages uint8 [n_pages, H, page_size, D] and
    scale fp32 [n_pages, H, page_size]."""
    w = "kv_page_store"
    T, H, D, ld = _rows(w, kv, "kv")
    n_pages, hp, ps, dp = _pool(w, pages, scale)
    _need((hp, dp) == (H, D), w, "kv and pages must have the same heads and head size")
    _need(_slots(w, slot) == T, w, "slot must have one entry per token")
    handle = _on(w, stream, (kv, slot, pages, scale))
    _check(lib().mfp8_kv_page_store(kv.data_ptr(), ld, slot.data_ptr(), T, H, D, pages.data_ptr(), scale.data_ptr(),
                                    n_pages, ps, handle), "mfp8_kv_page_store")


def kv_page_read(pages, scale, slot, out=None, stream=None):
    """The rows in slot int64 [T] of a paged cache as bf16 [T, H, D] (zeros for a negative slot)."""
    import torch
    w = "kv_page_read"
    n_pages, H, ps, D = _pool(w, pages, scale)
    T = _slots(w, slot)
    handle = _on(w, stream, (pages, scale, slot, out))
    if out is None:
        out = _new(pages, (T, H, D), torch.bfloat16, stream)
    else:
        _need(out.dtype is torch.bfloat16 and out.shape == (T, H, D) and out.is_contiguous(), w,
              "out must be contiguous bf16 [T, H, D]")
    _check(lib().mfp8_kv_page_read(pages.data_ptr(), scale.data_ptr(), n_pages, ps, slot.data_ptr(), T, H, D,
                                   out.data_ptr(), handle), "mfp8_kv_page_read")
    return out


def rope_kv_store(qkv, n_heads, pos, inv_freq, slot, k_pages, k_scale, v_pages, v_scale, axis=None, layout=ROPE_HALF,
                  mscale=1.0, out=None, stream=None):
    """What stands between qkv_proj and attention: qkv bf16 [T, (n_heads + 2
    Hkv) D] (rows may be strided) -> rotated queries bf16 [T, n_heads, D];
    rotated keys and values are quantized into their slots.  Hkv and D are
    those of the pages."""
    import torch
    w = "rope_kv_store"
    shape = _pool(w, k_pages, k_scale)
    _need(_pool(w, v_pages, v_scale) == shape, w, "k_pages and v_pages must have one shape")
    n_pages, Hkv, ps, D = shape
    if qkv.dtype is not torch.bfloat16 or qkv.dim() != 2 or qkv.shape[1] != (n_heads + 2 * Hkv) * D or (
            qkv.shape[0] and qkv.stride(1) != 1):
        raise ValueError(f"{w}: qkv must be bf16 [T, (n_heads + 2 Hkv) D]")
    T = qkv.shape[0]
    n_axes, rot = _rope_args(w, T, pos, inv_freq, axis)
    _need(_slots(w, slot) == T, w, "slot must have one entry per token")
    handle = _on(w, stream, (qkv, pos, inv_freq, axis, slot, k_pages, k_scale, v_pages, v_scale, out))
    if out is None:
        out = _new(qkv, (T, n_heads, D), qkv.dtype, stream)
    else:
        _need(out.dtype is torch.bfloat16 and out.shape == (T, n_heads, D) and out.is_contiguous(), w,
              "out must be contiguous bf16 [T, n_heads, D]")
    _check(lib().mfp8_rope_kv_store(qkv.data_ptr(), qkv.stride(0) if T > 1 else qkv.shape[1], T, n_heads, Hkv, D,
                                    pos.data_ptr(), n_axes, _ptr(axis), inv_freq.data_ptr(), rot, layout, mscale,
                                    slot.data_ptr(), out.data_ptr(), k_pages.data_ptr(), k_scale.data_ptr(),
                                    v_pages.data_ptr(), v_scale.data_ptr(), n_pages, ps, handle), "mfp8_rope_kv_store")
    return out


@functools.lru_cache(maxsize=1024)
def _attention_workspace(*sizes):
    return mfp8_prefix_attention_workspace_bytes(*sizes)


def prefix_attention(q, q_start, kv_len, page_table, prefix_pages, prefix_len, k_pages, k_scale, v_pages, v_scale,
                     max_q, scale=None, out=None, want_lse=False, workspace=None, path=ATTEND_AUTO, stream=None):
    """Attention of a batch that shares a prefix, over the paged FP8 cache.
    q bf16 [T, Hq, D] (tokens may be strided); q_start int32 [B + 1]: sequence
    b has the query tokens q_start[b] .. q_start[b + 1] - 1, at most max_q;
    kv_len int32 [B]: its own cached tokens, the query tokens the last of them;
    page_table int32 [B, max_pages] (rows may be strided) or None;
    prefix_pages int32 [>= ceil(prefix_len / page_size)] or None, prefix_len
    an int; scale defaults to D ** -0.5.  -> bf16 [T, Hq, D], with want_lse
    also the natural log-sum-exp fp32 [T, Hq]."""
    import torch
    w = "prefix_attention"
    i32 = torch.int32
    T, Hq, D, ldq = _rows(w, q, "q")
    shape = _pool(w, k_pages, k_scale)
    _need(_pool(w, v_pages, v_scale) == shape, w, "k_pages and v_pages must have one shape")
    n_pages, Hkv, ps, dp = shape
    _need(dp == D, w, "q and the pages must have one head size")
    if kv_len.dtype is not i32 or kv_len.dim() != 1 or not kv_len.is_contiguous():
        raise ValueError(f"{w}: kv_len must be contiguous int32 [B]")
    B = kv_len.shape[0]
    if q_start.dtype is not i32 or q_start.shape != (B + 1,) or not q_start.is_contiguous():
        raise ValueError(f"{w}: q_start must be contiguous int32 [B + 1]")
    max_pages = ld = 0
    if page_table is not None:
        if page_table.dtype is not i32 or page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError(f"{w}: page_table must be int32 [B, max_pages]")
        max_pages = page_table.shape[1]
        _need(max_pages < 2 or page_table.stride(1) == 1, w, "the rows of page_table must be contiguous")
        ld = page_table.stride(0) if B > 1 else max_pages
    if prefix_len:
        _need(prefix_pages is not None and prefix_pages.dtype is i32 and prefix_pages.dim() == 1
              and prefix_pages.is_contiguous() and 0 < prefix_len <= prefix_pages.shape[0] * ps, w,
              "prefix_pages must be contiguous int32 and cover prefix_len")
    handle = _on(w, stream, (q, q_start, kv_len, page_table, prefix_pages, k_pages, k_scale, v_pages, v_scale, out,
                             workspace))
    if out is None:
        out = _new(q, (T, Hq, D), q.dtype, stream)
    else:
        _need(out.dtype is torch.bfloat16 and out.shape == (T, Hq, D) and out.is_contiguous(), w,
              "out must be contiguous bf16 [T, Hq, D]")
    lse = _new(q, (T, Hq), torch.float32, stream) if want_lse else None
    if workspace is None:
        nbytes = _attention_workspace(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, ps)
        if nbytes:
            workspace = _new(q, (nbytes,), torch.uint8, stream)
    else:
        _need(workspace.is_contiguous(), w, "workspace must be contiguous")
        nbytes = workspace.nbytes
    _check(lib().mfp8_prefix_attention(
        q.data_ptr(), ldq, T, Hq, Hkv, D, q_start.data_ptr(), kv_len.data_ptr(), B, max_q, k_pages.data_ptr(),
        k_scale.data_ptr(), v_pages.data_ptr(), v_scale.data_ptr(), n_pages, ps, _ptr(prefix_pages), prefix_len,
        page_table.data_ptr() if max_pages else None, ld, max_pages, scale if scale is not None else D ** -0.5,
        out.data_ptr(), _ptr(lse), _ptr(workspace), nbytes, path, handle), "mfp8_prefix_attention")
    return (out, lse) if want_lse else out


def e4m3_encode(values, stream=None):
    """fp32 CUDA tensor -> uint8 codes from the device's conversion."""
    import torch
    out = torch.empty(values.shape, dtype=torch.uint8, device=values.device)
    _check(mfp8_e4m3_encode_f32(_ptr(values), values.numel(), _ptr(out), _stream_handle(stream)),
           "mfp8_e4m3_encode_f32")
    return out


def device_status(stream=None):
    return mfp8_get_device_status(_stream_handle(stream))
