"""Python binding of libhstu_b200 (the C ABI in include/hstu.h): argument marshalling only.

Every step of the HSTU layer forward runs in the library's CUDA kernels for sm_100a; this module
passes device pointers, sizes and the current CUDA stream through ctypes.  PyTorch supplies device
memory and streams.  There is no CPU implementation here: if the compiled library is missing,
importing this package raises.

The layer ("Actions Speak Louder than Words" paper notes, section 3.1, Eqs. 1-3):
    [U|V|Q|K] = SiLU(X W1 + b1)
    AV_i      = sum_{j<=i} scale * SiLU(q_i.k_j + rab^{p,t}(i, j)) v_j      (per head, jagged, causal)
    Y         = (LayerNorm(AV) * U) W2 + b2 + X
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhstu_b200.so")

HSTU_OK, HSTU_ERR_INVALID_ARG, HSTU_ERR_UNSUPPORTED, HSTU_ERR_CUDA = 0, 1, 2, 3
HSTU_ERR_DEVICE_TIMEOUT, HSTU_ERR_DEVICE_BAD_OFFSETS = 4, 5
HSTU_F32, HSTU_BF16 = 0, 1

# Every symbol include/hstu.h declares.
EXPORTED = ["hstu_layer_fwd", "hstu_layer_fwd_workspace_size", "hstu_f1_fwd", "hstu_attention_fwd",
            "hstu_attention_workspace_size", "hstu_ln_gate_fwd", "hstu_f2_fwd",
            "hstu_token_embed_fwd", "hstu_status_string", "hstu_get_device_status", "hstu_version",
            "hstu_launch_count", "hstu_attention_fwd_noalloc", "hstu_selftest_bounded_wait",
            "hstu_selftest_scratch_cache", "hstu_ln_f2_fwd",
            "hstu_candidate_workspace_size", "hstu_candidate_attention_fwd",
            "hstu_candidate_layer_workspace_size", "hstu_candidate_layer_fwd",
            "hstu_cache_append", "hstu_paged_attention_workspace_size", "hstu_paged_attention_fwd",
            "hstu_paged_layer_workspace_size", "hstu_paged_layer_fwd",
            "hstu_cache_evict_workspace_size", "hstu_cache_evict",
            "hstu_stochastic_length_workspace_size", "hstu_stochastic_length", "hstu_gather_rows",
            "hstu_attention_bwd_workspace_size", "hstu_attention_bwd",
            "hstu_layer_bwd_workspace_size", "hstu_layer_bwd", "hstu_layer_pipeline_create",
            "hstu_layer_pipeline_submit", "hstu_layer_pipeline_sync",
            "hstu_layer_pipeline_timing_begin", "hstu_layer_pipeline_timing_end",
            "hstu_layer_pipeline_destroy"]


class HstuShape(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
                ("max_seq_len", ctypes.c_int64), ("d_model", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("n_pos_buckets", ctypes.c_int32), ("n_time_buckets", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("ln_eps", ctypes.c_float)]


class HstuPagedCache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("timestamps", ctypes.c_void_p),
                ("weights", ctypes.c_void_p)]


class HstuError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


def _load() -> ctypes.CDLL:
    from . import build as _build
    try:
        _build.build()          # no-op unless a source is newer than the library
    except Exception as e:      # no nvcc here: use the shipped library if there is one
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing and could not be built ({e}); "
                              "this package has no CPU fallback") from e
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, F32, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    SH = ctypes.POINTER(HstuShape)
    PC = ctypes.POINTER(HstuPagedCache)
    sig = {
        "hstu_layer_fwd": ([SH, P, P, P, P, P, P, P, P, P, P, P, P, F32, P, P, S, P], ctypes.c_int),
        "hstu_layer_fwd_workspace_size": ([SH], S),
        "hstu_f1_fwd": ([SH, P, P, P, P, P], ctypes.c_int),
        "hstu_attention_fwd": ([SH, P, P, P, P, P, P, F32, P, P, S, P], ctypes.c_int),
        "hstu_attention_workspace_size": ([SH], S),
        "hstu_attention_fwd_noalloc": ([SH, P, P, P, P, P, P, F32, P, P], ctypes.c_int),
        "hstu_ln_gate_fwd": ([SH, P, P, P, P, P, P], ctypes.c_int),
        "hstu_f2_fwd": ([SH, P, P, P, P, P, P], ctypes.c_int),
        "hstu_ln_f2_fwd": ([SH, P, P, P, P, P, P, P, P, P], ctypes.c_int),
        "hstu_token_embed_fwd": ([I64, I32, P, P, P, I64, P, I64, P, P], ctypes.c_int),
        "hstu_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "hstu_get_device_status": ([P], ctypes.c_int),
        "hstu_version": ([], ctypes.c_char_p),
        "hstu_launch_count": ([], ctypes.c_uint64),
        "hstu_selftest_bounded_wait": ([ctypes.c_uint64, P, P], ctypes.c_int),
        "hstu_selftest_scratch_cache": ([], ctypes.c_int32),
        "hstu_candidate_workspace_size": ([SH, I64], S),
        "hstu_candidate_attention_fwd": ([SH, P, P, P, I64, I64, P, P, P, P, P, P, F32, P, P, S, P],
                                         ctypes.c_int),
        "hstu_candidate_layer_workspace_size": ([SH, I64], S),
        "hstu_stochastic_length_workspace_size": ([I64], S),
        "hstu_stochastic_length": ([I64, I64, P, I64, ctypes.c_double, P, P, P, P, P, S, P],
                                   ctypes.c_int),
        "hstu_gather_rows": ([I64, P, I64, P, P, I64, P, P], ctypes.c_int),
        "hstu_attention_bwd_workspace_size": ([SH], S),
        "hstu_attention_bwd": ([SH, P, P, P, P, P, P, F32, P, P, P, P, P, P, P, S, P], ctypes.c_int),
        "hstu_candidate_layer_fwd": ([SH, P, P, P, I64, I64, P, P, P, P, P, P, P, P, P, P, P, P, F32,
                                      P, P, S, P], ctypes.c_int),
        "hstu_cache_append": ([PC, I64, I64, P, P, P, P, I64, P, P, P], ctypes.c_int),
        "hstu_paged_attention_workspace_size": ([SH], S),
        "hstu_paged_attention_fwd": ([SH, PC, P, P, I64, P, P, P, P, P, P, F32, I32, P, P, S, P],
                                     ctypes.c_int),
        "hstu_paged_layer_workspace_size": ([SH], S),
        "hstu_paged_layer_fwd": ([SH, PC, P, P, I64, P, P, P, P, P, P, P, P, P, P, P, P, F32, I32, P,
                                  P, S, P], ctypes.c_int),
        "hstu_cache_evict_workspace_size": ([PC, I64, I64], S),
        "hstu_cache_evict": ([PC, I64, P, I64, P, P, I64, I64, P, P, S, P], ctypes.c_int),
        "hstu_layer_bwd_workspace_size": ([SH], S),
        "hstu_layer_pipeline_create": ([SH, I32, ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
        "hstu_layer_pipeline_submit": ([P, SH, P, P, P, P, P, P, P, P, P, P, P, P, F32, P],
                                       ctypes.c_int),
        "hstu_layer_pipeline_sync": ([P], ctypes.c_int),
        "hstu_layer_pipeline_timing_begin": ([P], ctypes.c_int),
        "hstu_layer_pipeline_timing_end": ([P, ctypes.POINTER(ctypes.c_float)], ctypes.c_int),
        "hstu_layer_pipeline_destroy": ([P], None),
        "hstu_layer_bwd": ([SH, P, P, P, P, P, P, P, P, P, P, P, F32, P, S, P, P, P, P, P, P, P, P,
                            P, P, P, S, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def status_string(code: int) -> str:
    return _lib.hstu_status_string(int(code)).decode()


def version() -> str:
    return _lib.hstu_version().decode()


def selftest_bounded_wait(limit_ns: int, result, stream=None) -> None:
    """Runs the device self-test of the library's bounded mbarrier wait (see the C header):
    `result` is a CUDA int64 tensor of 4 elements; the device status word is left set to
    HSTU_ERR_DEVICE_TIMEOUT for the caller to read with device_status()."""
    _check(_lib.hstu_selftest_bounded_wait(int(limit_ns), _ptr(result), _stream(stream)),
           "hstu_selftest_bounded_wait")


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(_lib.hstu_launch_count())


def _check(rc: int, what: str) -> None:
    if rc != HSTU_OK:
        raise HstuError(rc, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libhstu_b200 must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return HSTU_BF16
    if t.dtype == torch.float32:
        return HSTU_F32
    raise ValueError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def make_shape(num_seqs: int, total_tokens: int, max_seq_len: int, d_model: int, num_heads: int,
               d_qk: int, d_v: int, dtype: int, n_pos_buckets: int = 0, n_time_buckets: int = 0,
               ln_eps: float = 1e-5) -> HstuShape:
    return HstuShape(int(num_seqs), int(total_tokens), int(max_seq_len), int(d_model),
                     int(num_heads), int(d_qk), int(d_v), int(n_pos_buckets), int(n_time_buckets),
                     int(dtype), float(ln_eps))


def shape_for(X: torch.Tensor, seq_offsets: torch.Tensor, num_heads: int, d_qk: int, d_v: int,
              max_seq_len: int, pos_table=None, time_table=None, ln_eps: float = 1e-5) -> HstuShape:
    return make_shape(seq_offsets.numel() - 1, X.shape[0], max_seq_len, X.shape[1], num_heads,
                      d_qk, d_v, _dtype_code(X),
                      0 if pos_table is None else pos_table.shape[1],
                      0 if time_table is None else time_table.shape[1], ln_eps)


def workspace_size(shape: HstuShape) -> int:
    return int(_lib.hstu_layer_fwd_workspace_size(ctypes.byref(shape)))


def attention_workspace_size(shape: HstuShape) -> int:
    return int(_lib.hstu_attention_workspace_size(ctypes.byref(shape)))


def alloc_workspace(shape: HstuShape, device) -> torch.Tensor:
    n = workspace_size(shape)
    if n == 0 and shape.total_tokens > 0:
        raise HstuError(HSTU_ERR_INVALID_ARG, "hstu_layer_fwd_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def hstu_layer_fwd(X: torch.Tensor, seq_offsets: torch.Tensor, timestamps: Optional[torch.Tensor],
                   W1: torch.Tensor, b1: Optional[torch.Tensor], W2: torch.Tensor,
                   b2: Optional[torch.Tensor], ln_w: torch.Tensor, ln_b: torch.Tensor,
                   pos_table: Optional[torch.Tensor] = None,
                   time_table: Optional[torch.Tensor] = None,
                   alibi_slopes: Optional[torch.Tensor] = None, scale: Optional[float] = None, *,
                   num_heads: int, d_qk: Optional[int] = None, d_v: Optional[int] = None,
                   max_seq_len: int, ln_eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One HSTU layer on device tensors.  `scale` defaults to 1/max_seq_len."""
    hd = X.shape[1] // num_heads
    d_qk = hd if d_qk is None else d_qk
    d_v = hd if d_v is None else d_v
    shape = shape_for(X, seq_offsets, num_heads, d_qk, d_v, max_seq_len, pos_table, time_table,
                      ln_eps)
    if scale is None:
        scale = 1.0 / max(1, max_seq_len)
    if out is None:
        out = torch.empty_like(X)
    if workspace is None:
        workspace = alloc_workspace(shape, X.device)
    rc = _lib.hstu_layer_fwd(ctypes.byref(shape), _ptr(X), _ptr(seq_offsets), _ptr(timestamps),
                             _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(ln_w), _ptr(ln_b),
                             _ptr(pos_table), _ptr(time_table), _ptr(alibi_slopes), float(scale),
                             _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "hstu_layer_fwd")
    return out


def hstu_f1_fwd(shape: HstuShape, X, W1, b1, uvqk, stream=None):
    _check(_lib.hstu_f1_fwd(ctypes.byref(shape), _ptr(X), _ptr(W1), _ptr(b1), _ptr(uvqk),
                            _stream(stream)), "hstu_f1_fwd")
    return uvqk


def hstu_attention_fwd(shape: HstuShape, uvqk, seq_offsets, timestamps, pos_table, time_table,
                       alibi_slopes, scale: float, av, workspace=None, stream=None):
    if workspace is None:
        workspace = torch.empty(max(256, attention_workspace_size(shape)), dtype=torch.uint8,
                                device=uvqk.device)
    _check(_lib.hstu_attention_fwd(ctypes.byref(shape), _ptr(uvqk), _ptr(seq_offsets),
                                   _ptr(timestamps), _ptr(pos_table), _ptr(time_table),
                                   _ptr(alibi_slopes), float(scale), _ptr(av), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "hstu_attention_fwd")
    return av


def hstu_attention_fwd_noalloc(shape: HstuShape, uvqk, seq_offsets, timestamps, pos_table,
                               time_table, alibi_slopes, scale: float, av, stream=None):
    """hstu_attention_fwd with the tile schedule in the library's fixed device scratch array (no
    workspace argument, nothing allocated).  Calls that overlap on the GPU share that array and race."""
    _check(_lib.hstu_attention_fwd_noalloc(ctypes.byref(shape), _ptr(uvqk), _ptr(seq_offsets),
                                           _ptr(timestamps), _ptr(pos_table), _ptr(time_table),
                                           _ptr(alibi_slopes), float(scale), _ptr(av),
                                           _stream(stream)), "hstu_attention_fwd_noalloc")
    return av


def candidate_workspace_size(shape: HstuShape, num_candidates: int) -> int:
    return int(_lib.hstu_candidate_workspace_size(ctypes.byref(shape), int(num_candidates)))


def hstu_candidate_attention_fwd(shape: HstuShape, uvqk_hist, hist_offsets, hist_timestamps,
                                 uvqk_cand, cand_offsets, cand_timestamps, pos_table, time_table,
                                 alibi_slopes, scale: float, av_cand, max_candidates: int,
                                 workspace=None, stream=None):
    """M-FALCON candidate attention (see the C header): `shape` is the history's shape."""
    Tc = int(uvqk_cand.shape[0])
    if workspace is None:
        workspace = torch.empty(max(256, candidate_workspace_size(shape, Tc)), dtype=torch.uint8,
                                device=uvqk_cand.device)
    _check(_lib.hstu_candidate_attention_fwd(
        ctypes.byref(shape), _ptr(uvqk_hist), _ptr(hist_offsets), _ptr(hist_timestamps), Tc,
        int(max_candidates), _ptr(uvqk_cand), _ptr(cand_offsets), _ptr(cand_timestamps),
        _ptr(pos_table), _ptr(time_table), _ptr(alibi_slopes), float(scale), _ptr(av_cand),
        _ptr(workspace), workspace.numel(), _stream(stream)), "hstu_candidate_attention_fwd")
    return av_cand


def candidate_layer_workspace_size(shape: HstuShape, num_candidates: int) -> int:
    return int(_lib.hstu_candidate_layer_workspace_size(ctypes.byref(shape), int(num_candidates)))


def hstu_candidate_layer_fwd(shape: HstuShape, uvqk_hist, hist_offsets, hist_timestamps, X_cand,
                             cand_offsets, cand_timestamps, W1, b1, W2, b2, ln_w, ln_b, pos_table,
                             time_table, alibi_slopes, scale: float, out_cand, max_candidates: int,
                             workspace=None, stream=None):
    """One HSTU layer over the candidates given the history's UVQK of the same layer."""
    Tc = int(X_cand.shape[0])
    if workspace is None:
        workspace = torch.empty(max(256, candidate_layer_workspace_size(shape, Tc)),
                                dtype=torch.uint8, device=X_cand.device)
    _check(_lib.hstu_candidate_layer_fwd(
        ctypes.byref(shape), _ptr(uvqk_hist), _ptr(hist_offsets), _ptr(hist_timestamps), Tc,
        int(max_candidates), _ptr(X_cand), _ptr(cand_offsets), _ptr(cand_timestamps), _ptr(W1),
        _ptr(b1), _ptr(W2), _ptr(b2), _ptr(ln_w), _ptr(ln_b), _ptr(pos_table), _ptr(time_table),
        _ptr(alibi_slopes), float(scale), _ptr(out_cand), _ptr(workspace), workspace.numel(),
        _stream(stream)), "hstu_candidate_layer_fwd")
    return out_cand


class PagedCache:
    """One layer's paged key-value cache (see the C header): the caller's tensors and the struct that
    names them.  k, v [num_pages, H, page_size, hd]; positions [num_pages, page_size] int32;
    timestamps [num_pages, page_size] int64; weights [num_pages, H, page_size] fp32; the last three
    may be None.  The tensors are written in place, never exchanged: the struct holds their
    addresses."""

    def __init__(self, k, v, positions=None, timestamps=None, weights=None):
        if k.dim() != 4 or not k.is_cuda:
            raise ValueError("k is a CUDA tensor [num_pages, num_heads, page_size, head_dim]")
        pages, H, ps, hd = k.shape
        self._tensors = k, v, positions, timestamps, weights
        self.device, self.dtype = k.device, k.dtype
        self.num_pages, self.num_heads, self.page_size, self.head_dim = pages, H, ps, hd
        n = pages * ps
        self.struct = HstuPagedCache(
            pages, ps, H, hd, _dtype_code(k), _arg("k", k, k.dtype, n * H * hd, k.device),
            _arg("v", v, k.dtype, n * H * hd, k.device),
            _arg("positions", positions, torch.int32, n, k.device),
            _arg("timestamps", timestamps, torch.int64, n, k.device),
            _arg("weights", weights, torch.float32, n * H, k.device))
        self.ref = ctypes.byref(self.struct)

    k, v, positions, timestamps, weights = (property(lambda self, i=i: self._tensors[i]) for i in range(5))

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, num_heads: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", positions: bool = True,
                 timestamps: bool = True, weights: bool = True) -> "PagedCache":
        """A cache of new, zeroed tensors."""
        z = lambda shape, dt, wanted=True: torch.zeros(shape, dtype=dt, device=device) if wanted else None  # noqa: E731
        kv = (num_pages, num_heads, page_size, head_dim)
        return cls(z(kv, dtype), z(kv, dtype), z((num_pages, page_size), torch.int32, positions),
                   z((num_pages, page_size), torch.int64, timestamps),
                   z((num_pages, num_heads, page_size), torch.float32, weights))


def _refuse(name: str, t: torch.Tensor, dtype, numel: int, device):
    raise ValueError(f"{name}: a contiguous {dtype} tensor of {numel} elements on {device} is wanted, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _arg(name: str, t: Optional[torch.Tensor], dtype, numel: int, device):
    """Address of a tensor argument of the paged cache's calls, checked; None for None."""
    return _args(device, ((name, t, dtype, numel),))[0]


def _args(device, wanted):
    """Addresses of several (name, tensor, dtype, elements), checked."""
    index, out = device.index, []
    for name, t, dtype, numel in wanted:
        if t is None:
            out.append(None)
        elif t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.get_device() == index:
            out.append(t.data_ptr())
        else:
            _refuse(name, t, dtype, numel, device)
    return out


def _call(fn, what: str, device, stream, *args) -> None:
    """Calls a library function with `device` current (kernels launch on the current device), on
    `stream` or that device's current stream."""
    index = device.index
    if stream is None:
        # the address alone: building a torch.cuda.Stream takes longer than the launch
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != HSTU_OK:
        raise HstuError(rc, what)


def _new(shape, dtype, device, stream):
    """A tensor that the call's stream may use and, once it is released, reuse."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(page_table):
    if page_table.dim() != 2:
        raise ValueError("page_table is [num_seqs, max_pages]")
    return page_table.shape


def _space(workspace, size, device, stream):
    """The workspace to use: the caller's (any contiguous tensor on the device) or a new one."""
    if workspace is None:
        return _new(max(256, size()), torch.uint8, device, stream)
    if workspace.get_device() != device.index or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {device} is wanted")
    return workspace


def hstu_cache_append(cache: PagedCache, uvqk, seq_offsets, timestamps, page_table, cache_lens,
                      next_positions=None, stream=None) -> None:
    """The K and V rows of a jagged U|V|Q|K batch into the cache (see the C header); cache_lens is
    the caller's to advance."""
    B, M = _rows(page_table)
    T, i64 = int(uvqk.shape[0]), torch.int64
    _call(_lib.hstu_cache_append, "hstu_cache_append", cache.device, stream, cache.ref, B, T,
          *_args(cache.device, (
              ("uvqk", uvqk, cache.dtype, T * 4 * cache.num_heads * cache.head_dim),
              ("seq_offsets", seq_offsets, i64, B + 1), ("timestamps", timestamps, i64, T),
              ("page_table", page_table, torch.int32, B * M))), M,
          *_args(cache.device, (("cache_lens", cache_lens, i64, B),
                                ("next_positions", next_positions, i64, B))))


def paged_attention_workspace_size(shape: HstuShape) -> int:
    return int(_lib.hstu_paged_attention_workspace_size(ctypes.byref(shape)))


def hstu_paged_attention_fwd(shape: HstuShape, cache: PagedCache, uvqk, page_table, cache_lens,
                             next_positions, timestamps, pos_table, time_table, alibi_slopes,
                             scale: float, av, append: bool = True, workspace=None, stream=None):
    """Attention of one new token a sequence over its cached tokens and itself (see the C header);
    with `append` the token joins the cache.  Fills and returns av [B, H*hd] (fp32)."""
    B, M = _rows(page_table)
    w, dev, i64, f32 = cache.num_heads * cache.head_dim, cache.device, torch.int64, torch.float32
    if shape.num_seqs != B:
        raise ValueError(f"page_table has {B} rows, the shape {shape.num_seqs} sequences")
    H = shape.num_heads
    up, tp, lp, np_, sp, pos, tim, ali, ap = _args(dev, (
        ("uvqk", uvqk, cache.dtype, B * 4 * w), ("page_table", page_table, torch.int32, B * M),
        ("cache_lens", cache_lens, i64, B), ("next_positions", next_positions, i64, B),
        ("timestamps", timestamps, i64, B), ("pos_table", pos_table, f32, H * shape.n_pos_buckets),
        ("time_table", time_table, f32, H * shape.n_time_buckets),
        ("alibi_slopes", alibi_slopes, f32, H), ("av", av, f32, B * w)))
    ws = _space(workspace, lambda: paged_attention_workspace_size(shape), dev, stream)
    _call(_lib.hstu_paged_attention_fwd, "hstu_paged_attention_fwd", dev, stream, ctypes.byref(shape),
          cache.ref, up, tp, M, lp, np_, sp, pos, tim, ali, scale, 1 if append else 0, ap,
          ws.data_ptr(), ws.nbytes)
    return av


def paged_layer_workspace_size(shape: HstuShape) -> int:
    return int(_lib.hstu_paged_layer_workspace_size(ctypes.byref(shape)))


def hstu_paged_layer_fwd(shape: HstuShape, cache: PagedCache, X, page_table, cache_lens,
                         next_positions, timestamps, W1, b1, W2, b2, ln_w, ln_b, pos_table,
                         time_table, alibi_slopes, scale: float, out=None, append: bool = True,
                         workspace=None, stream=None):
    """One HSTU layer over one new token a sequence, against the layer's paged cache."""
    B, M = _rows(page_table)
    w, d, dt, dev = cache.num_heads * cache.head_dim, shape.d_model, cache.dtype, cache.device
    if shape.num_seqs != B:
        raise ValueError(f"page_table has {B} rows, the shape {shape.num_seqs} sequences")
    if out is None:
        out = _new(X.shape, dt, dev, stream)
    H, i64, f32 = shape.num_heads, torch.int64, torch.float32
    xp, tp, lp, np_, sp, pos, tim, ali, op, *weights = _args(dev, (
        ("X", X, dt, B * d), ("page_table", page_table, torch.int32, B * M),
        ("cache_lens", cache_lens, i64, B), ("next_positions", next_positions, i64, B),
        ("timestamps", timestamps, i64, B), ("pos_table", pos_table, f32, H * shape.n_pos_buckets),
        ("time_table", time_table, f32, H * shape.n_time_buckets),
        ("alibi_slopes", alibi_slopes, f32, H), ("out", out, dt, B * d),
        ("W1", W1, dt, d * 4 * w), ("b1", b1, dt, 4 * w), ("W2", W2, dt, w * d), ("b2", b2, dt, d),
        ("ln_w", ln_w, dt, w), ("ln_b", ln_b, dt, w)))
    ws = _space(workspace, lambda: paged_layer_workspace_size(shape), dev, stream)
    _call(_lib.hstu_paged_layer_fwd, "hstu_paged_layer_fwd", dev, stream, ctypes.byref(shape),
          cache.ref, xp, tp, M, lp, np_, sp, *weights, pos, tim, ali, scale, 1 if append else 0, op,
          ws.data_ptr(), ws.nbytes)
    return out


def cache_evict_workspace_size(cache: PagedCache, num_seqs: int, max_pages: int) -> int:
    return int(_lib.hstu_cache_evict_workspace_size(cache.ref, int(num_seqs), int(max_pages)))


def hstu_cache_evict(cache: PagedCache, page_table, cache_lens, next_positions, budget: int,
                     recent: int, new_lens=None, workspace=None, stream=None):
    """Cuts sequences above `budget` cached tokens to their `recent` newest and the most attended of
    the others (see the C header).  Returns new_lens [B] (cache_lens itself is allowed)."""
    B, M = _rows(page_table)
    dev, i64 = cache.device, torch.int64
    if new_lens is None:
        new_lens = _new(B, i64, dev, stream)
    tp, lp, np_, ep = _args(dev, (
        ("page_table", page_table, torch.int32, B * M), ("cache_lens", cache_lens, i64, B),
        ("next_positions", next_positions, i64, B), ("new_lens", new_lens, i64, B)))
    ws = _space(workspace, lambda: cache_evict_workspace_size(cache, B, M), dev, stream)
    _call(_lib.hstu_cache_evict, "hstu_cache_evict", dev, stream, cache.ref, B, tp, M, lp, np_, budget,
          recent, ep, ws.data_ptr(), ws.nbytes)
    return new_lens


def hstu_attention_bwd(shape: HstuShape, uvqk, seq_offsets, timestamps, pos_table, time_table,
                       alibi_slopes, scale: float, dav, dq, dk, dv, dpos_table=None,
                       dtime_table=None, workspace=None, stream=None):
    """Backward of Eq. 2 (see the C header): fills dq, dk, dv and the table gradients."""
    if workspace is None:
        workspace = torch.empty(max(256, int(_lib.hstu_attention_bwd_workspace_size(ctypes.byref(shape)))),
                                dtype=torch.uint8, device=uvqk.device)
    _check(_lib.hstu_attention_bwd(ctypes.byref(shape), _ptr(uvqk), _ptr(seq_offsets), _ptr(timestamps),
                                   _ptr(pos_table), _ptr(time_table), _ptr(alibi_slopes), float(scale),
                                   _ptr(dav), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dpos_table),
                                   _ptr(dtime_table), _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "hstu_attention_bwd")
    return dq, dk, dv


def layer_bwd_workspace_size(shape: HstuShape) -> int:
    return int(_lib.hstu_layer_bwd_workspace_size(ctypes.byref(shape)))


def hstu_layer_bwd(shape: HstuShape, X, seq_offsets, timestamps, W1, b1, W2, ln_w, ln_b,
                   pos_table, time_table, alibi_slopes, scale: float, fwd_workspace, dY, dX, dW1,
                   db1, dW2, db2, dln_w, dln_b, dpos_table=None, dtime_table=None, workspace=None,
                   stream=None):
    """Backward of one layer (see the C header): `fwd_workspace` is the workspace a preceding
    hstu_layer_fwd call with the same inputs filled; fills dX and every parameter gradient."""
    if workspace is None:
        workspace = torch.empty(max(256, layer_bwd_workspace_size(shape)), dtype=torch.uint8,
                                device=X.device)
    _check(_lib.hstu_layer_bwd(ctypes.byref(shape), _ptr(X), _ptr(seq_offsets), _ptr(timestamps),
                               _ptr(W1), _ptr(b1), _ptr(W2), _ptr(ln_w), _ptr(ln_b),
                               _ptr(pos_table), _ptr(time_table), _ptr(alibi_slopes), float(scale),
                               _ptr(fwd_workspace), fwd_workspace.numel(), _ptr(dY), _ptr(dX),
                               _ptr(dW1), _ptr(db1), _ptr(dW2), _ptr(db2), _ptr(dln_w),
                               _ptr(dln_b), _ptr(dpos_table), _ptr(dtime_table), _ptr(workspace),
                               workspace.numel(), _stream(stream)), "hstu_layer_bwd")
    return {"dX": dX, "dW1": dW1, "db1": db1, "dW2": dW2, "db2": db2, "dln_w": dln_w,
            "dln_b": dln_b, "dpos": dpos_table, "dtime": dtime_table}


class LayerPipeline:
    """hstu_layer_fwd over batches in host memory, the copies in and out overlapped with the
    layers of neighbouring batches (see the C header).  Host tensors should be pinned."""

    def __init__(self, capacity: HstuShape, depth: int = 2):
        self._p = ctypes.c_void_p()
        _check(_lib.hstu_layer_pipeline_create(ctypes.byref(capacity), int(depth),
                                               ctypes.byref(self._p)), "hstu_layer_pipeline_create")

    def submit(self, shape: HstuShape, X_host, seq_offsets_host, timestamps_host, W1, b1, W2, b2,
               ln_w, ln_b, pos_table, time_table, alibi_slopes, scale: float, out_host):
        _check(_lib.hstu_layer_pipeline_submit(
            self._p, ctypes.byref(shape), _ptr(X_host), _ptr(seq_offsets_host),
            _ptr(timestamps_host), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(ln_w), _ptr(ln_b),
            _ptr(pos_table), _ptr(time_table), _ptr(alibi_slopes), float(scale), _ptr(out_host)),
            "hstu_layer_pipeline_submit")
        return out_host

    def sync(self) -> None:
        _check(_lib.hstu_layer_pipeline_sync(self._p), "hstu_layer_pipeline_sync")

    def timing_begin(self) -> None:
        _check(_lib.hstu_layer_pipeline_timing_begin(self._p), "hstu_layer_pipeline_timing_begin")

    def timing_end(self) -> float:
        ms = ctypes.c_float()
        _check(_lib.hstu_layer_pipeline_timing_end(self._p, ctypes.byref(ms)),
               "hstu_layer_pipeline_timing_end")
        return float(ms.value)

    def close(self) -> None:
        if self._p:
            _lib.hstu_layer_pipeline_destroy(self._p)
            self._p = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hstu_stochastic_length(seq_offsets, max_len: int, alpha: float, u, keys, new_offsets, index,
                           workspace=None, stream=None):
    """Stochastic Length on the device (see the C header); returns (new_offsets, index)."""
    B = int(seq_offsets.numel()) - 1
    T = int(keys.numel())
    if workspace is None:
        workspace = torch.empty(max(256, int(_lib.hstu_stochastic_length_workspace_size(B))),
                                dtype=torch.uint8, device=seq_offsets.device)
    _check(_lib.hstu_stochastic_length(B, T, _ptr(seq_offsets), int(max_len), float(alpha),
                                       _ptr(u), _ptr(keys), _ptr(new_offsets), _ptr(index),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
           "hstu_stochastic_length")
    return new_offsets, index


def hstu_gather_rows(index, src, dst, row_count=None, stream=None):
    """dst[r] = src[index[r]] for r < row_count (a device int64 scalar) or all of dst's rows."""
    max_rows = int(dst.shape[0])
    row_bytes = int(dst[0].numel() * dst.element_size()) if dst.dim() > 1 else dst.element_size()
    _check(_lib.hstu_gather_rows(max_rows, _ptr(row_count), row_bytes, _ptr(index), _ptr(src),
                                 int(src.shape[0]), _ptr(dst), _stream(stream)), "hstu_gather_rows")
    return dst


def hstu_ln_gate_fwd(shape: HstuShape, av, uvqk, ln_w, ln_b, g, stream=None):
    _check(_lib.hstu_ln_gate_fwd(ctypes.byref(shape), _ptr(av), _ptr(uvqk), _ptr(ln_w), _ptr(ln_b),
                                 _ptr(g), _stream(stream)), "hstu_ln_gate_fwd")
    return g


def hstu_f2_fwd(shape: HstuShape, g, W2, b2, X, out, stream=None):
    _check(_lib.hstu_f2_fwd(ctypes.byref(shape), _ptr(g), _ptr(W2), _ptr(b2), _ptr(X), _ptr(out),
                            _stream(stream)), "hstu_f2_fwd")
    return out


def hstu_ln_f2_fwd(shape: HstuShape, av, uvqk, ln_w, ln_b, W2, b2, X, out, stream=None):
    """out = (LayerNorm(av) * U) W2 + b2 + X in one kernel (bf16, H*d_v == d in {128, 256, 512})."""
    _check(_lib.hstu_ln_f2_fwd(ctypes.byref(shape), _ptr(av), _ptr(uvqk), _ptr(ln_w), _ptr(ln_b),
                               _ptr(W2), _ptr(b2), _ptr(X), _ptr(out), _stream(stream)),
           "hstu_ln_f2_fwd")
    return out


def hstu_token_embed_fwd(item_ids, action_ids, item_table, action_table, out=None, stream=None):
    T = item_ids.numel()
    d = item_table.shape[1]
    if out is None:
        out = torch.empty((T, d), dtype=item_table.dtype, device=item_table.device)
    _check(_lib.hstu_token_embed_fwd(T, d, _ptr(item_ids), _ptr(action_ids), _ptr(item_table),
                                     item_table.shape[0], _ptr(action_table), action_table.shape[0],
                                     _ptr(out), _stream(stream)), "hstu_token_embed_fwd")
    return out


def device_status(stream=None) -> int:
    """Synchronises `stream`, then reads and clears the library's device status word."""
    return int(_lib.hstu_get_device_status(_stream(stream)))
