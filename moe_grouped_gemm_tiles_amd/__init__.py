"""Python binding of libdg (fine-grained-scaled FP8 GEMM for MI355X / gfx950).

A thin ctypes layer over the C ABI in ``include/dg.h``: it checks tensor
dtypes/devices, passes ``data_ptr()`` values and the current HIP stream, and
raises ``RuntimeError`` with the library's status text on failure.  All
arithmetic runs in the HIP kernels; PyTorch only provides device memory and
the stream.  Names mirror the DeepGEMM README ("Interfaces", "Utilities")
as mirrored on the page "Weight gradient kernels for dense and MoE models #95":

* ``fp8_gemm_nt((a, sfa), (b, sfb), d, c=None, workspace=None)``
* ``m_grouped_fp8_gemm_nt_contiguous((a, sfa), (b, sfb), d, m_indices)``
* ``m_grouped_fp8_gemm_nt_masked((a, sfa), (b, sfb), d, masked_m, expected_m)``
* ``k_grouped_fp8_gemm_nt_contiguous((a, sfa), (b, sfb), d, ks, c=None)``
* ``wgrad_fp8_gemm_nt((a, sfa), (b, sfb), d)`` and
  ``k_grouped_wgrad_fp8_gemm_nt((a, sfa), (b, sfb), d, ks)`` (D += ..., FP32)
* ``per_token_cast_to_fp8(x, q, sf)`` and ``per_block_cast_to_fp8(w, q, sf)``
  (the caller's FP8 cast, writing the scale layouts the GEMMs take)
* ``fp8_mqa_logits(q, (kv, kv_sf), weights, ks, ke, clean_logits, out)``
  (README "V3.2 MQA kernels for the indexer")
* ``add_rms_norm_cast_to_fp8(x, weight, eps, q, sf, residual, residual_out, y, rstd)``
  (residual addition, RMS norm and the per-token cast in one pass) and its
  gradient ``rms_norm_backward(dy, s, weight, rstd, dx, dw, dresidual)``
* ``fp8_moe_few_tokens((x, sfx), (w13, sf13), (w2, sf2), topk_ids, topk_weights, out)``
  (a whole gated expert layer for a few tokens, two launches)
* ``clip_grad_norm(grads, max_norm, norm, out)`` (global norm over many tensors
  and clipping by it; ``tensor_list`` keeps the descriptors between calls)
* ``cast_to_mxfp4(x, q, sf, y, masked_m)`` (microscaled 4-bit quantisation) and the
  products ``mxfp4_gemm_nt((a, sfa), (b, sfb), d, c, workspace)``,
  ``m_grouped_mxfp4_gemm_nt_contiguous((a, sfa), (b, sfb), d, m_indices)``,
  ``m_grouped_mxfp4_gemm_nt_masked((a, sfa), (b, sfb), d, masked_m, expected_m)``
* ``moe_router(logits, topk_ids, topk_weights, counts, prob_sum, loss, ...)`` (scores,
  choice of experts, weights, rows per expert, balance loss) and its gradient
  ``moe_router_backward(logits, topk_ids, dweights, dlogits, counts, prob_sum, dloss, ...)``
* ``get_mk_alignment_for_contiguous_layout()``, ``get_sf_aligned_size(mn)``,
  ``set_num_cus(n)`` / ``get_num_cus()``, ``get_workspace_size(m, n, k)`` and
  ``alloc_workspace(m, n, k)``

Skinny dense GEMMs (M <= 128) split K across workgroups and need a split-K
workspace (``get_workspace_size``): zero-filled device memory that the caller
keeps and passes to every call (``alloc_workspace`` makes one); each call
leaves it ready for the next.  Without one, the dense calls take a fresh
workspace from torch's allocator per call and clear its counters (one small
fill kernel before the GEMM).

The three M-side GEMMs take either FP32 scales or UE8M0 scales packed four
per int32 along K (the README's "Interfaces > Notices" names both formats);
the binding picks the entry point from the scale tensors' dtype.

Operands follow the ``(tensor, scale)`` pair convention of the README:
``a`` is E4M3 (``torch.float8_e4m3fn`` or ``torch.uint8`` codes) ``[M, K]``
(masked: ``[G, M_max, K]``), ``sfa`` is FP32 ``[K/128, ld]`` transposed
(masked: ``[G, K/128, ld]``), ``b`` is E4M3 ``[N, K]`` (grouped
``[G, N, K]``), ``sfb`` is FP32 ``[ceil(N/128), K/128]`` (grouped
``[G, ceil(N/128), K/128]``), ``d`` is a caller-allocated BF16 or FP32 tensor.
With UE8M0 scales, ``sfa`` is int32 ``[ceil(K/512), ld]`` (masked
``[G, ceil(K/512), ld]``) and ``sfb`` int32 ``[ceil(N/128), ceil(K/512)]``
(grouped ``[G, ...]``).

The 4-bit forms take bytes of two E2M1 codes (``torch.uint8`` or
``torch.float4_e2m1fn_x2``): ``a`` is ``[M, K/2]`` (masked ``[G, M_max, K/2]``), ``b``
``[N, K/2]`` (grouped ``[G, N, K/2]``), and both scales are int32 words of four E8M0 bytes,
transposed: ``sfa`` ``[K/128, ld >= M]``, ``sfb`` ``[K/128, ld >= N]`` (with a leading ``G``
where the operand has one).
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "fp8_gemm_nt",
    "m_grouped_fp8_gemm_nt_contiguous",
    "m_grouped_fp8_gemm_nt_masked",
    "k_grouped_fp8_gemm_nt_contiguous",
    "wgrad_fp8_gemm_nt",
    "k_grouped_wgrad_fp8_gemm_nt",
    "per_token_cast_to_fp8",
    "per_block_cast_to_fp8",
    "fp8_mqa_logits",
    "add_rms_norm_cast_to_fp8",
    "rms_norm_backward",
    "alloc_rms_norm_backward_workspace",
    "fp8_moe_few_tokens",
    "get_moe_workspace_size",
    "alloc_moe_workspace",
    "cast_to_mxfp4",
    "mxfp4_gemm_nt",
    "m_grouped_mxfp4_gemm_nt_contiguous",
    "m_grouped_mxfp4_gemm_nt_masked",
    "get_mxfp4_workspace_size",
    "alloc_mxfp4_workspace",
    "moe_router",
    "moe_router_backward",
    "alloc_moe_router_workspace",
    "clip_grad_norm",
    "alloc_clip_workspace",
    "TensorList",
    "tensor_list",
    "transform_sf_into_required_layout",
    "get_mn_major_tma_aligned_tensor",
    "get_mn_major_tma_aligned_packed_ue8m0_tensor",
    "get_mk_alignment_for_contiguous_layout",
    "get_sf_aligned_size",
    "set_num_cus",
    "get_num_cus",
    "get_workspace_size",
    "alloc_workspace",
    "set_num_sms",
    "get_num_sms",
    "get_tma_aligned_size",
    "library_path",
    "load_library",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdg.so")
_lib = None

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_STATUS = {0: "DG_SUCCESS"}

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int
_sz = ctypes.c_size_t

_f = ctypes.c_float

_SIGNATURES = {
    "dg_fp8_gemm_nt": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _i32,
                              _i32, _i32, _i32, _vp, _sz, _vp]),
    "dg_get_workspace_size": (_sz, [_i32, _i32, _i32]),
    "dg_fp8_gemm_nt_noalloc": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _i32,
                                      _i32, _i32, _i32, _vp]),
    "dg_m_grouped_fp8_gemm_nt_contiguous": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp,
                                                   _i32, _i32, _i32, _i32, _vp]),
    "dg_m_grouped_fp8_gemm_nt_masked": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp,
                                               _i32, _i32, _i32, _i32, _i32, _vp]),
    "dg_fp8_gemm_nt_ue8m0": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _i32,
                                    _i32, _i32, _i32, _vp, _sz, _vp]),
    "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp,
                                                         _i32, _i32, _i32, _i32, _vp]),
    "dg_m_grouped_fp8_gemm_nt_masked_ue8m0": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp,
                                                     _i32, _i32, _i32, _i32, _i32, _vp]),
    "dg_k_grouped_fp8_gemm_nt_contiguous": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                                   _i32, _i32, _i32, _i32, _vp]),
    "dg_wgrad_fp8_gemm_nt": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _sz,
                                    _vp]),
    "dg_k_grouped_wgrad_fp8_gemm_nt": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]),
    "dg_k_grouped_fp8_gemm_nt_contiguous_ue8m0": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                                         _i32, _i32, _i32, _i32, _vp]),
    "dg_k_grouped_wgrad_fp8_gemm_nt_ue8m0": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                                    _vp]),
    "dg_per_token_cast_to_fp8": (_i32, [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp]),
    "dg_per_block_cast_to_fp8": (_i32, [_vp, _i64, _i32, _vp, _i64, _vp, _i32, _i32, _i32, _vp]),
    "dg_fp8_mqa_logits": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp]),
    "dg_add_rms_norm_cast_to_fp8": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i32, _f, _vp, _i64, _vp, _i64,
                                           _i32, _vp, _i64, _vp, _i32, _i32, _vp]),
    "dg_rms_norm_backward": (_i32, [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _i32,
                                    _i32, _i32, _vp, _sz, _vp]),
    "dg_get_rms_norm_backward_workspace_size": (_sz, [_i32, _i32]),
    "dg_fp8_moe_few_tokens": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                     _i32, _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "dg_fp8_moe_few_tokens_ue8m0": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                           _i32, _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "dg_get_moe_workspace_size": (_sz, [_i32, _i32, _i32]),
    "dg_cast_to_mxfp4": (_i32, [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _vp]),
    "dg_mxfp4_gemm_nt": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                                _i32, _i32, _i32, _vp, _sz, _vp]),
    "dg_get_mxfp4_workspace_size": (_sz, [_i32, _i32, _i32]),
    "dg_m_grouped_mxfp4_gemm_nt_contiguous": (_i32, [_vp, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp,
                                                     _i32, _i32, _i32, _i32, _vp]),
    "dg_m_grouped_mxfp4_gemm_nt_masked": (_i32, [_vp, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp,
                                                 _i32, _i32, _i32, _i32, _i32, _vp]),
    "dg_moe_router": (_i32, [_vp, _i64, _i32, _vp, _vp, _i32, _i32, _f, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                             _vp, _sz, _vp]),
    "dg_get_moe_router_workspace_size": (_sz, [_i32, _i32]),
    "dg_moe_router_backward": (_i32, [_vp, _i64, _i32, _i32, _i32, _f, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                      _i32, _i32, _i32, _vp]),
    "dg_clip_grad_norm": (_i32, [_vp, _vp, _i32, _f, _vp, _vp, _sz, _vp]),
    "dg_get_clip_workspace_size": (_sz, []),
    "dg_transform_sf_into_required_layout": (_i32, [_vp, _vp, _i32, _i32, _i32, _i64, _i32, _vp]),
    "dg_get_mk_alignment_for_contiguous_layout": (_i32, []),
    "dg_get_sf_aligned_size": (_i64, [_i64]),
    "dg_set_num_cus": (_i32, [_i32]),
    "dg_get_num_cus": (_i32, []),
    "dg_internal_set_tile_n": (_i32, [_i32]),
    "dg_internal_dense_plan": (_i32, [_i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "dg_internal_mxfp4_plan": (_i32, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "dg_status_string": (ctypes.c_char_p, [_i32]),
    "dg_last_hip_error": (ctypes.c_char_p, []),
}


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libdg.so (built in-tree by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libdg.so not built: run `python -m moe_grouped_gemm_tiles_amd.build` "
                          f"(expected at {_LIB_PATH})")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        lib = load_library()
        msg = lib.dg_status_string(status).decode()
        hip = lib.dg_last_hip_error().decode()
        raise RuntimeError(msg + (f" ({hip})" if hip and status == 3 else ""))


def _stream(t: torch.Tensor) -> int:
    """The current HIP stream of t's device (0.1 us; building a torch.cuda.Stream for it takes 2 us)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _unit_last_stride(t: torch.Tensor) -> bool:
    return t.numel() == 0 or t.size(-1) == 1 or t.stride(-1) == 1


def _ld(t: torch.Tensor, dim: int = 0, align: int = 1) -> int:
    """Leading dimension (elements between consecutive indices of ``dim``).

    A dimension of size 1 may carry any stride in torch (and numpy), so there
    the dense row length, rounded up to ``align`` elements, is passed instead;
    the library never steps along that dimension then.
    """
    if t.size(dim) > 1:
        return t.stride(dim)
    row = 1
    for s in t.shape[dim + 1:]:
        row *= s
    return (row + align - 1) // align * align


def _fp8(t: torch.Tensor, name: str):
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{name} must be torch.float8_e4m3fn or uint8 codes, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not _unit_last_stride(t):
        raise ValueError(f"{name} must be K-contiguous")


def _f32(t: torch.Tensor, name: str):
    if t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a float32 GPU tensor")
    if not _unit_last_stride(t):
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _sf(sfa: torch.Tensor, sfb: torch.Tensor) -> bool:
    """Checks a scale pair; True for packed UE8M0 (int32), False for FP32."""
    if sfa.dtype != sfb.dtype or sfa.dtype not in (torch.float32, torch.int32):
        raise TypeError("sfa and sfb must both be float32 (FP32 scales) or both int32 (packed UE8M0)")
    for t, nm in ((sfa, "sfa"), (sfb, "sfb")):
        if not t.is_cuda:
            raise TypeError(f"{nm} must be a GPU tensor")
        if not _unit_last_stride(t):
            raise ValueError(f"{nm} must be contiguous in its last dimension")
    return sfa.dtype == torch.int32


def _sf_rows(k: int, ue8m0: bool) -> int:
    """Scale rows along K: K/128 FP32 scales, or ceil(K/512) packed UE8M0 words."""
    return (k // 128 + 3) // 4 if ue8m0 else k // 128


def _out(t: torch.Tensor, name: str = "d") -> int:
    if t.dtype not in _DTYPES or not t.is_cuda:
        raise TypeError(f"{name} must be a bfloat16 or float32 GPU tensor")
    if not _unit_last_stride(t):
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _DTYPES[t.dtype]


def _dense_contig(t: torch.Tensor, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def get_workspace_size(m: int, n: int, k: int) -> int:
    """Bytes of split-K workspace a dense M x N x K call needs on the current device (0: none)."""
    return int(load_library().dg_get_workspace_size(m, n, k))


def alloc_workspace(m: int, n: int, k: int, device=None) -> torch.Tensor | None:
    """A zero-filled split-K workspace for dense M x N x K calls (None when they need none).
    Keep it and pass it to every call of that shape; calls sharing it must not overlap."""
    size = get_workspace_size(m, n, k)
    if size == 0:
        return None
    return torch.zeros(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


_WS_ALIGN = 256  # the library's alignment rule for workspaces


def _workspace(m: int, n: int, k: int, workspace: torch.Tensor | None, like: torch.Tensor):
    """(pointer, bytes) of the split-K workspace for a dense call; without one, a fresh
    zero-filled workspace from torch's allocator (filled on the current stream)."""
    size = get_workspace_size(m, n, k)
    if size == 0:
        return None, 0
    if workspace is None:
        workspace = torch.zeros(size + _WS_ALIGN, dtype=torch.uint8, device=like.device)
        off = (-workspace.data_ptr()) % _WS_ALIGN
        workspace = workspace[off:off + size]
    elif not workspace.is_cuda or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the output's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fp8_gemm_nt(a_pair, b_pair, d: torch.Tensor, c: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None):
    """D = C + A @ B.T with A [M,K], B [N,K] E4M3 and FP32 or packed-UE8M0 fine-grained scales.
    ``workspace``: split-K workspace for skinny M (``alloc_workspace``), or None."""
    lib = load_library()
    a, sfa = a_pair
    b, sfb = b_pair
    _fp8(a, "a")
    _fp8(b, "b")
    ue = _sf(sfa, sfb)
    _dense_contig(sfb, "sfb")
    dt = _out(d)
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or d.shape != (m, n):
        raise ValueError(f"shape mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}, d {tuple(d.shape)}")
    kr = _sf_rows(k, ue)
    if sfa.dim() != 2 or sfa.shape[0] != kr or sfb.shape != ((n + 127) // 128, kr):
        raise ValueError(f"scale shapes: sfa {tuple(sfa.shape)}, sfb {tuple(sfb.shape)}")
    c_ptr, ldc = None, 0
    if c is not None:
        if c.dtype != d.dtype or c.shape != d.shape or not _unit_last_stride(c) or not c.is_cuda:
            raise ValueError("c must match d's dtype and shape")
        c_ptr, ldc = c.data_ptr(), _ld(c, 0, 16 // c.element_size())
    fn = lib.dg_fp8_gemm_nt_ue8m0 if ue else lib.dg_fp8_gemm_nt
    es = d.element_size()
    ws, ws_bytes = _workspace(m, n, k, workspace, d)
    st = fn(a.data_ptr(), _ld(a, 0, 16), sfa.data_ptr(), _ld(sfa, 0, 4), b.data_ptr(), _ld(b, 0, 16),
            sfb.data_ptr(), c_ptr, ldc, d.data_ptr(), _ld(d, 0, 16 // es), dt, m, n, k, ws, ws_bytes, _stream(d))
    _check(st)
    return d


def m_grouped_fp8_gemm_nt_contiguous(a_pair, b_pair, d: torch.Tensor, m_indices: torch.Tensor):
    """Contiguous-layout M-grouped GEMM; rows whose group index is -1 are left unwritten."""
    lib = load_library()
    a, sfa = a_pair
    b, sfb = b_pair
    for t, nm in ((a, "a"), (b, "b"), (sfb, "sfb"), (d, "d"), (m_indices, "m_indices")):
        _dense_contig(t, nm)
    _fp8(a, "a")
    _fp8(b, "b")
    ue = _sf(sfa, sfb)
    dt = _out(d)
    if m_indices.dtype != torch.int32 or not m_indices.is_cuda:
        raise TypeError("m_indices must be an int32 GPU tensor")
    m_total, k = a.shape
    g, n, kb_ = b.shape
    if kb_ != k or d.shape != (m_total, n) or m_indices.shape != (m_total,):
        raise ValueError("shape mismatch")
    kr = _sf_rows(k, ue)
    if sfa.dim() != 2 or sfa.shape[0] != kr or sfb.shape != (g, (n + 127) // 128, kr):
        raise ValueError("scale shape mismatch")
    fn = lib.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0 if ue else lib.dg_m_grouped_fp8_gemm_nt_contiguous
    st = fn(a.data_ptr(), sfa.data_ptr(), _ld(sfa, 0, 4), b.data_ptr(), sfb.data_ptr(), d.data_ptr(), dt,
            m_indices.data_ptr(), m_total, n, k, g, _stream(d))
    _check(st)
    return d


def m_grouped_fp8_gemm_nt_masked(a_pair, b_pair, d: torch.Tensor, masked_m: torch.Tensor,
                                 expected_m: int = 0):
    """Masked-layout M-grouped GEMM; rows at or beyond masked_m[g] are left unwritten."""
    lib = load_library()
    a, sfa = a_pair
    b, sfb = b_pair
    for t, nm in ((a, "a"), (sfa, "sfa"), (b, "b"), (sfb, "sfb"), (d, "d"), (masked_m, "masked_m")):
        _dense_contig(t, nm)
    _fp8(a, "a")
    _fp8(b, "b")
    ue = _sf(sfa, sfb)
    dt = _out(d)
    if masked_m.dtype != torch.int32 or not masked_m.is_cuda:
        raise TypeError("masked_m must be an int32 GPU tensor")
    g, m_max, k = a.shape
    n = b.shape[1]
    if b.shape != (g, n, k) or d.shape != (g, m_max, n) or masked_m.shape != (g,):
        raise ValueError("shape mismatch")
    kr = _sf_rows(k, ue)
    if sfa.dim() != 3 or sfa.shape[:2] != (g, kr) or sfb.shape != (g, (n + 127) // 128, kr):
        raise ValueError("scale shape mismatch")
    fn = lib.dg_m_grouped_fp8_gemm_nt_masked_ue8m0 if ue else lib.dg_m_grouped_fp8_gemm_nt_masked
    # sfa is contiguous [G, rows, L]: the library steps groups by rows * L, so L itself
    # (not a rounded-up stride) is the leading dimension it must validate
    st = fn(a.data_ptr(), sfa.data_ptr(), sfa.shape[2], b.data_ptr(), sfb.data_ptr(), d.data_ptr(), dt,
            masked_m.data_ptr(), g, m_max, n, k, int(expected_m), _stream(d))
    _check(st)
    return d


def _k_grouped_args(a_pair, b_pair, d: torch.Tensor, ks: torch.Tensor):
    a, sfa = a_pair
    b, sfb = b_pair
    for t, nm in ((a, "a"), (b, "b"), (sfb, "sfb"), (d, "d"), (ks, "ks")):
        _dense_contig(t, nm)
    _fp8(a, "a")
    _fp8(b, "b")
    ue = _sf(sfa, sfb)
    if d.dtype != torch.float32 or not d.is_cuda:
        raise TypeError("d must be a float32 GPU tensor")
    if ks.dtype != torch.int32 or not ks.is_cuda:
        raise TypeError("ks must be an int32 GPU tensor")
    m, k = a.shape
    n = b.shape[0]
    g = ks.shape[0]
    if b.shape != (n, k) or d.shape != (g, m, n) or ks.dim() != 1:
        raise ValueError("shape mismatch")
    kr = _sf_rows(k, ue)
    if sfa.dim() != 2 or sfa.shape[0] != kr or sfb.shape != ((n + 127) // 128, kr):
        raise ValueError("scale shape mismatch")
    return a, sfa, b, sfb, g, m, n, k, ue


def k_grouped_fp8_gemm_nt_contiguous(a_pair, b_pair, d: torch.Tensor, ks: torch.Tensor,
                                     c: torch.Tensor | None = None):
    """K-grouped GEMM: D[g] = C[g] + A[:, K_g] @ B[:, K_g].T (FP32), K_g given by ks (int32, device);
    FP32 scales or packed UE8M0 words (int32), by the scale tensors' dtype."""
    lib = load_library()
    a, sfa, b, sfb, g, m, n, k, ue = _k_grouped_args(a_pair, b_pair, d, ks)
    c_ptr = None
    if c is not None:
        if c.dtype != torch.float32 or c.shape != d.shape or not c.is_contiguous() or not c.is_cuda:
            raise ValueError("c must be a contiguous float32 GPU tensor shaped like d")
        c_ptr = c.data_ptr()
    fn = lib.dg_k_grouped_fp8_gemm_nt_contiguous_ue8m0 if ue else lib.dg_k_grouped_fp8_gemm_nt_contiguous
    st = fn(a.data_ptr(), sfa.data_ptr(), _ld(sfa, 0, 4), b.data_ptr(), sfb.data_ptr(), c_ptr, d.data_ptr(),
            ks.data_ptr(), g, m, n, k, _stream(d))
    _check(st)
    return d


def wgrad_fp8_gemm_nt(a_pair, b_pair, d: torch.Tensor, workspace: torch.Tensor | None = None):
    """Dense weight gradient: D += A @ B.T in FP32 (D is read and written).
    ``workspace``: split-K workspace for skinny M (``alloc_workspace``), or None."""
    lib = load_library()
    a, sfa = a_pair
    b, sfb = b_pair
    _fp8(a, "a")
    _fp8(b, "b")
    _f32(sfa, "sfa")
    _f32(sfb, "sfb")
    _dense_contig(sfb, "sfb")
    if d.dtype != torch.float32 or not d.is_cuda or not _unit_last_stride(d):
        raise TypeError("d must be a float32 GPU tensor, contiguous in its last dimension")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or d.shape != (m, n):
        raise ValueError("shape mismatch")
    if sfa.dim() != 2 or sfa.shape[0] != k // 128 or sfb.shape != ((n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    ws, ws_bytes = _workspace(m, n, k, workspace, d)
    st = lib.dg_wgrad_fp8_gemm_nt(a.data_ptr(), _ld(a, 0, 16), sfa.data_ptr(), _ld(sfa, 0, 4), b.data_ptr(),
                                  _ld(b, 0, 16), sfb.data_ptr(), d.data_ptr(), _ld(d, 0, 4), m, n, k, ws, ws_bytes,
                                  _stream(d))
    _check(st)
    return d


def k_grouped_wgrad_fp8_gemm_nt(a_pair, b_pair, d: torch.Tensor, ks: torch.Tensor):
    """K-grouped weight gradient: D[g] += A[:, K_g] @ B[:, K_g].T in FP32."""
    lib = load_library()
    a, sfa, b, sfb, g, m, n, k, ue = _k_grouped_args(a_pair, b_pair, d, ks)
    fn = lib.dg_k_grouped_wgrad_fp8_gemm_nt_ue8m0 if ue else lib.dg_k_grouped_wgrad_fp8_gemm_nt
    st = fn(a.data_ptr(), sfa.data_ptr(), _ld(sfa, 0, 4), b.data_ptr(), sfb.data_ptr(), d.data_ptr(),
            ks.data_ptr(), g, m, n, k, _stream(d))
    _check(st)
    return d


def _cast_args(x: torch.Tensor, q: torch.Tensor, sf: torch.Tensor):
    if x.dtype not in _DTYPES or not x.is_cuda or x.dim() != 2 or not _unit_last_stride(x):
        raise TypeError("x must be a 2-D bfloat16 or float32 GPU tensor, contiguous in its last dimension")
    _fp8(q, "q")
    if q.shape != x.shape:
        raise ValueError("q must have x's shape")
    if sf.dtype not in (torch.float32, torch.int32) or not sf.is_cuda or not _unit_last_stride(sf):
        raise TypeError("sf must be a float32 (FP32 scales) or int32 (packed UE8M0) GPU tensor")
    return _DTYPES[x.dtype], sf.dtype == torch.int32


def per_token_cast_to_fp8(x: torch.Tensor, q: torch.Tensor, sf: torch.Tensor):
    """Per-(row, 128-K) FP8 cast of x [M, K] into q [M, K] and the transposed scales sf:
    FP32 [K/128, ld >= M] or packed UE8M0 int32 [ceil(K/512), ld >= M]."""
    lib = load_library()
    dt, ue = _cast_args(x, q, sf)
    m, k = x.shape
    if sf.dim() != 2 or sf.shape[0] != _sf_rows(k, ue) or sf.shape[1] < m:
        raise ValueError(f"sf shape {tuple(sf.shape)} does not fit x {tuple(x.shape)}")
    st = lib.dg_per_token_cast_to_fp8(x.data_ptr(), _ld(x, 0, 16 // x.element_size()), dt, q.data_ptr(),
                                      _ld(q, 0, 8), sf.data_ptr(), _ld(sf, 0, 4), int(ue), m, k, _stream(x))
    _check(st)
    return q, sf


def per_block_cast_to_fp8(w: torch.Tensor, q: torch.Tensor, sf: torch.Tensor):
    """Per-128x128-block FP8 cast of w [N, K] into q [N, K] and sf: FP32 [ceil(N/128), K/128]
    or packed UE8M0 int32 [ceil(N/128), ceil(K/512)]."""
    lib = load_library()
    dt, ue = _cast_args(w, q, sf)
    n, k = w.shape
    _dense_contig(sf, "sf")
    if sf.shape != ((n + 127) // 128, _sf_rows(k, ue)):
        raise ValueError(f"sf shape {tuple(sf.shape)} does not fit w {tuple(w.shape)}")
    st = lib.dg_per_block_cast_to_fp8(w.data_ptr(), _ld(w, 0, 16 // w.element_size()), dt, q.data_ptr(),
                                      _ld(q, 0, 8), sf.data_ptr(), int(ue), n, k, _stream(w))
    _check(st)
    return q, sf


def fp8_mqa_logits(q: torch.Tensor, kv_pair, weights: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor,
                   clean_logits: bool, out: torch.Tensor):
    """Weighted-ReLU MQA logits: q E4M3 [S, H, D], kv (E4M3 [S_kv, D], FP32 scales [S_kv]),
    weights FP32 [S, H], key ranges ks/ke int32 [S] -> out FP32 [S, S_kv] (caller-allocated)."""
    lib = load_library()
    kv, kv_sf = kv_pair
    for t, nm in ((q, "q"), (kv, "kv"), (kv_sf, "kv_sf"), (weights, "weights"), (ks, "ks"), (ke, "ke")):
        _dense_contig(t, nm)
    _fp8(q, "q")
    _fp8(kv, "kv")
    _f32(kv_sf, "kv_sf")
    _f32(weights, "weights")
    if out.dtype != torch.float32 or not out.is_cuda or not _unit_last_stride(out):
        raise TypeError("out must be a float32 GPU tensor, contiguous in its last dimension")
    for t, nm in ((ks, "ks"), (ke, "ke")):
        if t.dtype != torch.int32 or not t.is_cuda:
            raise TypeError(f"{nm} must be an int32 GPU tensor")
    s, h, d = q.shape
    s_kv = kv.shape[0]
    if kv.shape != (s_kv, d) or kv_sf.shape != (s_kv,) or weights.shape != (s, h) or ks.shape != (s,) \
            or ke.shape != (s,) or out.shape != (s, s_kv):
        raise ValueError("shape mismatch")
    st = lib.dg_fp8_mqa_logits(q.data_ptr(), kv.data_ptr(), kv_sf.data_ptr(), weights.data_ptr(), ks.data_ptr(),
                               ke.data_ptr(), out.data_ptr(), _ld(out, 0, 1), s, s_kv, h, d, int(bool(clean_logits)),
                               _stream(out))
    _check(st)
    return out


def _like(t: torch.Tensor, dtype, dev: int, shape, name: str):
    """(pointer, row stride) of a 2-D operand of the given dtype, device and shape."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must have the input's dtype, device and shape {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    if not _unit_last_stride(t):
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr(), _ld(t, 0, 16 // t.element_size())


def _flat(t: torch.Tensor, dtype, dev: int, shape, name: str) -> int:
    """Pointer of a contiguous operand of the given dtype, device and shape."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the input's device")
    return t.data_ptr()


def _norm_input(x: torch.Tensor, weight: torch.Tensor, name: str):
    """(dtype, device index, shape, dtype code, pointer, row stride) of a norm's first operand, and
    (dtype code, pointer) of its weight."""
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    code = _DTYPES.get(dtype)
    if code is None or dev < 0 or len(shape) != 2:
        raise TypeError(f"{name} must be a 2-D bfloat16 or float32 GPU tensor")
    wcode = _DTYPES.get(weight.dtype)
    if wcode is None:
        raise TypeError("weight must be bfloat16 or float32")
    ptr, ld = _like(x, dtype, dev, shape, name)
    return dtype, dev, shape, code, ptr, ld, wcode, _flat(weight, weight.dtype, dev, shape[1:], "weight")


def _codes(t: torch.Tensor, dev: int, shape, name: str, align: int):
    """(pointer, row stride) of a 2-D operand of E4M3 codes."""
    if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
        raise TypeError(f"{name} must be torch.float8_e4m3fn or uint8 codes, got {t.dtype}")
    if t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be on the input's device and of shape {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    if not _unit_last_stride(t):
        raise ValueError(f"{name} must be K-contiguous")
    return t.data_ptr(), _ld(t, 0, align)


def _row_scales(sf: torch.Tensor, dev: int, m: int, k: int, name: str):
    """(UE8M0?, pointer, row stride) of transposed row scales [K/128 (or packed words), ld >= M]."""
    ue = sf.dtype is torch.int32
    if not ue and sf.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32 (FP32 scales) or int32 (packed UE8M0)")
    shape = sf.shape
    if sf.get_device() != dev or len(shape) != 2 or shape[0] != _sf_rows(k, ue) or shape[1] < m:
        raise ValueError(f"{name} shape {tuple(shape)} does not fit M = {m}, K = {k}")
    if shape[0] > 1 and sf.is_contiguous():
        return ue, sf.data_ptr(), shape[1]
    if not _unit_last_stride(sf):
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return ue, sf.data_ptr(), _ld(sf, 0, 4)


def _scratch(workspace: torch.Tensor | None, size: int, dev: int):
    """(tensor to keep alive, pointer, bytes) of a workspace with any contents; without one, a
    fresh one from torch's allocator (its blocks are at least 512-byte aligned)."""
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the output's device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def add_rms_norm_cast_to_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float, q: torch.Tensor, sf: torch.Tensor,
                             residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                             y: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """s = x + residual, v = s / sqrt(mean(s^2) + eps) * weight, and v's per-token FP8 cast in one
    pass: x [M, K] -> q E4M3 [M, K], sf FP32 [K/128, ld >= M] or packed UE8M0 int32 [ceil(K/512), ld]
    (the GEMMs' a operand), residual_out = s (may be residual itself).  Optional outputs: y = v in
    x's dtype, rstd FP32 [M] for ``rms_norm_backward``."""
    lib = _lib or load_library()
    dtype, dev, shape, code, xp, ldx, wcode, wp = _norm_input(x, weight, "x")
    m, k = shape
    qp, ldq = _codes(q, dev, shape, "q", 8)
    ue, sfp, ld_sf = _row_scales(sf, dev, m, k, "sf")
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    rp = rop = yp = rstdp = None
    ldr = ldro = ldy = 0
    if residual is not None:
        rp, ldr = _like(residual, dtype, dev, shape, "residual")
        rop, ldro = _like(residual_out, dtype, dev, shape, "residual_out")
    if y is not None:
        yp, ldy = _like(y, dtype, dev, shape, "y")
    if rstd is not None:
        rstdp = _flat(rstd, torch.float32, dev, shape[:1], "rstd")
    st = lib.dg_add_rms_norm_cast_to_fp8(xp, ldx, rp, ldr, rop, ldro, code, wp, wcode, eps, qp, ldq, sfp, ld_sf, ue, yp,
                                         ldy, rstdp, m, k, _stream(x))
    if st:
        _check(st)
    return q, sf


def alloc_rms_norm_backward_workspace(m: int, k: int, device=None) -> torch.Tensor:
    """A workspace for ``rms_norm_backward`` of [m, k] inputs (any contents)."""
    size = int(load_library().dg_get_rms_norm_backward_workspace_size(m, k))
    return torch.empty(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                      dw: torch.Tensor, dresidual: torch.Tensor | None = None, accumulate: bool = False,
                      workspace: torch.Tensor | None = None):
    """Gradient of the norm of ``add_rms_norm_cast_to_fp8``: dy [M, K] (of v), s the stored sum, rstd
    the forward's -> dx (of x and of residual alike; dresidual, the gradient that reached
    residual_out, is added) and dw FP32 [K] (overwritten, or added to with ``accumulate``).
    dx may be dy or dresidual itself."""
    lib = _lib or load_library()
    dtype, dev, shape, code, dyp, lddy, wcode, wp = _norm_input(dy, weight, "dy")
    m, k = shape
    sp, lds = _like(s, dtype, dev, shape, "s")
    dxp, lddx = _like(dx, dtype, dev, shape, "dx")
    rstdp = _flat(rstd, torch.float32, dev, shape[:1], "rstd")
    dwp = _flat(dw, torch.float32, dev, shape[1:], "dw")
    drp, lddr = _like(dresidual, dtype, dev, shape, "dresidual") if dresidual is not None else (None, 0)
    ws, wsp, wsb = _scratch(workspace, 0 if workspace is not None
                            else lib.dg_get_rms_norm_backward_workspace_size(m, k), dev)
    st = lib.dg_rms_norm_backward(dyp, lddy, sp, lds, code, wp, wcode, rstdp, drp, lddr, dxp, lddx, dwp, accumulate, m,
                                  k, wsp, wsb, _stream(dy))
    if st:
        _check(st)
    return dx, dw


def get_moe_workspace_size(m: int, top_k: int, inter: int) -> int:
    """Bytes of workspace ``fp8_moe_few_tokens`` needs for m tokens."""
    return int(load_library().dg_get_moe_workspace_size(m, top_k, inter))


def alloc_moe_workspace(m: int, top_k: int, inter: int, device=None) -> torch.Tensor:
    """A workspace for ``fp8_moe_few_tokens`` with up to m tokens (any contents)."""
    size = get_moe_workspace_size(m, top_k, inter)
    return torch.empty(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


def fp8_moe_few_tokens(x_pair, w13_pair, w2_pair, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                       out: torch.Tensor, workspace: torch.Tensor | None = None):
    """A whole gated expert layer for a few tokens: x E4M3 [M, H], w13 E4M3 [E, 2I, H] (gate rows,
    then up rows), w2 E4M3 [E, H, I], their scales in the GEMMs' layouts (FP32, or all packed UE8M0
    int32), topk_ids int32 [M, top_k] (ids outside [0, E) add nothing), topk_weights FP32
    [M, top_k] -> out BF16 [M, H]."""
    lib = _lib or load_library()
    x, sfx = x_pair
    w13, sf13 = w13_pair
    w2, sf2 = w2_pair
    dev = out.get_device()
    if dev < 0 or x.dim() != 2 or w13.dim() != 3 or topk_ids.dim() != 2:
        raise ValueError("x, topk_ids and out must be 2-D and the weights 3-D GPU tensors")
    shape = x.shape
    m, h = shape
    e, i, top_k = w13.shape[0], w13.shape[1] // 2, topk_ids.shape[1]
    xp, ldx = _codes(x, dev, shape, "x", 16)
    ue, sfxp, ld_sfx = _row_scales(sfx, dev, m, h, "sfx")
    sft = torch.int32 if ue else torch.float32
    for t, nm in ((w13, "w13"), (w2, "w2")):
        if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
            raise TypeError(f"{nm} must be torch.float8_e4m3fn or uint8 codes, got {t.dtype}")
    if out.dtype is not torch.bfloat16:
        raise TypeError("out must be a bfloat16 tensor")
    w13p = _flat(w13, w13.dtype, dev, (e, 2 * i, h), "w13")
    sf13p = _flat(sf13, sft, dev, (e, 2 * i // 128, _sf_rows(h, ue)), "sf13")
    w2p = _flat(w2, w2.dtype, dev, (e, h, i), "w2")
    sf2p = _flat(sf2, sft, dev, (e, h // 128, _sf_rows(i, ue)), "sf2")
    idp = _flat(topk_ids, torch.int32, dev, (m, top_k), "topk_ids")
    twp = _flat(topk_weights, torch.float32, dev, (m, top_k), "topk_weights")
    op, ldo = _like(out, torch.bfloat16, dev, shape, "out")
    ws, wsp, wsb = _scratch(workspace, 0 if workspace is not None else lib.dg_get_moe_workspace_size(m, top_k, i), dev)
    fn = lib.dg_fp8_moe_few_tokens_ue8m0 if ue else lib.dg_fp8_moe_few_tokens
    st = fn(xp, ldx, sfxp, ld_sfx, w13p, sf13p, w2p, sf2p, idp, twp, op, ldo, m, top_k, e, h, i, wsp, wsb, _stream(out))
    if st:
        _check(st)
    return out


class _Tensor(ctypes.Structure):
    """dg_tensor of the C ABI."""
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int)]


class TensorList:
    """The descriptors of a list of contiguous BF16 / FP32 tensors on one GPU, made once.  It holds
    references to the tensors, and is good for as long as each of them keeps its storage: every use
    checks their addresses and sizes (0.2 us a tensor) and raises ValueError where ``t.data = ...``,
    ``set_`` or ``resize_`` has given one another.  It knows nothing of other tensors that take their
    place: gradients that a backward pass makes anew (after ``zero_grad(set_to_none=True)``, torch's
    default) need a new list, or plain lists, each step."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.dev = self.tensors[0].get_device() if self.tensors else -1
        self.table = (_Tensor * max(1, len(self.tensors)))()
        for d, t in zip(self.table, self.tensors):
            if t.dtype not in _DTYPES or not t.is_cuda:
                raise TypeError("tensors must be bfloat16 or float32 GPU tensors")
            if t.get_device() != self.dev or not t.is_contiguous():
                raise ValueError("tensors must be contiguous and on one device")
            d.data, d.numel, d.dtype = t.data_ptr(), t.numel(), _DTYPES[t.dtype]
        self._places = self._now()

    def _now(self):
        return list(map(torch.Tensor.data_ptr, self.tensors)), list(map(torch.Tensor.numel, self.tensors))

    def __len__(self):
        return len(self.tensors)


def tensor_list(tensors) -> TensorList:
    """A ``TensorList`` for ``clip_grad_norm``."""
    return TensorList(tensors)


def _described(tensors, name: str) -> TensorList:
    """A list of tensors as a ``TensorList``; one that was made earlier has to describe its tensors still."""
    if not isinstance(tensors, TensorList):
        return TensorList(tensors)
    if tensors._now() != tensors._places:
        raise ValueError(f"{name}: a tensor's storage or size has changed since its TensorList was made")
    return tensors


def alloc_clip_workspace(device=None) -> torch.Tensor:
    """A workspace for ``clip_grad_norm`` (any contents)."""
    size = int(load_library().dg_get_clip_workspace_size())
    return torch.empty(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


def clip_grad_norm(grads, max_norm: float, norm: torch.Tensor, out=None, workspace: torch.Tensor | None = None):
    """norm[0] = sqrt(sum of all squares) and out = grads * min(1, max_norm / (norm + 1e-6)); without
    ``out`` in place.  grads and out: lists of tensors, or a ``TensorList`` kept between calls for tensors
    that keep their storage (gradients that are zeroed, not made anew)."""
    lib = _lib or load_library()
    grads = _described(grads, "grads")
    dev = norm.get_device()
    if norm.dtype is not torch.float32 or dev < 0 or norm.numel() != 1:
        raise TypeError("norm must be a float32 GPU tensor with one element")
    n = len(grads.tensors)
    if n and grads.dev != dev:
        raise ValueError("grads must be on norm's device")
    table = None
    if out is not None:
        out = _described(out, "out")
        if len(out.tensors) != n or (n and out.dev != dev):
            raise ValueError("out must have as many tensors as grads, on norm's device")
        table = out.table
    ws, wsp, wsb = _scratch(workspace, 0 if workspace is not None else lib.dg_get_clip_workspace_size(), dev)
    st = lib.dg_clip_grad_norm(grads.table, table, n, max_norm, norm.data_ptr(), wsp, wsb, _stream(norm))
    if st:
        _check(st)
    return norm


def _fp4(t: torch.Tensor, dev: int, ndim: int, name: str):
    """(pointer, bytes between rows) of an operand of packed 4-bit codes."""
    if t.dtype is not torch.uint8 and t.dtype is not torch.float4_e2m1fn_x2:
        raise TypeError(f"{name} must be bytes of two E2M1 codes (uint8 or float4_e2m1fn_x2), got {t.dtype}")
    if t.get_device() != dev or t.dim() != ndim:
        raise ValueError(f"{name} must be a {ndim}-D tensor on the output's device")
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    if ndim != 2 or not _unit_last_stride(t):
        raise ValueError(f"{name} must be contiguous" + (" in its last dimension" if ndim == 2 else ""))
    return t.data_ptr(), _ld(t, 0, 16)


def _fp4_scales(sf: torch.Tensor, dev: int, lead, kw: int, rows: int, name: str):
    """(pointer, words between scale rows) of packed scales [*lead, kw, ld >= rows]."""
    shape = tuple(sf.shape)
    if sf.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32 words of four E8M0 scales")
    if sf.get_device() != dev or shape[:-1] != (*lead, kw) or shape[-1] < rows:
        raise ValueError(f"{name} shape {shape} does not fit {(*lead, kw)} scale words of {rows} rows")
    if lead:
        _dense_contig(sf, name)
        return sf.data_ptr(), shape[-1]
    if not _unit_last_stride(sf):
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return sf.data_ptr(), _ld(sf, 0, 4)


def cast_to_mxfp4(x: torch.Tensor, q: torch.Tensor, sf: torch.Tensor, y: torch.Tensor | None = None,
                  masked_m: torch.Tensor | None = None):
    """Microscaled 4-bit cast of x [M, K] (or [G, M, K]): q [..., M, K/2] bytes of two E2M1 codes, sf int32
    [..., K/128, ld >= M] packed E8M0 scales of 32 values each, the operands of the mxfp4 GEMMs.  ``y``: the
    values they stand for, in x's dtype (for a straight-through forward; may be x).  ``masked_m`` int32 [G]:
    rows of each group that are there; the others are neither read nor written."""
    lib = _lib or load_library()
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    code, nd = _DTYPES.get(dtype), len(shape)
    if code is None or dev < 0 or nd not in (2, 3):
        raise TypeError("x must be a 2-D or 3-D bfloat16 or float32 GPU tensor")
    g, (m, k) = (1 if nd == 2 else shape[0]), shape[-2:]
    if nd == 2:
        xp, ldx = _like(x, dtype, dev, shape, "x")
    else:
        xp, ldx = _flat(x, dtype, dev, shape, "x"), k
    lead = tuple(shape[:-2])
    qp, ldq = _fp4(q, dev, nd, "q")
    if tuple(q.shape) != (*lead, m, k // 2) or k % 2:
        raise ValueError(f"q shape {tuple(q.shape)} does not fit x {tuple(shape)}")
    sfp, ld_sf = _fp4_scales(sf, dev, lead, k // 128, m, "sf")
    yp, ldy, mp = None, 0, None
    if y is not None:
        yp, ldy = _like(y, dtype, dev, shape, "y") if nd == 2 else (_flat(y, dtype, dev, shape, "y"), k)
    if masked_m is not None:
        if nd != 3:
            raise ValueError("masked_m goes with a 3-D x")
        mp = _flat(masked_m, torch.int32, dev, shape[:1], "masked_m")
    st = lib.dg_cast_to_mxfp4(xp, ldx, code, qp, ldq, sfp, ld_sf, yp, ldy, mp, g, m, k, _stream(x))
    if st:
        _check(st)
    return q, sf


def get_mxfp4_workspace_size(m: int, n: int, k: int) -> int:
    """Bytes of workspace a dense ``mxfp4_gemm_nt`` needs on the current device (0: none)."""
    return int(load_library().dg_get_mxfp4_workspace_size(m, n, k))


def alloc_mxfp4_workspace(m: int, n: int, k: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace for ``mxfp4_gemm_nt`` of these sizes (None when it needs none).  Keep it and pass
    it to every call of that shape; calls sharing it must not overlap."""
    size = get_mxfp4_workspace_size(m, n, k)
    if size == 0:
        return None
    return torch.zeros(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


def mxfp4_gemm_nt(a_pair, b_pair, d: torch.Tensor, c: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """D = C + A @ B.T with A [M, K], B [N, K] microscaled 4-bit operands (``cast_to_mxfp4``), D BF16 or FP32.
    ``workspace``: ``alloc_mxfp4_workspace``'s, or None."""
    lib = _lib or load_library()
    (a, sfa), (b, sfb) = a_pair, b_pair
    dev, es = d.get_device(), d.element_size()
    dt = _out(d)
    ap, lda = _fp4(a, dev, 2, "a")
    bp, ldb = _fp4(b, dev, 2, "b")
    m, kh = a.shape
    n = b.shape[0]
    if b.shape[1] != kh or d.shape != (m, n):
        raise ValueError(f"shape mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}, d {tuple(d.shape)}")
    kw = kh // 64
    sfap, ld_sfa = _fp4_scales(sfa, dev, (), kw, m, "sfa")
    sfbp, ld_sfb = _fp4_scales(sfb, dev, (), kw, n, "sfb")
    cp, ldc = None, 0
    if c is not None:
        if c.dtype != d.dtype or c.shape != d.shape or not _unit_last_stride(c) or c.get_device() != dev:
            raise ValueError("c must match d's dtype, shape and device")
        cp, ldc = c.data_ptr(), _ld(c, 0, 16 // es)
    size = lib.dg_get_mxfp4_workspace_size(m, n, 2 * kh)
    wp, wb = None, 0
    if size:
        if workspace is None:
            workspace = torch.zeros(size, dtype=torch.uint8, device=dev)
        _, wp, wb = _scratch(workspace, size, dev)
    st = lib.dg_mxfp4_gemm_nt(ap, lda, sfap, ld_sfa, bp, ldb, sfbp, ld_sfb, cp, ldc, d.data_ptr(), _ld(d, 0, 16 // es), dt,
                              m, n, 2 * kh, wp, wb, _stream(d))
    if st:
        _check(st)
    return d


def m_grouped_mxfp4_gemm_nt_contiguous(a_pair, b_pair, d: torch.Tensor, m_indices: torch.Tensor):
    """Contiguous-layout M-grouped product of 4-bit operands; rows whose group index is -1 are left unwritten."""
    lib = _lib or load_library()
    (a, sfa), (b, sfb) = a_pair, b_pair
    dev = d.get_device()
    dt = _out(d)
    _dense_contig(a, "a")
    _dense_contig(d, "d")
    ap, _ = _fp4(a, dev, 2, "a")
    bp, _ = _fp4(b, dev, 3, "b")
    m_total, kh = a.shape
    g, n = b.shape[:2]
    if b.shape[2] != kh or d.shape != (m_total, n):
        raise ValueError("shape mismatch")
    sfap, ld_sfa = _fp4_scales(sfa, dev, (), kh // 64, m_total, "sfa")
    sfbp, ld_sfb = _fp4_scales(sfb, dev, (g,), kh // 64, n, "sfb")
    ip = _flat(m_indices, torch.int32, dev, (m_total,), "m_indices")
    st = lib.dg_m_grouped_mxfp4_gemm_nt_contiguous(ap, sfap, ld_sfa, bp, sfbp, ld_sfb, d.data_ptr(), dt, ip, m_total, n,
                                                   2 * kh, g, _stream(d))
    if st:
        _check(st)
    return d


def m_grouped_mxfp4_gemm_nt_masked(a_pair, b_pair, d: torch.Tensor, masked_m: torch.Tensor, expected_m: int = 0):
    """Masked-layout M-grouped product of 4-bit operands; rows at or beyond masked_m[g] are left unwritten."""
    lib = _lib or load_library()
    (a, sfa), (b, sfb) = a_pair, b_pair
    dev = d.get_device()
    dt = _out(d)
    _dense_contig(d, "d")
    ap, _ = _fp4(a, dev, 3, "a")
    bp, _ = _fp4(b, dev, 3, "b")
    g, m_max, kh = a.shape
    n = b.shape[1]
    if b.shape != (g, n, kh) or d.shape != (g, m_max, n):
        raise ValueError("shape mismatch")
    sfap, ld_sfa = _fp4_scales(sfa, dev, (g,), kh // 64, m_max, "sfa")
    sfbp, ld_sfb = _fp4_scales(sfb, dev, (g,), kh // 64, n, "sfb")
    mp = _flat(masked_m, torch.int32, dev, (g,), "masked_m")
    st = lib.dg_m_grouped_mxfp4_gemm_nt_masked(ap, sfap, ld_sfa, bp, sfbp, ld_sfb, d.data_ptr(), dt, mp, g, m_max, n,
                                               2 * kh, int(expected_m), _stream(d))
    if st:
        _check(st)
    return d


_SCORES = {"softmax": 0, "sigmoid": 1}


def _router_input(logits: torch.Tensor, topk_ids: torch.Tensor, score: str):
    """(dtype code, device index, shape, top_k, pointer, row stride, pointer of the ids, score code)."""
    dtype, dev, shape = logits.dtype, logits.get_device(), logits.shape
    code = _DTYPES.get(dtype)
    if code is None or dev < 0 or len(shape) != 2:
        raise TypeError("logits must be a 2-D bfloat16 or float32 GPU tensor")
    sc = _SCORES.get(score)
    if sc is None:
        raise ValueError(f"score must be one of {tuple(_SCORES)}, got {score!r}")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [M, top_k]")
    if not _unit_last_stride(logits):
        raise ValueError("logits must be contiguous in its last dimension")
    k = topk_ids.shape[1]
    return (code, dev, shape, k, logits.data_ptr(), _ld(logits), _flat(topk_ids, torch.int32, dev, (shape[0], k), "topk_ids"),
            sc)


def alloc_moe_router_workspace(m: int, num_experts: int, device=None) -> torch.Tensor:
    """A workspace for ``moe_router`` of [m, num_experts] logits (any contents)."""
    size = int(load_library().dg_get_moe_router_workspace_size(m, num_experts))
    return torch.empty(size, dtype=torch.uint8, device=device if device is not None else torch.cuda.current_device())


def moe_router(logits: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, counts: torch.Tensor | None = None,
               prob_sum: torch.Tensor | None = None, loss: torch.Tensor | None = None, *, score: str = "softmax",
               bias: torch.Tensor | None = None, mask: torch.Tensor | None = None, normalize: bool = True,
               scale: float = 1.0, workspace: torch.Tensor | None = None):
    """Choice of experts for logits [M, E]: topk_ids int32 [M, top_k] (largest first, -1 where there is none left) and
    topk_weights FP32 [M, top_k], ``scale`` times the chosen scores, divided by their sum with ``normalize``.
    ``bias`` FP32 [E] is added to the scores for the choice alone; rows whose ``mask`` (bool [M]) is false are
    padding.  Optional: counts int32 [E], how often each expert was chosen, and with them prob_sum FP32 [E], the sums
    of the rows' score shares, and the balance loss FP32 [1], E * sum(counts * prob_sum) / (sum(counts) *
    sum(prob_sum))."""
    lib = _lib or load_library()
    code, dev, shape, k, xp, ld, idp, sc = _router_input(logits, topk_ids, score)
    m, e = shape
    wp = _flat(topk_weights, torch.float32, dev, (m, k), "topk_weights")
    bp = mp = cp = pp = lp = wsp = None
    wsb = 0
    if bias is not None:
        bp = _flat(bias, torch.float32, dev, (e,), "bias")
    if mask is not None:
        mp = _flat(mask, torch.bool, dev, (m,), "mask")
    if (prob_sum is None) != (loss is None) or (loss is not None and counts is None):
        raise ValueError("prob_sum and loss go together, and with counts")
    if counts is not None:
        cp = _flat(counts, torch.int32, dev, (e,), "counts")
        workspace, wsp, wsb = _scratch(workspace, 0 if workspace is not None
                                       else lib.dg_get_moe_router_workspace_size(m, e), dev)
        if loss is not None:
            pp, lp = _flat(prob_sum, torch.float32, dev, (e,), "prob_sum"), _flat(loss, torch.float32, dev, (1,), "loss")
    st = lib.dg_moe_router(xp, ld, code, bp, mp, sc, normalize, scale, idp, wp, cp, pp, lp, m, e, k, wsp, wsb,
                           _stream(logits))
    if st:
        _check(st)
    return topk_ids, topk_weights


def moe_router_backward(logits: torch.Tensor, topk_ids: torch.Tensor, dweights: torch.Tensor, dlogits: torch.Tensor,
                        counts: torch.Tensor | None = None, prob_sum: torch.Tensor | None = None,
                        dloss: torch.Tensor | None = None, *, score: str = "softmax", normalize: bool = True,
                        scale: float = 1.0):
    """Gradient of ``moe_router`` by the logits: dweights FP32 [M, top_k] is that of topk_weights, dloss FP32 [1] that of
    the balance loss (with the forward's counts and prob_sum, or their sums over data-parallel ranks) -> dlogits
    [M, E] in logits' dtype (may be logits itself)."""
    lib = _lib or load_library()
    code, dev, shape, k, xp, ld, idp, sc = _router_input(logits, topk_ids, score)
    m, e = shape
    dwp = _flat(dweights, torch.float32, dev, (m, k), "dweights")
    if dlogits.dtype is not logits.dtype or dlogits.get_device() != dev or dlogits.shape != shape \
            or not _unit_last_stride(dlogits):
        raise ValueError("dlogits must have logits' dtype, device and shape and be contiguous in its last dimension")
    cp = pp = lp = None
    if not (counts is None) == (prob_sum is None) == (dloss is None):
        raise ValueError("counts, prob_sum and dloss go together")
    if dloss is not None:
        cp = _flat(counts, torch.int32, dev, (e,), "counts")
        pp, lp = _flat(prob_sum, torch.float32, dev, (e,), "prob_sum"), _flat(dloss, torch.float32, dev, (1,), "dloss")
    st = lib.dg_moe_router_backward(xp, ld, code, sc, normalize, scale, idp, dwp, cp, pp, lp, dlogits.data_ptr(),
                                    _ld(dlogits), m, e, k, _stream(logits))
    if st:
        _check(st)
    return dlogits


def transform_sf_into_required_layout(sf: torch.Tensor, ue8m0: bool = False) -> torch.Tensor:
    """Per-row scales FP32 [mn, kb] (or [G, mn, kb]) -> the GEMM's sfa layout: FP32 [kb, ld]
    (or [G, kb, ld]) transposed with ld = get_sf_aligned_size(mn), or with ``ue8m0`` the packed
    int32 words [ceil(kb/4), ld] holding each scale's exponent byte (powers of two)."""
    lib = load_library()
    if sf.dtype != torch.float32 or not sf.is_cuda or sf.dim() not in (2, 3):
        raise TypeError("sf must be a float32 GPU tensor [mn, kb] or [G, mn, kb]")
    x = sf.contiguous()
    g, mn, kb = (1, *x.shape) if x.dim() == 2 else x.shape
    ld = int(lib.dg_get_sf_aligned_size(mn))
    rows = (kb + 3) // 4 if ue8m0 else kb
    out = torch.empty((g, rows, ld), dtype=torch.int32 if ue8m0 else torch.float32, device=x.device)
    _check(lib.dg_transform_sf_into_required_layout(x.data_ptr(), out.data_ptr(), g, mn, kb, ld,
                                                    1 if ue8m0 else 0, _stream(out)))
    return out[0] if sf.dim() == 2 else out


def get_mn_major_tma_aligned_tensor(sf: torch.Tensor) -> torch.Tensor:
    """Transposed, 16-byte aligned FP32 scales (the README's name for the FP32 form)."""
    return transform_sf_into_required_layout(sf, ue8m0=False)


def get_mn_major_tma_aligned_packed_ue8m0_tensor(sf: torch.Tensor) -> torch.Tensor:
    """Transposed, aligned scales packed into UE8M0 words (scales must be powers of two)."""
    return transform_sf_into_required_layout(sf, ue8m0=True)


def get_mk_alignment_for_contiguous_layout() -> int:
    return load_library().dg_get_mk_alignment_for_contiguous_layout()


def get_sf_aligned_size(mn: int) -> int:
    return load_library().dg_get_sf_aligned_size(mn)


def set_num_cus(n: int):
    _check(load_library().dg_set_num_cus(n))


def get_num_cus() -> int:
    return load_library().dg_get_num_cus()


def _set_tile_n_for_tests(w: int):
    """Force the width of the 256-row tiles (256, 224 or 160; 0 = chosen per call).
    Not part of the API: the tests use it to cover every tile width."""
    _check(load_library().dg_internal_set_tile_n(w))


def _dense_plan_for_tests(m: int, n: int, k: int, cus: int) -> dict:
    """The tile, K split and workspace size a dense call of this shape gets on a
    device with `cus` usable CUs.  Not part of the API: the tests pin the planner."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    ws = ctypes.c_size_t(0)
    _check(load_library().dg_internal_dense_plan(m, n, k, cus, *[ctypes.byref(v) for v in vals], ctypes.byref(ws)))
    bm, bn, splits, sps = (v.value for v in vals)
    return dict(bm=bm, bn=bn, splits=splits, slabs_per_split=sps, ws_bytes=ws.value)


def _mxfp4_plan_for_tests(mode: str, rows: int, n: int, k: int, cus: int = 256, groups: int = 1, most_rows: int = 0) -> dict:
    """The tile, K split and workspace size a 4-bit call gets.  Not part of the API: the tests pin the planner."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    ws = ctypes.c_size_t(0)
    _check(load_library().dg_internal_mxfp4_plan(("dense", "contiguous", "masked").index(mode), groups, rows, max(rows, most_rows),
                                                 n, k, cus, *[ctypes.byref(v) for v in vals], ctypes.byref(ws)))
    bm, bn, streaming, splits = (v.value for v in vals)
    return dict(bm=bm, bn=bn, streaming=bool(streaming), splits=splits, ws_bytes=ws.value)


# The README's names for the same utilities ("Utilities": set_num_sms / get_num_sms cap the
# compute units used; get_tma_aligned_size is the aligned leading dimension of the scales).
set_num_sms = set_num_cus
get_num_sms = get_num_cus
get_tma_aligned_size = get_sf_aligned_size
