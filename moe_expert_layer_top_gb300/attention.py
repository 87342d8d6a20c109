"""The attention in front of the MoE step, for PyTorch device memory and streams.

Three calls over the C ABI, in the order a decoder layer makes them:

* ``qkv_append``: RMSNorm of each query and key head, rotary positions, and
  the MXFP4 append of keys and values to a paged cache;
* ``attend_paged``: attention of the newest rows of each sequence (single
  tokens, or the rows of a verify step) over that cache;
* ``attend_prompt``: causal attention over packed prompts in 16 bits. Given
  ``k_cached`` and ``v_cached`` of ``qkv_append`` it attends over the very
  values that later steps read from the cache.

PyTorch only supplies device memory and streams here; every step runs in
libmoe.so, and a failed call raises. Sizes that live on the device (lengths,
pages, slots, positions) are checked there: pass ``d_status``, an int32 tensor
set to MOE_OK, and look at it when convenient (MOE_ERR_DEVICE_BOUNDS: something
was out of range and was not accessed).

The calls run on the tensors' device and on its current stream unless ``stream``
is given. Outputs and workspaces come from PyTorch's allocator, so calls on
several streams and captured graphs do not share any. A tensor that is used on
another stream than the one it was allocated on is kept alive by the caller
(``Tensor.record_stream``), as for any PyTorch operator.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import abi

_DTYPES = {torch.bfloat16: abi.MOE_DTYPE_BF16, torch.float16: abi.MOE_DTYPE_F16}


@dataclass
class KVCacheMXFP4:
    """A paged key/value cache in MXFP4 (uint8 tensors, contiguous, on one CUDA device).

    k_codes, v_codes:   [pages][kv heads][page size][head_dim/2], two E2M1 codes per byte (element 2i low)
    k_scales, v_scales: [pages][kv heads][page size][head_dim/32], UE8M0
    """
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    def __post_init__(self):
        pages, heads, page, half = _shape(self.k_codes, 4, "k_codes")
        want = {"k_codes": half, "v_codes": half, "k_scales": half // 16, "v_scales": half // 16}
        for name, width in want.items():
            t = getattr(self, name)
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.device != self.k_codes.device:
                raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor on the cache's device")
            if tuple(t.shape) != (pages, heads, page, width):
                raise ValueError(f"{name} must have shape {(pages, heads, page, width)}, not {tuple(t.shape)}")

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda") -> "KVCacheMXFP4":
        def make(width):
            return torch.empty((num_pages, num_kv_heads, page_size, width), dtype=torch.uint8, device=device)
        return cls(make(head_dim // 2), make(head_dim // 32), make(head_dim // 2), make(head_dim // 32))

    @property
    def head_dim(self) -> int:
        return 2 * self.k_codes.shape[3]

    @property
    def num_kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    def as_abi(self) -> abi.MoeKvCache:
        pages, heads, page, half = self.k_codes.shape
        return abi.MoeKvCache(self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                              self.v_scales.data_ptr(), pages, page, heads, 2 * half)


def rope_table(positions: int, rotary_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [positions][rotary_dim]: rotary_dim/2 cosines, then as many sines, of p * theta^(-2i/rotary_dim).
    The angles are computed in 64 bits: in 32, those of far positions would be off by whole radians."""
    freq = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().to(device)


def _shape(t: torch.Tensor, dims: int, name: str):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    return t.shape


def _rows(t: torch.Tensor, name: str, like: torch.Tensor | None = None) -> int:
    """Row stride of a [rows][heads][dim] tensor whose rows are contiguous."""
    rows, heads, dim = _shape(t, 3, name)
    if not t.is_cuda or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a CUDA tensor in bf16 or fp16")
    if like is not None and (t.device != like.device or t.dtype != like.dtype):
        raise ValueError(f"{name} must have the device and type of q")
    if t.numel() == 0:  # strides of an empty tensor say nothing
        return heads * dim
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return t.stride(0) if rows > 1 else heads * dim


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, like: torch.Tensor) -> torch.Tensor:
    if t.dtype != dtype or t.device != like.device or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on q's device")
    return t


def _status(t: torch.Tensor | None, like: torch.Tensor):
    if t is not None and (t.dtype != torch.int32 or t.device != like.device or t.numel() < 1):
        raise ValueError("d_status must be an int32 tensor on q's device")
    return t


def _out(out: torch.Tensor | None, q: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    return out


def _stream(stream, like: torch.Tensor):
    return stream if stream is not None else torch.cuda.current_stream(like.device)


def qkv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, positions: torch.Tensor | None = None,
               rope: torch.Tensor | None = None, interleaved: bool = False, q_norm: torch.Tensor | None = None,
               k_norm: torch.Tensor | None = None, eps: float = 1e-6, cache: KVCacheMXFP4 | None = None,
               slots: torch.Tensor | None = None, q_out: torch.Tensor | None = None, rotated_keys: bool = False,
               cached_values: bool = False, d_status: torch.Tensor | None = None, stream=None) -> dict:
    """Norm, rotation and append of T tokens in one pass.

    q [T][heads][D], k and v [T][kv heads][D] (bf16 or fp16; views of one fused projection are fine).
    rope fp32 [positions][R] as from ``rope_table``, R <= D, with positions int32 [T]; None: no rotation.
    q_norm, k_norm [D]: RMSNorm weights; None: that part is not normalised.
    cache with slots int64 [T] (page * page size + offset; negative: the token is not cached).
    q_out: a contiguous output for q, which may be q itself.

    Returns {"q"}, plus "k" (rotated keys in 16 bits) with rotated_keys, plus "k_cached" and "v_cached" (the
    values that the 4-bit cache keeps) with cached_values.
    """
    q_stride, k_stride, v_stride = _rows(q, "q"), _rows(k, "k", q), _rows(v, "v", q)
    T, H, D = q.shape
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != D:
        raise ValueError("k and v must be [T][kv heads][D] with the T and D of q")
    K = k.shape[1]
    R = 0
    if rope is not None:
        if rope.dim() != 2 or rope.dtype != torch.float32 or rope.device != q.device or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous fp32 [positions][rotary_dim] tensor on q's device")
        if positions is None:
            raise ValueError("rope needs positions")
        _vector(positions, "positions", torch.int32, T, q)
        R = rope.shape[1]
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None:
            _vector(w, name, q.dtype, D, q)
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots go together")
    if cache is not None:
        if cache.k_codes.device != q.device or (cache.num_kv_heads, cache.head_dim) != (K, D):
            raise ValueError("the cache must be on q's device, with the kv heads and head size of k")
        _vector(slots, "slots", torch.int64, T, q)
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != q.device or not q_out.is_contiguous():
        raise ValueError("q_out must be contiguous, with the shape, type and device of q")
    out = {"q": q_out}
    kv = dict(size=(T, K, D), dtype=q.dtype, device=q.device)
    if rotated_keys:
        out["k"] = torch.empty(**kv)
    if cached_values:
        out["k_cached"], out["v_cached"] = torch.empty(**kv), torch.empty(**kv)
    io = abi.MoeQkvAppendIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, T, H, K, D,
                            _DTYPES[q.dtype], R, int(interleaved), rope.shape[0] if rope is not None else 0,
                            abi.ptr(rope), abi.ptr(positions) if R else None, abi.ptr(q_norm), abi.ptr(k_norm), eps,
                            abi.ptr(slots), q_out.data_ptr(), abi.ptr(out.get("k")), abi.ptr(out.get("k_cached")),
                            abi.ptr(out.get("v_cached")))
    with torch.cuda.device(q.device):
        abi.check("moe_qkv_append", abi.moe_qkv_append(io, cache.as_abi() if cache is not None else None,
                                                       _status(d_status, q), _stream(stream, q)))
    return out


def attend_paged(q: torch.Tensor, cache: KVCacheMXFP4, page_table: torch.Tensor, lengths: torch.Tensor,
                 cu_rows: torch.Tensor, *, max_rows: int = 1, scale: float | None = None,
                 out: torch.Tensor | None = None, return_lse: bool = False, d_status: torch.Tensor | None = None,
                 stream=None):
    """Attention of the newest rows of each sequence over the MXFP4 cache.

    q [rows][heads][D]; page_table int32 [sequences][pages]; lengths int32 [sequences], the tokens in the
    cache with the query rows among them; cu_rows int32 [sequences + 1]: sequence b has rows
    cu_rows[b] .. cu_rows[b + 1] - 1, its last tokens, each seeing the keys up to itself. max_rows: the rows a
    sequence usually has at most (it picks the kernel variant; the result does not depend on it).
    scale: of the scores, 1/sqrt(D) by default. Rows that see no key give 0 and lse -inf.

    Returns out [rows][heads][D], and with return_lse also lse fp32 [rows][heads].
    """
    q_stride = _rows(q, "q")
    T, H, D = q.shape
    B = lengths.shape[0] if lengths.dim() == 1 else -1
    _vector(lengths, "lengths", torch.int32, B, q)
    _vector(cu_rows, "cu_rows", torch.int32, B + 1, q)
    if page_table.dtype != torch.int32 or page_table.device != q.device or page_table.dim() != 2 or \
            page_table.shape[0] != B or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [sequences][pages] tensor on q's device")
    if cache.k_codes.device != q.device or cache.head_dim != D:
        raise ValueError("the cache must be on q's device, with q's head size")
    out = _out(out, q)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    io = abi.MoeAttendPagedIO(q.data_ptr(), q_stride, out.data_ptr(), _rows(out, "out", q), abi.ptr(lse),
                              page_table.data_ptr(), lengths.data_ptr(), cu_rows.data_ptr(), B, T,
                              page_table.shape[1], max_rows, H, _DTYPES[q.dtype],
                              D ** -0.5 if scale is None else scale)
    c = cache.as_abi()
    st = _stream(stream, q)
    with torch.cuda.device(q.device), torch.cuda.stream(_torch_stream(st, q) if stream is not None else None):
        n = abi.moe_attend_paged_workspace(io, c)
        workspace = torch.empty((n,), dtype=torch.uint8, device=q.device) if n else None
        abi.check("moe_attend_paged", abi.moe_attend_paged(io, c, workspace, n, _status(d_status, q), st))
    return (out, lse) if return_lse else out


def _torch_stream(st, like: torch.Tensor):
    """The stream as a torch stream: the workspace is allocated on it, so that it is not handed out again before
    the call has run."""
    return torch.cuda.ExternalStream(st, device=like.device) if isinstance(st, int) else st


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, cu_keys: torch.Tensor, *,
                  causal: bool = True, scale: float | None = None, out: torch.Tensor | None = None,
                  return_lse: bool = False, d_status: torch.Tensor | None = None, stream=None):
    """Attention over packed prompts, or over chunks of prompts with the keys before them.

    q [rows][heads][D], k and v [keys][kv heads][D]; cu_rows, cu_keys int32 [sequences + 1]. Row i of a sequence
    with n rows and m keys sees keys 0 .. m - n + i (causal), or all m. Rows that see no key give 0 and lse -inf.

    Returns out [rows][heads][D], and with return_lse also lse fp32 [rows][heads].
    """
    q_stride, k_stride, v_stride = _rows(q, "q"), _rows(k, "k", q), _rows(v, "v", q)
    T, H, D = q.shape
    if k.shape != v.shape or k.shape[2] != D:
        raise ValueError("k and v must be [keys][kv heads][D] with the D of q")
    n = cu_rows.shape[0] if cu_rows.dim() == 1 else 0
    if n < 1:
        raise ValueError("cu_rows needs an entry for each sequence and one for the end")
    _vector(cu_rows, "cu_rows", torch.int32, n, q)
    _vector(cu_keys, "cu_keys", torch.int32, n, q)
    out = _out(out, q)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    io = abi.MoeAttendPromptIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, out.data_ptr(),
                               _rows(out, "out", q), abi.ptr(lse), cu_rows.data_ptr(), cu_keys.data_ptr(), n - 1, T,
                               k.shape[0], H, k.shape[1], D, _DTYPES[q.dtype], int(causal),
                               D ** -0.5 if scale is None else scale)
    with torch.cuda.device(q.device):
        abi.check("moe_attend_prompt", abi.moe_attend_prompt(io, _status(d_status, q), _stream(stream, q)))
    return (out, lse) if return_lse else out
