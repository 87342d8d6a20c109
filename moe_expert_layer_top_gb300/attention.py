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
is given. Outputs and workspaces come from PyTorch's allocator, on the stream
of the call, so calls on several streams and captured graphs do not share any
and none is handed out again before the call has run. A tensor that is used on
another stream than the one it was allocated on is kept alive by the caller
(``Tensor.record_stream``), as for any PyTorch operator.
"""
from __future__ import annotations

import functools

import torch

from . import abi

_DTYPES = {torch.bfloat16: abi.MOE_DTYPE_BF16, torch.float16: abi.MOE_DTYPE_F16}


class KVCacheMXFP4:
    """A paged key/value cache in MXFP4 (uint8 tensors, contiguous, on one CUDA device; the four stay the same).

    k_codes, v_codes:   [pages][kv heads][page size][head_dim/2], two E2M1 codes per byte (element 2i low)
    k_scales, v_scales: [pages][kv heads][page size][head_dim/32], UE8M0
    """
    __slots__ = ("_parts", "_abi", "device", "num_kv_heads", "head_dim")

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor):
        pages, heads, page, half = shape = _shape(k_codes, 4, "k_codes")
        device, scales = k_codes.get_device(), (pages, heads, page, half // 16)
        parts = (k_codes, k_scales, v_codes, v_scales)
        for name, t, want in zip(("k_codes", "k_scales", "v_codes", "v_scales"), parts, (shape, scales, shape, scales)):
            if t.dtype is not torch.uint8 or device < 0 or t.get_device() != device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor on the cache's device")
            if t.shape != want:
                raise ValueError(f"{name} must have shape {tuple(want)}, not {tuple(t.shape)}")
        self._parts = parts
        self.device, self.num_kv_heads, self.head_dim = device, heads, 2 * half
        self._abi = abi.MoeKvCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                                   pages, page, heads, 2 * half)

    k_codes = property(lambda self: self._parts[0])
    k_scales = property(lambda self: self._parts[1])
    v_codes = property(lambda self: self._parts[2])
    v_scales = property(lambda self: self._parts[3])
    page_size = property(lambda self: self._parts[0].shape[2])

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda") -> "KVCacheMXFP4":
        def make(width):
            return torch.empty((num_pages, num_kv_heads, page_size, width), dtype=torch.uint8, device=device)
        return cls(make(head_dim // 2), make(head_dim // 32), make(head_dim // 2), make(head_dim // 32))

    def as_abi(self) -> abi.MoeKvCache:
        return self._abi


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


def _rows(t: torch.Tensor, name: str, device: int, dtype: torch.dtype) -> int:
    """Row stride of a [rows][heads][dim] tensor whose rows are contiguous, on the device and in the type of q."""
    rows, heads, dim = _shape(t, 3, name)
    if t.get_device() != device or t.dtype is not dtype:
        raise ValueError(f"{name} must have the device and type of q")
    step, head, one = t.stride()
    if (one != 1 or head != dim) and t.numel() and ((dim > 1 and one != 1) or (heads > 1 and head != dim)):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return step if rows > 1 else heads * dim


def _queries(q: torch.Tensor) -> tuple[int, torch.dtype, int]:
    """Device and type of q, which the other tensors share, and the type's code."""
    _shape(q, 3, "q")
    device, dtype = q.get_device(), q.dtype
    if device < 0 or dtype not in _DTYPES:
        raise ValueError("q must be a CUDA tensor in bf16 or fp16")
    return device, dtype, _DTYPES[dtype]


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, device: int) -> int:
    """Address of a contiguous vector."""
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on q's device")
    return t.data_ptr()


def _status(t: torch.Tensor | None, device: int) -> int | None:
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.get_device() != device or t.numel() < 1:
        raise ValueError("d_status must be an int32 tensor on q's device")
    return t.data_ptr()


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A tensor that belongs to the stream of the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(out: torch.Tensor | None, q: torch.Tensor, device: int, dtype: torch.dtype, stream) -> tuple[torch.Tensor, int]:
    """The output tensor and its row stride."""
    if out is None:
        return _empty(q.shape, dtype, q.device, stream), q.shape[1] * q.shape[2]
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    return out, _rows(out, "out", device, dtype)


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)  # current_stream() without its Stream object
    return abi.stream_ptr(stream)


def _on(device: int, name: str, fn, *args):
    """Calls an entry point with the device current, and checks its status."""
    if torch._C._cuda_getDevice() == device:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != abi.MOE_OK:
        abi.check(name, status)


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
    device, dtype, code = _queries(q)
    q_stride, k_stride, v_stride = (_rows(q, "q", device, dtype), _rows(k, "k", device, dtype),
                                    _rows(v, "v", device, dtype))
    T, H, D = q.shape
    K = k.shape[1]
    if k.shape != (T, K, D) or v.shape != (T, K, D):
        raise ValueError("k and v must be [T][kv heads][D] with the T and D of q")
    R = table_rows = 0
    rope_at = positions_at = slots_at = abi_cache = None
    if rope is not None:
        if rope.dim() != 2 or rope.dtype is not torch.float32 or rope.get_device() != device or \
                not rope.is_contiguous():
            raise ValueError("rope must be a contiguous fp32 [positions][rotary_dim] tensor on q's device")
        if positions is None:
            raise ValueError("rope needs positions")
        positions_at = _vector(positions, "positions", torch.int32, T, device)
        table_rows, R = rope.shape
        rope_at = rope.data_ptr()
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots go together")
    if cache is not None:
        if cache.device != device or cache.num_kv_heads != K or cache.head_dim != D:
            raise ValueError("the cache must be on q's device, with the kv heads and head size of k")
        slots_at = _vector(slots, "slots", torch.int64, T, device)
        abi_cache = cache.as_abi()
    if q_out is None:
        q_out = _empty((T, H, D), dtype, q.device, stream)
    elif q_out.shape != q.shape or q_out.dtype is not dtype or q_out.get_device() != device or \
            not q_out.is_contiguous():
        raise ValueError("q_out must be contiguous, with the shape, type and device of q")
    out = {"q": q_out}
    k_at = k_cached_at = v_cached_at = None
    if rotated_keys:
        out["k"] = _empty((T, K, D), dtype, q.device, stream)
        k_at = out["k"].data_ptr()
    if cached_values:
        out["k_cached"] = _empty((T, K, D), dtype, q.device, stream)
        out["v_cached"] = _empty((T, K, D), dtype, q.device, stream)
        k_cached_at, v_cached_at = out["k_cached"].data_ptr(), out["v_cached"].data_ptr()
    io = abi.MoeQkvAppendIO(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, T, H, K, D, code, R,
        int(interleaved), table_rows, rope_at, positions_at,
        None if q_norm is None else _vector(q_norm, "q_norm", dtype, D, device),
        None if k_norm is None else _vector(k_norm, "k_norm", dtype, D, device),
        eps, slots_at, q_out.data_ptr(), k_at, k_cached_at, v_cached_at)
    _on(device, "moe_qkv_append", abi.moe_qkv_append, io, abi_cache, _status(d_status, device),
        _raw_stream(stream, device))
    return out


@functools.lru_cache(maxsize=1024)
def _paged_workspace(device: int, rows: int, max_rows: int, heads: int, kv_heads: int, dim: int) -> int:
    """Bytes of workspace, which depend on these sizes alone."""
    io = abi.MoeAttendPagedIO(num_rows=rows, max_rows=max_rows, num_heads=heads)
    with torch.cuda.device(device):
        return abi.moe_attend_paged_workspace(
            io, abi.MoeKvCache(page_size=16, num_kv_heads=kv_heads, head_dim=dim))


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
    device, dtype, code = _queries(q)
    q_stride = _rows(q, "q", device, dtype)
    T, H, D = q.shape
    B = lengths.shape[0] if lengths.dim() == 1 else -1
    lengths_at = _vector(lengths, "lengths", torch.int32, B, device)
    cu_at = _vector(cu_rows, "cu_rows", torch.int32, B + 1, device)
    if page_table.dtype is not torch.int32 or page_table.get_device() != device or page_table.dim() != 2 or \
            page_table.shape[0] != B or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [sequences][pages] tensor on q's device")
    c = cache.as_abi()
    if cache.device != device or cache.head_dim != D:
        raise ValueError("the cache must be on q's device, with q's head size")
    out, out_stride = _out(out, q, device, dtype, stream)
    lse = _empty((T, H), torch.float32, q.device, stream) if return_lse else None
    io = abi.MoeAttendPagedIO(q.data_ptr(), q_stride, out.data_ptr(), out_stride,
                              lse.data_ptr() if return_lse else None, page_table.data_ptr(), lengths_at, cu_at, B, T,
                              page_table.shape[1], max_rows, H, code, D ** -0.5 if scale is None else scale)
    n = _paged_workspace(device, T, max_rows, H, cache.num_kv_heads, D)
    workspace = _empty((n,), torch.uint8, q.device, stream)
    _on(device, "moe_attend_paged", abi.moe_attend_paged, io, c, workspace.data_ptr(), n, _status(d_status, device),
        _raw_stream(stream, device))
    return (out, lse) if return_lse else out


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, cu_keys: torch.Tensor, *,
                  causal: bool = True, scale: float | None = None, out: torch.Tensor | None = None,
                  return_lse: bool = False, d_status: torch.Tensor | None = None, stream=None):
    """Attention over packed prompts, or over chunks of prompts with the keys before them.

    q [rows][heads][D], k and v [keys][kv heads][D]; cu_rows, cu_keys int32 [sequences + 1]. Row i of a sequence
    with n rows and m keys sees keys 0 .. m - n + i (causal), or all m. Rows that see no key give 0 and lse -inf.

    Returns out [rows][heads][D], and with return_lse also lse fp32 [rows][heads].
    """
    device, dtype, code = _queries(q)
    q_stride, k_stride, v_stride = (_rows(q, "q", device, dtype), _rows(k, "k", device, dtype),
                                    _rows(v, "v", device, dtype))
    T, H, D = q.shape
    N, K = k.shape[:2]
    if k.shape != (N, K, D) or v.shape != (N, K, D):
        raise ValueError("k and v must be [keys][kv heads][D] with the D of q")
    n = cu_rows.shape[0] if cu_rows.dim() == 1 else 0
    if n < 1:
        raise ValueError("cu_rows needs an entry for each sequence and one for the end")
    cu_rows_at = _vector(cu_rows, "cu_rows", torch.int32, n, device)
    cu_keys_at = _vector(cu_keys, "cu_keys", torch.int32, n, device)
    out, out_stride = _out(out, q, device, dtype, stream)
    lse = _empty((T, H), torch.float32, q.device, stream) if return_lse else None
    io = abi.MoeAttendPromptIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride,
                               out.data_ptr(), out_stride, lse.data_ptr() if return_lse else None, cu_rows_at,
                               cu_keys_at, n - 1, T, N, H, K, D, code, int(causal),
                               D ** -0.5 if scale is None else scale)
    _on(device, "moe_attend_prompt", abi.moe_attend_prompt, io, _status(d_status, device),
        _raw_stream(stream, device))
    return (out, lse) if return_lse else out
