"""Torch-facing wrapper: checks tensors, allocates outputs with torch and
passes raw pointers plus a CUDA stream (the caller's ``stream``, else the
current one) to the C ABI.  All arithmetic happens in the library's kernels.

Outputs and temporaries that a call allocates are allocated while the stream
the kernels run on is current.  torch's caching allocator ties a block to the
stream that was current at allocation and reuses it only in that stream's
order.  A temporary freed when the call returns, such as the backward's
workspace, is therefore not handed to other work before the kernels that use
it have finished.
"""

from __future__ import annotations

import math
from contextlib import contextmanager

import torch

from . import _lib


def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


@contextmanager
def _on(device, stream):
    """Make ``device`` and the call's stream current; yields the stream
    handle for the C ABI."""
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream(device)
        with torch.cuda.stream(s):
            yield int(s.cuda_stream)


def _check_cuda(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def _check_out(t: torch.Tensor, name: str, dtype: torch.dtype, shape):
    """A caller-supplied output must match the shape the kernel writes: the
    library writes through raw pointers and cannot see a buffer's size."""
    _check_cuda(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_ring: int, causal: bool,
        scale: float | None = None, out: torch.Tensor | None = None,
        lse: torch.Tensor | None = None, stream=None):
    """Ring-ordered attention forward.  q [B, L, Hq, d], k/v [B, L, Hkv, d]
    (bf16, contiguous, on the GPU).  Returns (out bf16 [B, L, Hq, d],
    lse fp32 [B, Hq, L]).  ``scale`` defaults to 1/sqrt(d)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_cuda(t, n, torch.bfloat16, 4)
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape:
        raise ValueError(f"k/v shape {tuple(k.shape)}/{tuple(v.shape)} does not match q {tuple(q.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(q.device, stream) as sh:
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device)
        _check_out(out, "out", torch.bfloat16, (B, L, Hq, d))
        _check_out(lse, "lse", torch.float32, (B, Hq, L))
        _lib.ring_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), B, Hq, Hkv, L, d, n_ring, causal, scale, sh)
    return out, lse


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
        dout: torch.Tensor, lse: torch.Tensor, n_ring: int, causal: bool,
        scale: float | None = None, dq: torch.Tensor | None = None,
        dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
        workspace: torch.Tensor | None = None, stream=None):
    """Backward pass of ``fwd``: q/k/v/n_ring/causal/scale as given to it, its
    out (bf16 [B, L, Hq, d]) and lse (fp32 [B, Hq, L]), and dout (bf16, like
    out).  Returns (dq, dk, dv) in bf16.  ``workspace`` (any CUDA tensor of at
    least ``ring_attn_bwd_workspace_size`` bytes) is allocated if omitted."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check_cuda(t, n, torch.bfloat16, 4)
    _check_cuda(lse, "lse", torch.float32, 3)
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape:
        raise ValueError(f"k/v shape {tuple(k.shape)}/{tuple(v.shape)} does not match q {tuple(q.shape)}")
    if out.shape != q.shape or dout.shape != q.shape or lse.shape != (B, Hq, L):
        raise ValueError("out/dout/lse shapes do not match q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(q.device, stream) as sh:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        for t, n, ref in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
            _check_cuda(t, n, torch.bfloat16, 4)
            if t.shape != ref.shape:
                raise ValueError(f"{n} shape does not match")
        need = _lib.ring_attn_bwd_workspace_size(B, Hq, L)
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
        _lib.ring_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                           dv.data_ptr(), workspace.data_ptr(), ws_bytes, B, Hq, Hkv, L, d,
                           n_ring, causal, scale, sh)
    return dq, dk, dv


def bwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                dout: torch.Tensor, lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                dv: torch.Tensor, n_ring: int, causal: bool, scale: float | None = None,
                stream=None):
    """``bwd`` through ring_attn_bwd_noalloc: no workspace, results written
    into the given dq/dk/dv (bf16, shapes of q/k/v); B * Hq * L must not
    exceed 1,048,576."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"),
                 (dk, "dk"), (dv, "dv")):
        _check_cuda(t, n, torch.bfloat16, 4)
    _check_cuda(lse, "lse", torch.float32, 3)
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape or out.shape != q.shape or \
            dout.shape != q.shape or lse.shape != (B, Hq, L):
        raise ValueError("k/v/out/dout/lse shapes do not match q")
    for t, n, ref in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _check_out(t, n, torch.bfloat16, tuple(ref.shape))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(q.device, stream) as sh:
        _lib.ring_attn_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                   dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), B, Hq, Hkv, L, d, n_ring, causal, scale, sh)
    return dq, dk, dv


def bwd_visit(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
              dout: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, diag: int,
              parts: int, dq_acc: torch.Tensor | None = None, dk_acc: torch.Tensor | None = None,
              dv_acc: torch.Tensor | None = None, fold_q: bool = False, fold_kv: bool = False,
              scale: float | None = None, dq: torch.Tensor | None = None, stream=None):
    """One backward ring visit (ring_attn_bwd_visit): the host's query block
    q/out/dout [B, l, Hq, d] (bf16) with its final lse [B, Hq, l] against the
    K/V block k/v [B, l, Hkv, d]; parts 1 (dQ, writes D to workspace), 2
    (dK/dV, reads D) or 3.  Accumulators are fp32 of the shapes of q and k."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check_cuda(t, n, torch.bfloat16, 4)
    _check_cuda(lse, "lse", torch.float32, 3)
    B, l, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, l, Hkv, d) or v.shape != k.shape or out.shape != q.shape or \
            dout.shape != q.shape or lse.shape != (B, Hq, l):
        raise ValueError("block shapes do not match")
    for t, n, ref in ((dq_acc, "dq_acc", q), (dk_acc, "dk_acc", k), (dv_acc, "dv_acc", k)):
        if t is not None:
            _check_cuda(t, n, torch.float32, 4)
            if t.shape != ref.shape:
                raise ValueError(f"{n} shape does not match")
    if dq is not None:
        _check_cuda(dq, "dq", torch.bfloat16, 4)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    with _on(q.device, stream) as sh:
        _lib.ring_attn_bwd_visit(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 dout.data_ptr(), lse.data_ptr(), ptr(dq_acc), ptr(dk_acc),
                                 ptr(dv_acc), ptr(dq), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), B, Hq, Hkv, l, d,
                                 diag, parts, fold_q, fold_kv, scale, sh)


def round_bf16(src: torch.Tensor, dst: torch.Tensor | None = None, stream=None):
    """fp32 -> bf16 (nearest even) through ring_attn_round_bf16."""
    if not src.is_cuda or src.dtype != torch.float32 or not src.is_contiguous():
        raise TypeError("src must be a contiguous fp32 CUDA tensor")
    with _on(src.device, stream) as sh:
        if dst is None:
            dst = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device)
        _check_out(dst, "dst", torch.bfloat16, tuple(src.shape))
        _lib.ring_attn_round_bf16(src.data_ptr(), dst.data_ptr(), src.numel(), sh)
    return dst


def fwd_visit(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o_acc: torch.Tensor,
              lse_acc: torch.Tensor, diag: int, fold: bool, scale: float | None = None,
              out: torch.Tensor | None = None, stream=None):
    """One ring visit: the query block q [B, l, Hq, d] against the K/V block
    k/v [B, l, Hkv, d] (bf16), written to (fold=False) or folded into
    (fold=True) the running fp32 accumulator o_acc [B, l, Hq, d] and
    lse_acc [B, Hq, l].  ``diag``: 0 every key, 1 keys c <= r, 2 keys c < r
    (local rows).  ``out`` (bf16, optional) receives the rounded
    accumulator.  Returns (o_acc, lse_acc, out)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_cuda(t, n, torch.bfloat16, 4)
    B, l, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, l, Hkv, d) or v.shape != k.shape:
        raise ValueError(f"k/v shape {tuple(k.shape)}/{tuple(v.shape)} does not match q {tuple(q.shape)}")
    _check_cuda(o_acc, "o_acc", torch.float32, 4)
    _check_cuda(lse_acc, "lse_acc", torch.float32, 3)
    if o_acc.shape != q.shape or lse_acc.shape != (B, Hq, l):
        raise ValueError("o_acc/lse_acc shapes do not match q")
    if out is not None:
        _check_cuda(out, "out", torch.bfloat16, 4)
        if out.shape != q.shape:
            raise ValueError("out shape does not match q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(q.device, stream) as sh:
        _lib.ring_attn_fwd_visit(q.data_ptr(), k.data_ptr(), v.data_ptr(), o_acc.data_ptr(),
                                 lse_acc.data_ptr(), 0 if out is None else out.data_ptr(),
                                 B, Hq, Hkv, l, d, diag, fold, scale, sh)
    return o_acc, lse_acc, out


def quantize_fp8(x: torch.Tensor, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
    """Block quantisation of x bf16 [B, L, H, d] to E4M3: returns (codes
    uint8 [B, L, H, d], scales fp32 [B, H, ceil(L / 128)]), one scale per
    128-row tile of each (batch, head).  The codes are raw E4M3 bit patterns
    (``codes.view(torch.float8_e4m3fn)`` reads them as FP8)."""
    _check_cuda(x, "x", torch.bfloat16, 4)
    B, L, H, d = x.shape
    with _on(x.device, stream) as sh:
        if codes is None:
            codes = torch.empty((B, L, H, d), dtype=torch.uint8, device=x.device)
        if scales is None:
            scales = torch.empty((B, H, (L + 127) // 128), dtype=torch.float32, device=x.device)
        _check_out(codes, "codes", torch.uint8, (B, L, H, d))
        _check_out(scales, "scales", torch.float32, (B, H, (L + 127) // 128))
        _lib.ring_attn_quantize_fp8(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), B, L, H, d,
                                    sh)
    return codes, scales


def fwd_fp8(q8: torch.Tensor, sq: torch.Tensor, k8: torch.Tensor, sk: torch.Tensor,
            v8: torch.Tensor, sv: torch.Tensor, n_ring: int, causal: bool,
            scale: float | None = None, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, stream=None):
    """Ring-ordered attention forward on FP8 inputs from ``quantize_fp8``:
    q8 [B, L, Hq, 128] with sq [B, Hq, L/128], k8/v8 [B, L, Hkv, 128] with
    sk/sv [B, Hkv, L/128].  Returns (out bf16 [B, L, Hq, 128], lse fp32
    [B, Hq, L]).  ``scale`` defaults to 1/sqrt(d)."""
    for t, n in ((q8, "q8"), (k8, "k8"), (v8, "v8")):
        _check_cuda(t, n, torch.uint8, 4)
    for t, n in ((sq, "sq"), (sk, "sk"), (sv, "sv")):
        _check_cuda(t, n, torch.float32, 3)
    B, L, Hq, d = q8.shape
    Hkv = k8.shape[2]
    if k8.shape != (B, L, Hkv, d) or v8.shape != k8.shape:
        raise ValueError(f"k8/v8 shape {tuple(k8.shape)}/{tuple(v8.shape)} does not match "
                         f"q8 {tuple(q8.shape)}")
    if L % 128 != 0 or (n_ring > 0 and (L // n_ring) % 128 != 0):
        raise ValueError(f"the FP8 forward needs L / n_ring to be a multiple of 128 "
                         f"(L={L}, n_ring={n_ring})")
    T = L // 128
    if sq.shape != (B, Hq, T) or sk.shape != (B, Hkv, T) or sv.shape != (B, Hkv, T):
        raise ValueError("scale tensors must be [B, H, L/128]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(q8.device, stream) as sh:
        if out is None:
            out = torch.empty((B, L, Hq, d), dtype=torch.bfloat16, device=q8.device)
        if lse is None:
            lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q8.device)
        _check_out(out, "out", torch.bfloat16, (B, L, Hq, d))
        _check_out(lse, "lse", torch.float32, (B, Hq, L))
        _lib.ring_attn_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), sq.data_ptr(),
                               sk.data_ptr(), sv.data_ptr(), out.data_ptr(), lse.data_ptr(), B,
                               Hq, Hkv, L, d, n_ring, causal, scale, sh)
    return out, lse


def merge(o_a: torch.Tensor, lse_a: torch.Tensor, o_b: torch.Tensor, lse_b: torch.Tensor,
          out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None, stream=None):
    """Log-sum-exp merge of two partials: o [rows, d] fp32, lse [rows] fp32."""
    _check_cuda(o_a, "o_a", torch.float32, 2)
    _check_cuda(o_b, "o_b", torch.float32, 2)
    _check_cuda(lse_a, "lse_a", torch.float32, 1)
    _check_cuda(lse_b, "lse_b", torch.float32, 1)
    rows, d = o_a.shape
    if tuple(o_b.shape) != (rows, d) or tuple(lse_a.shape) != (rows,) or tuple(lse_b.shape) != (rows,):
        raise ValueError("o_a, o_b must be [rows, d] and lse_a, lse_b [rows]")
    with _on(o_a.device, stream) as sh:
        if out is None:
            out = torch.empty_like(o_a)
        if lse_out is None:
            lse_out = torch.empty_like(lse_a)
        _check_out(out, "out", torch.float32, (rows, d))
        _check_out(lse_out, "lse_out", torch.float32, (rows,))
        _lib.ring_attn_merge(o_a.data_ptr(), lse_a.data_ptr(), o_b.data_ptr(), lse_b.data_ptr(),
                             out.data_ptr(), lse_out.data_ptr(), rows, d, sh)
    return out, lse_out


# ---------------------------------------------------------------- 4-bit K/V cache
_CODE = {torch.bfloat16: _lib.RA_BF16, torch.float16: _lib.RA_FP16, torch.float32: _lib.RA_FP32}
_workspace_bytes = None


# The current stream's handle without building a torch.cuda.Stream, which
# costs more than the rest of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_bf16, _f16, _f32, _i32, _u8 = (torch.bfloat16, torch.float16, torch.float32, torch.int32,
                                torch.uint8)
_native = {}


def _fn(name: str):
    f = _native.get(name)
    if f is None:
        f = _native[name] = _lib.function(name)
    return f


def _is(t, dtype, ndim: int, index: int) -> bool:
    """Whether t is a contiguous tensor of that type and rank on CUDA device
    `index` (one expression: these calls are counted in microseconds)."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim
            and t.get_device() == index and t.is_contiguous())


def _check_same_device(device, **tensors):
    for n, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{n} is on {t.device}, expected {device}")


def _check_rows(t: torch.Tensor, name: str):
    """[T, H, d] whose tokens may be strided (a slice of a fused projection),
    each token's [H, d] contiguous.  Returns T, H, d and the token stride in
    elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not _bf16 and t.dtype is not _f16:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be a 3-d tensor [T, H, d]")
    T, H, d = t.shape
    if t.is_contiguous():
        return T, H, d, H * d
    st = t.stride()
    if T == 0:
        return T, H, d, H * d
    if (d > 1 and st[2] != 1) or (H > 1 and st[1] != d):
        raise ValueError(f"each token's [H, d] of {name} must be contiguous")
    if T == 1:
        return T, H, d, H * d
    if st[0] < H * d:
        raise ValueError(f"the tokens of {name} must not overlap (stride {st[0]})")
    return T, H, d, st[0]


def _cache_shape(cache: torch.Tensor):
    """(num_pages, Hkv, page, d) of a cache tensor."""
    if not (isinstance(cache, torch.Tensor) and cache.is_cuda and cache.dtype is _u8
            and cache.dim() == 4 and cache.is_contiguous()):
        _check_cuda(cache, "cache", _u8, 4)
    P, Hkv, blocks, nbytes = cache.shape
    if (nbytes != 2176 and nbytes != 1152) or blocks < 1 or Hkv < 1:
        raise ValueError(f"cache must be [num_pages, Hkv, page / 16, 16 * (d + 8)] with d 64 or "
                         f"128, got {tuple(cache.shape)}")
    return P, Hkv, 16 * blocks, 128 if nbytes == 2176 else 64


def kv4_cache(num_pages: int, Hkv: int, d: int, page: int = 64, device="cuda") -> torch.Tensor:
    """An empty paged 4-bit K/V cache: uint8 [num_pages, Hkv, page / 16,
    16 * (d + 8)], d 64 or 128, page a multiple of 16."""
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    if page < 16 or page > 4096 or page % 16 != 0:
        raise ValueError(f"page must be a multiple of 16 up to 4096, got {page}")
    if num_pages < 0 or Hkv < 1:
        raise ValueError("num_pages must be >= 0 and Hkv >= 1")
    return torch.zeros((num_pages, Hkv, page // 16, 16 * (d + 8)), dtype=torch.uint8, device=device)


def kv4_pool(num_pages: int, device="cuda") -> torch.Tensor:
    """The stack of free pages of a new cache, int32 [num_pages + 1]: its
    size, then the pages, of which 0 is taken first."""
    return torch.arange(num_pages, -1, -1, dtype=torch.int32, device=device)


def kv4_plan(lens: torch.Tensor, add: torch.Tensor, table: torch.Tensor, pool: torch.Tensor,
             page: int, max_tokens: int, out=None, stream=None):
    """Block tables and slot maps of one step of a batch, on the GPU.
    lens [R]: cached tokens of each request; add [R]: new ones, -1 ends the
    request; table [R, W]: its pages; pool [num_pages + 1]: the stack of free
    pages (``kv4_pool``); all int32.  Ended requests give their pages back,
    then the others take what they need in their order.

    Returns (lens, table, pool, cu [R + 1], slots [max_tokens], shortage [1]):
    the state after the step, the new tokens before each request, their slots
    (-1 behind the last) and 0, or how many pages are missing (-1: numbers
    that do not fit), in which case nothing changes.  A page index outside
    [0, num_pages) gives slots of -1 and is reported by ``check_status``.
    ``out``: tensors of these shapes for the results; the first three may be
    the inputs themselves."""
    if not (isinstance(table, torch.Tensor) and table.is_cuda and table.dtype is _i32
            and table.dim() == 2 and table.is_contiguous()):
        _check_cuda(table, "table", _i32, 2)
    index = table.get_device()
    if not (_is(lens, _i32, 1, index) and _is(add, _i32, 1, index) and _is(pool, _i32, 1, index)):
        for t, n in ((lens, "lens"), (add, "add"), (pool, "pool")):
            _check_cuda(t, n, _i32, 1)
        _check_same_device(table.device, lens=lens, add=add, pool=pool)
    R, W = table.shape
    if lens.shape[0] != R or add.shape[0] != R:
        raise ValueError(f"lens {tuple(lens.shape)}, add {tuple(add.shape)} and table "
                         f"{tuple(table.shape)} do not belong together")
    num_pages = pool.shape[0] - 1
    if num_pages < 0:
        raise ValueError("pool must be [num_pages + 1]")
    if max_tokens < 0:
        raise ValueError(f"max_tokens must be >= 0, got {max_tokens}")
    if stream is not None or _current_device() != index:
        with _on(table.device, stream) as sh:
            return _plan(lens, add, table, pool, page, max_tokens, out, index, R, W, num_pages, sh)
    return _plan(lens, add, table, pool, page, max_tokens, out, index, R, W, num_pages,
                 _raw_stream(index))


def _plan(lens, add, table, pool, page, max_tokens, out, index, R, W, num_pages, sh):
    if out is None:
        new, dev = torch.empty, table.device
        out = (new(R, dtype=_i32, device=dev), new((R, W), dtype=_i32, device=dev),
               new(num_pages + 1, dtype=_i32, device=dev), new(R + 1, dtype=_i32, device=dev),
               new(max_tokens, dtype=_i32, device=dev), new(1, dtype=_i32, device=dev))
    else:
        for t, n, shape in zip(out, ("lens", "table", "pool", "cu", "slots", "shortage"),
                               ((R,), (R, W), (num_pages + 1,), (R + 1,), (max_tokens,), (1,)),
                               strict=True):
            if not (_is(t, _i32, len(shape), index) and t.shape == shape):
                _check_out(t, "out " + n, _i32, shape)
                _check_same_device(table.device, **{"out_" + n: t})
    lo, to, po, cu, slots, shortage = out
    st = _fn("ring_attn_kv4_plan")(
        lens.data_ptr(), add.data_ptr(), table.data_ptr(), pool.data_ptr(), lo.data_ptr(),
        to.data_ptr(), po.data_ptr(), cu.data_ptr(), slots.data_ptr(), shortage.data_ptr(), R, W,
        num_pages, page, max_tokens, sh)
    if st:
        _lib._check(st)
    return lo, to, po, cu, slots, shortage


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
               stream=None):
    """Quantise k, v [T, Hkv, d] (bf16 or fp16; tokens may be strided) into
    the cache at ``slots`` (int32 [T], distinct; -1 skips a token)."""
    T, H, dk, ks = _check_rows(k, "k")
    Tv, Hv, dv, vs = _check_rows(v, "v")
    P, Hkv, page, d = _cache_shape(cache)
    if not (T == Tv and H == Hv == Hkv and dk == dv == d and k.dtype is v.dtype):
        raise ValueError(f"k {tuple(k.shape)} {k.dtype} and v {tuple(v.shape)} {v.dtype} must be "
                         f"[T, {Hkv}, {d}] of one type")
    index = cache.get_device()
    if not (_is(slots, _i32, 1, index) and slots.shape[0] == T and k.get_device() == index
            and v.get_device() == index):
        _check_out(slots, "slots", _i32, (T,))
        _check_same_device(cache.device, k=k, v=v, slots=slots)
    if stream is not None or _current_device() != index:
        with _on(cache.device, stream) as sh:
            _append(k, ks, v, vs, slots, cache, T, Hkv, d, P, page, sh)
    else:
        _append(k, ks, v, vs, slots, cache, T, Hkv, d, P, page, _raw_stream(index))
    return cache


def _append(k, ks, v, vs, slots, cache, T, Hkv, d, P, page, sh):
    st = _fn("ring_attn_kv4_append")(k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(),
                                     cache.data_ptr(), T, Hkv, d, _CODE[k.dtype], P, page, sh)
    if st:
        _lib._check(st)


def kv4_read(cache: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """The cached keys and values at ``slots`` (int32 [T]; zeros for -1):
    (k, v) of ``dtype`` (bf16, fp16 or fp32), [T, Hkv, d]."""
    P, Hkv, page, d = _cache_shape(cache)
    index = cache.get_device()
    if not _is(slots, _i32, 1, index):
        _check_cuda(slots, "slots", _i32, 1)
        _check_same_device(cache.device, slots=slots)
    if dtype not in _CODE:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    if stream is not None or _current_device() != index:
        with _on(cache.device, stream) as sh:
            return _read(cache, slots, dtype, k, v, index, P, Hkv, page, d, sh)
    return _read(cache, slots, dtype, k, v, index, P, Hkv, page, d, _raw_stream(index))


def _read(cache, slots, dtype, k, v, index, P, Hkv, page, d, sh):
    T, dev = slots.shape[0], cache.device
    shape = (T, Hkv, d)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
    elif not (_is(k, dtype, 3, index) and k.shape == shape):
        _check_out(k, "k", dtype, shape)
        _check_same_device(dev, k=k)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=dev)
    elif not (_is(v, dtype, 3, index) and v.shape == shape):
        _check_out(v, "v", dtype, shape)
        _check_same_device(dev, v=v)
    st = _fn("ring_attn_kv4_read")(cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   T, Hkv, d, _CODE[dtype], P, page, sh)
    if st:
        _lib._check(st)
    return k, v


def kv4_workspace(device="cuda") -> torch.Tensor:
    """A workspace for ``kv4_fwd``, its counters zeroed as they have to be.
    One serves any number of calls that run one after the other."""
    global _workspace_bytes
    if _workspace_bytes is None:
        _workspace_bytes = _lib.ring_attn_kv4_workspace_size()
    w = torch.empty(_workspace_bytes, dtype=torch.uint8, device=device)
    w[:_lib.KV4_COUNTER_BYTES].zero_()
    return w


def kv4_fwd(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
            cu: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
            max_q: int | None = None, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
            workspace: torch.Tensor | None = None, stream=None):
    """Attention of new query tokens over the cached tokens of R requests.
    q [T, Hq, d] (bf16 or fp16; tokens may be strided); table int32 [R, W],
    lens int32 [R] and cu int32 [R + 1] as ``kv4_plan`` gives them: request
    r's query tokens are the rows cu[r] .. cu[r + 1] (without cu: one a
    request), its keys the first lens[r] cached tokens; causal: the query
    tokens are the last of these.  Returns (out [T, Hq, d] of q's type or
    ``out_dtype`` float32, lse fp32 [T, Hq]); rows from cu[R] on are not
    written.  ``max_q`` bounds the query tokens of a request (default T) and
    chooses the kernels: 1 while decoding.  ``out`` carries fp16 roundings of
    the weights (2^-11 at most) even as float32; ``lse`` does not.
    ``workspace`` (``kv4_workspace``) is made for the call if omitted."""
    T, Hq, dq, qs = _check_rows(q, "q")
    P, Hkv, page, d = _cache_shape(cache)
    if dq != d or Hq % Hkv != 0 or Hq < 1:
        raise ValueError(f"q {tuple(q.shape)} does not match a cache of {Hkv} heads of {d}")
    index = q.get_device()
    if not (_is(table, _i32, 2, index) and _is(lens, _i32, 1, index)
            and cache.get_device() == index):
        _check_cuda(table, "table", _i32, 2)
        _check_cuda(lens, "lens", _i32, 1)
        _check_same_device(q.device, cache=cache, table=table, lens=lens)
    R, W = table.shape
    if lens.shape[0] != R:
        raise ValueError(f"lens {tuple(lens.shape)} does not match table {tuple(table.shape)}")
    if cu is not None:
        if not (_is(cu, _i32, 1, index) and cu.shape[0] == R + 1):
            _check_out(cu, "cu", _i32, (R + 1,))
            _check_same_device(q.device, cu=cu)
    elif T != R:
        raise ValueError(f"without cu every request has one query token, got {T} for {R} requests")
    if out_dtype is None:
        out_dtype = q.dtype if out is None else out.dtype
    if out_dtype is not q.dtype and out_dtype is not _f32:
        raise TypeError(f"the output is {q.dtype} or float32, got {out_dtype}")
    shape = (P, Hkv, page, d, T, Hq, qs, R, W, T if max_q is None else max_q, causal,
             1.0 / math.sqrt(d) if scale is None else scale)
    if stream is not None or _current_device() != index:
        with _on(q.device, stream) as sh:
            return _cache_fwd(q, cache, table, lens, cu, out, lse, out_dtype, workspace, index,
                              shape, sh)
    return _cache_fwd(q, cache, table, lens, cu, out, lse, out_dtype, workspace, index, shape,
                      _raw_stream(index))


def _cache_fwd(q, cache, table, lens, cu, out, lse, out_dtype, workspace, index, shape, sh):
    P, Hkv, page, d, T, Hq, qs, R, W, max_q, causal, scale = shape
    dev = q.device
    if out is None:
        out = torch.empty((T, Hq, d), dtype=out_dtype, device=dev)
    elif not (_is(out, out_dtype, 3, index) and out.shape == (T, Hq, d)):
        _check_out(out, "out", out_dtype, (T, Hq, d))
        _check_same_device(dev, out=out)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=_f32, device=dev)
    elif not (_is(lse, _f32, 2, index) and lse.shape == (T, Hq)):
        _check_out(lse, "lse", _f32, (T, Hq))
        _check_same_device(dev, lse=lse)
    if workspace is None:
        workspace = kv4_workspace(dev)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    st = _fn("ring_attn_kv4_fwd")(
        q.data_ptr(), qs, cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
        0 if cu is None else cu.data_ptr(), out.data_ptr(), lse.data_ptr(), T, R, Hq, Hkv, d, W, P,
        page, max_q, bool(causal), scale, _CODE[q.dtype], _CODE[out_dtype], workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), sh)
    if st:
        _lib._check(st)
    return out, lse


def check_status(stream=None):
    with torch.cuda.device(torch.cuda.current_device()):
        _lib.ring_attn_check_status(_stream_handle(stream))


class _RingAttention(torch.autograd.Function):
    """Autograd bridge: forward through ring_attn_fwd (saving out and lse),
    backward through ring_attn_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, n_ring, causal, scale):
        out, lse = fwd(q, k, v, n_ring, causal, scale)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.n_ring, ctx.causal, ctx.scale = n_ring, causal, scale
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = bwd(q, k, v, out, dout.contiguous().to(torch.bfloat16), lse, ctx.n_ring,
                         ctx.causal, ctx.scale)
        return dq, dk, dv, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_ring: int, causal: bool,
              scale: float | None = None) -> torch.Tensor:
    """Differentiable ring-ordered attention on one GPU: the output of
    ``fwd``, with gradients for q, k and v from ``bwd``."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _RingAttention.apply(q, k, v, n_ring, causal, scale)
