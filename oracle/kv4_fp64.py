"""Plain definition of the paged 4-bit K/V cache in numpy: the element format
(in 64 bits, with the rounding steps it names), the block layout byte by
byte, one step of the page plan, and attention over cached values in fp64.
Test infrastructure only; shares no code with the CUDA path."""

from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def f16_toward_zero(x32: np.ndarray) -> np.ndarray:
    """float16 of non-negative float32 values, rounded towards zero."""
    h = x32.astype(np.float16)
    over = h.astype(np.float64) > x32.astype(np.float64)
    return np.where(over, np.nextafter(h, np.float16(0)), h)


def kv4_quantize(x):
    """(codes uint8, step float16, zero float16) of the last axis of x, values
    that float32 holds exactly.  A NaN in a vector: NaN step and zero, codes 0."""
    x = np.clip(np.asarray(x, np.float64), -65504.0, 65504.0)
    lo, hi = x.min(-1), x.max(-1)
    span = (hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15)
    step = np.maximum(f16_toward_zero(span), np.float16(2.0 ** -24))
    zero = lo.astype(np.float32).astype(np.float16)
    nan = np.isnan(lo)
    step, zero = np.where(nan, np.float16(np.nan), step), np.where(nan, np.float16(np.nan), zero)
    with np.errstate(invalid="ignore"):
        level = (x - zero.astype(np.float64)[..., None]) / step.astype(np.float64)[..., None]
    level = np.where(np.isnan(level), 0.0, level)
    return np.clip(np.rint(level), 0, 15).astype(np.uint8), step, zero


def kv4_values(codes, step, zero):
    """step * code + zero, one rounding to float32."""
    v = codes.astype(np.float64) * step.astype(np.float64)[..., None]
    return (v + zero.astype(np.float64)[..., None]).astype(np.float32)


def kv4_place(d: int, is_v: bool, i: int, e: int):
    """(byte, shift) in a block of the code of element e of its token i."""
    if not is_v:
        return i * (d // 2) + e // 2, 4 * (e % 2)
    h, t, s = i // 8, (i % 8) // 2, i % 2
    g, rest = e // (d // 8), e % (d // 8)
    w, b, n = rest // 4, (rest % 4) // 2, rest % 2
    at = (((h * 8 + g) * 4 + t) * (d // 32) + w) * 4 + s * 2 + b
    return 8 * d + 64 + at, 4 * n


def kv4_unpack(cache: np.ndarray, page: int, d: int):
    """(k codes, k params, v codes, v params) of a whole cache: codes uint8
    [num_pages, Hkv, page, d], params float16 [num_pages, Hkv, page, 2]."""
    P, Hkv = cache.shape[:2]
    out = []
    for is_v in (False, True):
        byte = np.zeros((BLOCK, d), np.int64)
        shift = np.zeros((BLOCK, d), np.uint8)
        for i in range(BLOCK):
            for e in range(d):
                byte[i, e], shift[i, e] = kv4_place(d, is_v, i, e)
        out.append(((cache[..., byte] >> shift) & 15).reshape(P, Hkv, page, d))
        off = 16 * d + 64 if is_v else 8 * d
        par = np.ascontiguousarray(cache[..., off:off + 64]).view(np.float16)
        out.append(par.reshape(P, Hkv, page, 2))
    return out


def kv4_plan(lens, add, table, pool, page: int, max_tokens: int):
    """One step of the page plan on Python lists (table: a list of lists):
    (lens, table, pool, cu, slots, shortage).  A page index outside the cache
    gives no slots."""
    R, W, num_pages = len(lens), len(table[0]) if table else 0, len(pool) - 1
    same = (list(lens), [list(r) for r in table], list(pool), [0] * (R + 1), [-1] * max_tokens)
    pages = lambda n: -(-n // page)  # noqa: E731
    room = W * page
    if any(n < 0 or n > room or a < -1 or n + max(a, 0) > room for n, a in zip(lens, add)):
        return (*same, -1)
    if sum(max(a, 0) for a in add) > max_tokens or not 0 <= pool[0] <= num_pages:
        return (*same, -1)
    stack = list(pool[1:1 + pool[0]])
    lens2, table2 = list(lens), [list(r) for r in table]
    for r in range(R):
        if add[r] < 0:
            for j in range(pages(lens[r])):
                stack.append(table2[r][j])
                table2[r][j] = -1
            lens2[r] = 0
    if len(stack) > num_pages:
        return (*same, -1)
    need = sum(pages(n + a) - pages(n) for n, a in zip(lens, add) if a >= 0)
    if need > len(stack):
        return (*same, need - len(stack))
    cu, slots = [0], []
    for r in range(R):
        if add[r] >= 0:
            for j in range(pages(lens[r]), pages(lens[r] + add[r])):
                table2[r][j] = stack.pop()
            for p in range(lens[r], lens[r] + add[r]):
                at = table2[r][p // page]
                slots.append(at * page + p % page if 0 <= at < num_pages else -1)
            lens2[r] += add[r]
        cu.append(len(slots))
    pool2 = [len(stack)] + stack + [-1] * (num_pages - len(stack))
    return lens2, table2, pool2, cu, slots + [-1] * (max_tokens - len(slots)), 0


def kv4_attention(q, k, v, n: int, causal: bool, scale: float):
    """q [n, Hq, d] over k, v [len, Hkv, d] (the cached values) in fp64: (out
    [n, Hq, d], lse [n, Hq], weights [n, Hq, len])."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    L, Hkv, d = k.shape
    Hq = q.shape[1]
    out = np.zeros((n, Hq, d))
    lse = np.full((n, Hq), -math.inf)
    w = np.zeros((n, Hq, L))
    for t in range(n):
        end = min(L, L - n + t + 1) if causal else L
        if end <= 0:
            continue
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s = scale * (k[:end, kv] @ q[t, h])
            m = s.max()
            z = m + math.log(np.exp(s - m).sum())
            w[t, h, :end] = np.exp(s - z)
            out[t, h] = w[t, h, :end] @ v[:end, kv]
            lse[t, h] = z
    return out, lse, w
