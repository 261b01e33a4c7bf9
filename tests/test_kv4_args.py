"""CPU-side checks of the 4-bit cache entry points: every refusal comes
before any CUDA call, and empty calls launch nothing."""

from __future__ import annotations

import os

import pytest
import torch

from ring_attention_ordered_b200 import _lib, api

INV, UNS = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
# fake, never-dereferenced device addresses, far apart
M = 1 << 32
A = [M * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from ring_attention_ordered_b200 import build
        build.build()
    return _lib.load()


def plan(lib, **kw):
    a = dict(lens=A[0], add=A[1], table=A[2], pool=A[3], lens_out=A[4], table_out=A[5],
             pool_out=A[6], cu=A[7], slots=A[8], shortage=A[9], R=4, W=8, num_pages=100, page=64,
             max_tokens=50)
    a.update(kw)
    return lib.ring_attn_kv4_plan(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INV), (dict(num_pages=-1), INV), (dict(max_tokens=-1), INV),
    (dict(R=8193), UNS), (dict(W=0), INV), (dict(R=8192, W=1 << 18), INV),
    (dict(page=0), INV), (dict(page=4097), INV), (dict(W=1 << 25, page=64), INV),
    (dict(num_pages=1 << 25), INV), (dict(max_tokens=1 << 31), INV),
    (dict(lens=0), INV), (dict(shortage=0), INV), (dict(cu=A[7] + 2), INV),
    (dict(lens_out=A[0] + 4), INV),          # overlaps lens without being it
    (dict(table_out=A[3]), INV),             # is the pool
    (dict(slots=A[2] + 16), INV),
    (dict(cu=A[1]), INV),
    (dict(shortage=A[8] + 4), INV),
])
def test_plan_refuses(lib, kw, status):
    assert plan(lib, **kw) == status
    assert _lib.last_error()


def append(lib, **kw):
    a = dict(k=A[0], ks=256, v=A[1], vs=256, slots=A[2], cache=A[3], T=10, Hkv=2, d=128, dtype=0,
             num_pages=100, page=64)
    a.update(kw)
    return lib.ring_attn_kv4_append(*a.values(), None)


CACHE = [(dict(Hkv=0), INV), (dict(d=96), UNS), (dict(d=256), UNS), (dict(num_pages=-1), INV),
         (dict(page=8), INV), (dict(page=40), INV), (dict(page=8192), INV),
         (dict(num_pages=1 << 25), INV), (dict(T=-1), INV), (dict(T=1 << 31), INV)]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(dtype=2), UNS), (dict(dtype=7), UNS), (dict(ks=248), INV), (dict(vs=260), INV),
    (dict(k=0), INV), (dict(slots=0), INV), (dict(k=A[0] + 8), INV), (dict(cache=A[3] + 4), INV),
    (dict(slots=A[2] + 1), INV), (dict(cache=A[0] + 64), INV), (dict(cache=A[2] + 16), INV),
])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status
    assert _lib.last_error()


def read(lib, **kw):
    a = dict(cache=A[0], slots=A[1], k=A[2], v=A[3], T=10, Hkv=2, d=128, dtype=0, num_pages=100,
             page=64)
    a.update(kw)
    return lib.ring_attn_kv4_read(*a.values(), None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(dtype=3), UNS), (dict(v=0), INV), (dict(v=A[2] + 16), INV), (dict(k=A[0]), INV),
    (dict(k=A[1]), INV), (dict(v=A[3] + 8), INV),
])
def test_read_refuses(lib, kw, status):
    assert read(lib, **kw) == status
    assert _lib.last_error()


def fwd(lib, **kw):
    a = dict(q=A[0], qs=512, cache=A[1], table=A[2], lens=A[3], cu=A[4], out=A[5], lse=A[6], T=10,
             R=3, Hq=4, Hkv=2, d=128, W=8, num_pages=100, page=64, max_q=5, causal=1, scale=0.1,
             dtype=0, out_dtype=0, ws=A[7], wsb=1 << 30)
    a.update(kw)
    return lib.ring_attn_kv4_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(R=-1), INV), (dict(Hq=0), INV), (dict(Hq=3), INV), (dict(W=0), INV),
    (dict(W=1 << 25), INV), (dict(max_q=-1), INV), (dict(causal=2), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(scale=-1.0), INV),
    (dict(dtype=2, out_dtype=2), UNS), (dict(out_dtype=1), UNS), (dict(qs=504), INV),
    (dict(qs=516), INV), (dict(cu=0), INV), (dict(q=0), INV), (dict(lens=0), INV),
    (dict(ws=0), INV), (dict(wsb=100), INV), (dict(q=A[0] + 2), INV), (dict(lse=A[6] + 2), INV),
    (dict(ws=A[7] + 4), INV), (dict(out=A[0]), INV), (dict(lse=A[5] + 16), INV),
    (dict(ws=A[1]), INV), (dict(ws=A[5] + 64), INV), (dict(lse=A[3]), INV),
    (dict(T=1 << 30, Hq=8), INV), (dict(T=1 << 23, R=1 << 23, max_q=1), UNS),
])
def test_fwd_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status
    assert _lib.last_error()


def test_empty_calls_launch_nothing(lib):
    assert append(lib, T=0, k=0, v=0, slots=0, cache=0) == _lib.RA_OK
    assert read(lib, T=0, k=0, v=0, slots=0, cache=0) == _lib.RA_OK
    assert fwd(lib, T=0, q=0, out=0, lse=0, ws=0, wsb=0) == _lib.RA_OK
    assert fwd(lib, T=0, R=0, cu=0, q=0, out=0, lse=0, ws=0, wsb=0) == _lib.RA_OK


def test_a_cache_of_no_pages_needs_no_memory(lib):
    """Its pointer is NULL (an empty tensor's is): such calls are not refused for
    it, those to a cache that has pages are."""
    for call in (append, read, fwd):
        assert call(lib, cache=0) == INV
        assert call(lib, cache=0, num_pages=0) != INV, _lib.last_error()


def test_workspace_size(lib):
    assert _lib.ring_attn_kv4_workspace_size() > 0
    assert lib.ring_attn_kv4_workspace_size(None) == INV


def test_wrapper_refuses_host_tensors_and_shapes():
    i32 = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = api.kv4_cache(3, 2, 64, page=32, device="cpu")
    assert cache.shape == (3, 2, 2, 16 * 72) and cache.dtype == torch.uint8
    assert api.kv4_pool(3, device="cpu").tolist() == [3, 2, 1, 0]
    assert api.kv4_pool(0, device="cpu").tolist() == [0]
    for call in (lambda: api.kv4_append(x, x, i32, cache), lambda: api.kv4_read(cache, i32),
                 lambda: api.kv4_fwd(x, cache, i32.view(4, 1), i32),
                 lambda: api.kv4_plan(i32, i32, i32.view(4, 1), i32, 16, 4)):
        with pytest.raises(TypeError):
            call()
    for kw in (dict(d=80), dict(d=64, page=24), dict(d=64, page=0), dict(d=64, num_pages=-1),
               dict(d=64, Hkv=0)):
        with pytest.raises(ValueError):
            api.kv4_cache(**{**dict(num_pages=1, Hkv=1, device="cpu"), **kw})
