"""Pins of the 4-bit cache oracle: the nearest level by exhaustive search,
the layout by writing and finding every place, the page plan by its
invariants and a worked example, attention against the dense oracle."""

from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import oracle
from oracle import kv4_fp64 as kv4


def _cases(d, n, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)).astype(np.float32)
    x[0] = 0.25                      # a constant vector
    x[1] = 0.0
    x[2, 0], x[2, 1] = 60000.0, -60000.0
    x[3] *= 2.0 ** -20               # steps among fp16's subnormals
    x[4] = np.arange(d) % 31 / 2.0   # every second value half way between two levels
    x[4, :2] = 0.0, 15.0
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("d", [64, 128])
def test_codes_are_the_nearest_levels(d):
    x = _cases(d, 40, 1)
    codes, step, zero = kv4.kv4_quantize(x)
    s, z = step.astype(np.float64), zero.astype(np.float64)
    levels = s[:, None] * np.arange(16) + z[:, None]
    far = np.abs(x[:, :, None] - levels[:, None, :])
    best = far.min(-1)
    got = np.take_along_axis(far, codes[..., None].astype(np.int64), -1)[..., 0]
    assert np.array_equal(got, best)
    ties = (far == best[..., None]).sum(-1) > 1
    assert ties.any() and (codes[ties] % 2 == 0).all()
    # the step is the largest fp16 not above the span / 15, and the floor holds
    span = ((x.max(-1) - x.min(-1)) / 15)
    assert (s[span >= 2.0 ** -24] <= span[span >= 2.0 ** -24] * (1 + 2.0 ** -23)).all()
    assert (s >= 2.0 ** -24).all() and s[0] == 2.0 ** -24
    v = kv4.kv4_values(codes, step, zero)
    assert np.array_equal(v[0], x[0]) and np.array_equal(v[1], x[1])
    assert np.isfinite(v.astype(np.float16)).all()
    # off by half a step at most (the top level may lie up to 15 ulp of the step low)
    assert (np.abs(v - x) <= s[:, None] * (0.5 + 15 * 2.0 ** -10) + 2.0 ** -25 * 16).all()


def test_a_fifteenth_by_a_product_and_one_correction():
    """q = x F, q + F (x - 15 q) with F = fl(1 / 15), fused (Markstein): the
    correctly rounded x / 15 for every float32 significand.  The binade does not matter: the
    steps are exact to powers of two, and where the quotient is below 2^-24, as any
    of a subnormal's would be, the step is 2^-24 whatever its last place."""
    F = np.float32(1) / np.float32(15)
    x = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(0x3F800000)).view(np.float32)
    q = x * F
    r = x.astype(np.float64) - 15.0 * q.astype(np.float64)   # 28 bits: exact
    assert np.array_equal(r.astype(np.float32).astype(np.float64), r)
    s = q.astype(np.float64) + r * np.float64(F)             # the product has 48 bits: exact
    # rounded to 64 bits first: no matter unless half way between two of 32 bits
    assert not ((s.view(np.uint64) & np.uint64((1 << 29) - 1)) == np.uint64(1 << 28)).any()
    assert np.array_equal(s.astype(np.float32), x / np.float32(15))


def test_nan_and_infinities():
    x = np.ones((3, 64))
    x[0, 5] = math.nan
    x[1, 7] = math.inf
    codes, step, zero = kv4.kv4_quantize(x)
    assert np.isnan(kv4.kv4_values(codes, step, zero)[0]).all()
    assert kv4.kv4_values(codes, step, zero)[1, 7] <= 65504 and codes[1, 7] == 15
    assert (kv4.kv4_values(codes, step, zero)[2] == 1).all()


@pytest.mark.parametrize("d", [64, 128])
def test_every_place_is_its_own(d):
    seen = set()
    for is_v in (False, True):
        lo = 8 * d + 64 if is_v else 0
        for i in range(16):
            for e in range(d):
                byte, shift = kv4.kv4_place(d, is_v, i, e)
                assert lo <= byte < lo + 8 * d and shift in (0, 4)
                seen.add((byte, shift))
    assert len(seen) == 2 * 16 * d
    # no byte is shared by two tokens
    owner = {}
    for i in range(16):
        for e in range(d):
            for is_v in (False, True):
                assert owner.setdefault(kv4.kv4_place(d, is_v, i, e)[0], i) == i


def test_plan_worked_example():
    # page 4; request 0 fills its page, 1 ends, 2 starts with 5 tokens
    lens, add = [3, 6, 0], [2, -1, 5]
    table = [[7, -1], [2, 5], [-1, -1]]
    pool = [3, 0, 1, 9, -1, -1, -1, -1, -1, -1, -1]
    got = kv4.kv4_plan(lens, add, table, pool, 4, 8)
    # pages 2, 5 come back on top of [0, 1, 9]; request 0 takes 5, request 2 takes 2 and 9
    assert got[0] == [5, 0, 5]
    assert got[1] == [[7, 5], [-1, -1], [2, 9]]
    assert got[2] == [2, 0, 1] + [-1] * 8
    assert got[3] == [0, 2, 2, 7]
    assert got[4] == [7 * 4 + 3, 5 * 4, 8, 9, 10, 11, 36, -1]
    assert got[5] == 0


def test_plan_keeps_every_page_once():
    r = random.Random(5)
    R, W, page, P = 6, 5, 16, 20
    lens, table, pool = [0] * R, [[-1] * W for _ in range(R)], [P] + list(range(P))
    for _ in range(200):
        add = [r.choice([-1, 0, 1, 1, 17]) for _ in range(R)]
        new = kv4.kv4_plan(lens, add, table, pool, page, 256)
        if new[5] != 0:
            assert new[:3] == (lens, table, pool) and set(new[4]) <= {-1}
            add = [-1] * R
            new = kv4.kv4_plan(lens, add, table, pool, page, 256)
        lens, table, pool = new[:3]
        used = [table[i][j] for i in range(R) for j in range(-(-lens[i] // page))]
        assert sorted(used + pool[1:1 + pool[0]]) == list(range(P))
        live = [s for s in new[4] if s >= 0]
        assert len(set(live)) == len(live) == new[3][-1]


def test_plan_gives_no_slots_of_pages_outside_the_cache():
    got = kv4.kv4_plan([3, 3], [2, 1], [[-1, -1], [3, -1]], [1, 5, -1, -1, -1], 4, 4)
    assert got[0] == [5, 4] and got[1] == [[-1, 5], [3, -1]]
    assert got[4] == [-1, -1, 15, -1] and got[5] == 0


def test_attention_is_the_dense_oracle():
    rng = np.random.default_rng(2)
    L, Hq, Hkv, d = 37, 4, 2, 64
    q, k, v = (rng.standard_normal((L, h, d)) for h in (Hq, Hkv, Hkv))
    o, lse, w = kv4.kv4_attention(q, k, v, L, True, 0.2)
    ref, ref_lse = oracle.attention(q[None], k[None], v[None], True, 0.2)
    assert np.allclose(o, ref[0], atol=1e-12)
    assert np.allclose(lse.T, ref_lse[0], atol=1e-12)
    # a single token is the last row; tokens beyond the cached ones see nothing
    o1, _, _ = kv4.kv4_attention(q[-1:], k, v, 1, True, 0.2)
    assert np.allclose(o1[0], o[-1])
    o2, l2, _ = kv4.kv4_attention(q[:5], k[:3], v[:3], 5, True, 0.2)
    assert (o2[:2] == 0).all() and np.isinf(l2[:2]).all() and np.isfinite(l2[2:]).all()
