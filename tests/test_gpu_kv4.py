"""GPU tests of the paged 4-bit K/V cache against its fp64 oracle: the page
plan and the codes exactly, the values after their one rounding, attention
within a tolerance derived from the kernel's arithmetic."""

from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

from oracle import kv4_fp64 as kv4

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ring_attention_ordered_b200 import _lib, api
    _lib.load()
    return api


@pytest.fixture(autouse=True)
def clean(ra):
    yield
    ra.check_status()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan
def random_plan(r, R, W, page, spare, most_add):
    """A state in which every page is in one place, and what is to be added."""
    room = W * page
    lens = [r.choice([0, 1, page, r.randint(0, room)]) for _ in range(R)]
    lens = [min(n, room) for n in lens]
    held = [-(-n // page) for n in lens]
    P = sum(held) + spare
    ids = list(range(P))
    r.shuffle(ids)
    table = [[ids.pop() for _ in range(h)] + [-1] * (W - h) for h in held]
    add = [r.choice([-1, 0, 1, r.randint(0, most_add)]) for _ in range(R)]
    add = [min(a, room - n) for a, n in zip(add, lens)]
    pool = [len(ids)] + ids + [-1] * (P - len(ids))
    return lens, add, table, pool


def check_plan(ra, lens, add, table, pool, page, max_tokens, in_place):
    want = kv4.kv4_plan(lens, add, table, pool, page, max_tokens)
    W = len(table[0]) if table else 3
    args = [i32(lens), i32(add), i32(table).view(len(lens), W), i32(pool)]
    out = None
    if in_place:
        out = (args[0], args[2], args[3], i32([7] * (len(lens) + 1)), i32([7] * max_tokens), i32([7]))
    kept = [a.clone() for a in args]
    got = ra.kv4_plan(*args, page, max_tokens, out=out)
    for g, w, name in zip(got, want, ("lens", "table", "pool", "cu", "slots", "shortage")):
        w = np.asarray([w] if name == "shortage" else w, np.int32).reshape(tuple(g.shape))
        assert np.array_equal(g.cpu().numpy(), w), name
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(args, kept))
    return want[5]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,W,page,spare,most_add,cap", [
    (1, 1, 16, 4, 16, 40), (7, 5, 16, 40, 60, 500), (32, 9, 64, 300, 3, 100),
    (513, 7, 48, 3600, 200, 70000), (1200, 4, 1, 4800, 3, 4000), (8192, 3, 32, 20000, 2, 20000),
    (40, 400, 16, 16000, 6000, 250001),
])
def test_plan(ra, R, W, page, spare, most_add, cap, in_place):
    r = random.Random(R * W)
    for _ in range(3):
        state = random_plan(r, R, W, page, spare, most_add)
        assert check_plan(ra, *state, page, cap, in_place) == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_that_cannot_be_met_changes_nothing(ra, in_place):
    r = random.Random(3)
    lens, add, table, pool = random_plan(r, 9, 6, 16, 0, 5)
    lens, add = [20] * 9, [16 * 4] * 9
    table = [[i, 9 + i] + [-1] * 4 for i in range(9)]
    pool = [2, 18, 19] + [-1] * 18
    assert check_plan(ra, lens, add, table, pool, 16, 9 * 64, in_place) == 9 * 4 - 2
    ok = [1] * 9
    for bad in (dict(lens=[20] * 8 + [-1]), dict(lens=[20] * 8 + [97]), dict(add=[1] * 8 + [-2]),
                dict(add=[1] * 8 + [77]), dict(add=[1] * 8 + [2 ** 31 - 1]),
                dict(pool=[22] + pool[1:]), dict(pool=[-1] + pool[1:])):
        a = dict(lens=lens, add=ok, table=table, pool=pool, page=16, max_tokens=200)
        a.update(bad)
        assert check_plan(ra, **a, in_place=in_place) == -1
    assert check_plan(ra, lens, ok, table, pool, 16, 8, in_place) == -1   # nine tokens
    assert check_plan(ra, lens, [0] * 9, table, pool, 16, 0, in_place) == 0


def test_plan_partly_in_place(ra):
    """Each of the three states by itself in the input's place."""
    r = random.Random(12)
    lens, add, table, pool = random_plan(r, 70, 6, 16, 300, 30)
    want = kv4.kv4_plan(lens, add, table, pool, 16, 2500)
    for place in (0, 1, 2):
        args = [i32(lens), i32(add), i32(table), i32(pool)]
        out = [torch.empty_like(args[0]), torch.empty_like(args[2]), torch.empty_like(args[3]),
               i32([0] * 71), i32([0] * 2500), i32([0])]
        out[place] = args[(0, 2, 3)[place]]
        got = ra.kv4_plan(*args, 16, 2500, out=out)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    with pytest.raises(Exception):
        ra.kv4_plan(*args, 16, 2500, out=[args[1]] + out[1:])   # overlaps `add`


def test_plan_of_no_request(ra):
    got = ra.kv4_plan(i32([]), i32([]), torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                      ra.kv4_pool(5), 16, 4)
    assert got[2].tolist() == [5, 4, 3, 2, 1, 0] and got[3].tolist() == [0]
    assert got[4].tolist() == [-1] * 4 and got[5].item() == 0


def test_plans_of_several_threads(ra):
    """Large and smaller plans launched by threads at the same time, through the C
    entry, which does not hold the interpreter: none takes another's room for its
    sums."""
    import threading

    from ring_attention_ordered_b200 import _lib
    plan = _lib.function("ring_attn_kv4_plan")
    kept, bad = [], []

    def arguments(R):
        lens, add, pool = i32([0] * R), i32([0] * R), ra.kv4_pool(1)
        table = torch.full((R, 1), -1, dtype=torch.int32, device="cuda")
        t = [lens, add, table, pool, lens, table, pool, i32([9] * (R + 1)), i32([0]), i32([9])]
        s = torch.cuda.Stream()
        kept.append((t, s))
        return [x.data_ptr() for x in t] + [R, 1, 1, 16, 0, s.cuda_stream]

    def run(args, go):
        go.wait()
        bad.extend(st for st in (plan(*args) for _ in range(6000)) if st)

    calls = [arguments(R) for R in (8192, 2600, 8191)]
    torch.cuda.synchronize()
    go = threading.Barrier(len(calls))
    threads = [threading.Thread(target=run, args=(a, go)) for a in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[0])
    for t, _ in kept:
        assert t[9].item() == 0 and not bool(t[7].any()) and t[3].tolist() == [1, 0]


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_reports_pages_outside_the_cache(ra, in_place):
    """Indices whose product with the page size is -16 + 15 = -1 (no slot), or
    wraps to a slot of page 0, or lies just behind the cache: no slots, one
    report, and the other requests' slots as ever.  One in a table that goes on
    (its request's last page has room), one released, one taken."""
    from ring_attention_ordered_b200 import _lib
    own = [7, 6]
    for bad in (-1, 1 << 28, (1 << 28) + 1, 8, -(1 << 28)):
        for lens, add, table, pool in (
                ([15, 17], [1, 2], [[bad, -1], own], [0] + [-1] * 8),
                ([20, 17], [-1, 15], [[5, bad], own], [1, 4] + [-1] * 7),
                ([0, 17], [20, 1], [[-1, -1], own], [2, bad, 3] + [-1] * 6)):
            check_plan(ra, lens, add, table, pool, 16, 24, in_place)
            with pytest.raises(_lib.RingAttnError) as e:
                ra.check_status()
            assert e.value.status == _lib.RA_ERR_INVALID_ARG
    # a table's entries behind a request's pages are not read
    check_plan(ra, [16, 17], [0, 1], [[5, 99], own], [0] + [-1] * 8, 16, 4, in_place)
    ra.check_status()


# ------------------------------------------------------------------ append, read
def vectors(T, Hkv, d, dtype, seed):
    """k and v with the vectors on which a quantiser can go wrong."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, T, Hkv, d, generator=g)
    if T >= 12:
        x[0, 0] = 0.0
        x[1, 0] = -1.75
        x[0, 1] *= 2.0 ** -22
        x[1, 2] = torch.arange(d) % 31 / 2.0
        x[1, 2, :, :2] = torch.tensor([0.0, 15.0])
        x[0, 3, :, 3] = math.nan
        x[1, 4, :, 5] = math.inf
        x[0, 4, :, 5] = -math.inf
        x[0, 5] = 1000.0 + 0.25 * torch.randn(Hkv, d, generator=g)
        x[1, 6] *= 20000
        x[1, 7] = torch.where(torch.arange(d) % 2 == 0, 0.0, 2.0 ** -24)
        x[0, 8] *= 2.0 ** -130
    return x[0].to(dtype), x[1].to(dtype)


def oracle_values(x):
    return kv4.kv4_quantize(x.double().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,Hkv,d,page", [(1, 1, 64, 16), (33, 3, 128, 48), (300, 2, 64, 64),
                                          (257, 8, 128, 16), (1, 5, 128, 128)])
def test_append_codes_and_read(ra, T, Hkv, d, page, dtype):
    k, v = vectors(T, Hkv, d, dtype, T + d)
    P = -(-T // page) + 2
    r = random.Random(T)
    slots = r.sample(range(P * page), T)
    if T > 20:
        slots[17] = -1
    cache = torch.randint(0, 256, (P, Hkv, page // 16, 16 * (d + 8)), dtype=torch.uint8,
                          device="cuda")
    before = kv4.kv4_unpack(cache.cpu().numpy(), page, d)
    ra.kv4_append(k.cuda(), v.cuda(), i32(slots), cache)
    after = kv4.kv4_unpack(cache.cpu().numpy(), page, d)
    used = [(i, s) for i, s in enumerate(slots) if s >= 0]
    idx = np.array([i for i, _ in used])
    pg, off = np.array([s // page for _, s in used]), np.array([s % page for _, s in used])
    want = {}
    for n, (x, name) in enumerate(((k, "k"), (v, "v"))):
        codes, step, zero = oracle_values(x)
        want[name] = (codes, step, zero)
        assert np.array_equal(after[2 * n][pg, :, off], codes[idx])
        par = after[2 * n + 1][pg, :, off]
        assert np.array_equal(par[..., 0], step[idx], equal_nan=True)
        assert np.array_equal(par[..., 1], zero[idx], equal_nan=True)
        # every other place is as it was
        keep = np.ones((P, page), bool)
        keep[pg, off] = False
        for a, b in ((before[2 * n], after[2 * n]),
                     (before[2 * n + 1].view(np.uint16), after[2 * n + 1].view(np.uint16))):
            assert np.array_equal(a.transpose(0, 2, 1, 3)[keep], b.transpose(0, 2, 1, 3)[keep])
    # read back, some slots twice, none where -1
    ask = slots + slots[:3] + [-1]
    for out in (torch.bfloat16, torch.float16, torch.float32):
        got = ra.kv4_read(cache, i32(ask), out)
        for y, name in zip(got, ("k", "v")):
            val = kv4.kv4_values(*want[name])
            ref = torch.zeros(len(ask), Hkv, d)
            for row, s in enumerate(ask):
                if s >= 0:
                    ref[row] = torch.from_numpy(val[slots.index(s)])
            ref = ref.to(out).cuda()
            assert torch.equal(torch.isnan(y), torch.isnan(ref))
            assert torch.equal(y.nan_to_num(0), ref.nan_to_num(0)), name


def test_append_of_every_border(ra):
    """Values on, just below and just above every border of the levels, for
    many steps and zeros: bf16 and fp16 neighbours of zero + (n + 1/2) step."""
    r = np.random.default_rng(0)
    d = 128
    for dtype in (torch.bfloat16, torch.float16):
        lo = torch.from_numpy(r.standard_normal(4000).astype(np.float32)).to(dtype)
        span = torch.from_numpy(np.exp2(r.uniform(-9, 5, 4000)).astype(np.float32)).to(dtype)
        hi = (lo.float() + span.float()).to(dtype)
        _, step, zero = kv4.kv4_quantize(torch.stack([lo, hi], -1).double().numpy())
        n = np.arange(15) + 0.5
        mid = step.astype(np.float64)[:, None] * n + zero.astype(np.float64)[:, None]
        mid = torch.from_numpy(mid).to(dtype)
        bits = mid.view(torch.int16)
        x = torch.cat([lo[:, None], hi[:, None], mid, (bits + 1).view(dtype),
                       (bits - 1).view(dtype)], -1)
        x = torch.minimum(torch.maximum(x, lo[:, None]), hi[:, None])
        x = torch.cat([x, lo[:, None].expand(-1, d - x.shape[1])], -1).view(1000, 4, d)
        cache = ra.kv4_cache(63, 4, d, page=16)
        ra.kv4_append(x.cuda(), x.cuda(), i32(list(range(1000))), cache)
        got = kv4.kv4_unpack(cache.cpu().numpy(), 16, d)
        codes, _, _ = kv4.kv4_quantize(x.double().numpy())
        for c in (got[0], got[2]):
            c = c.transpose(0, 2, 1, 3).reshape(-1, 4, d)[:1000]
            assert np.array_equal(c, codes)


def test_append_takes_strided_tokens(ra):
    T, Hq, Hkv, d = 50, 4, 2, 64
    qkv = torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    slots = i32(list(range(T)))
    a, b = ra.kv4_cache(4, Hkv, d, 16), ra.kv4_cache(4, Hkv, d, 16)
    ra.kv4_append(k, v, slots, a)
    ra.kv4_append(k.contiguous(), v.contiguous(), slots, b)
    assert torch.equal(a, b)
    table, lens, cu = i32([[0, 1, 2, 3]]), i32([T]), i32([0, T])
    o1, l1 = ra.kv4_fwd(q, a, table, lens, cu)
    o2, l2 = ra.kv4_fwd(q.contiguous(), a, table, lens, cu)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    with pytest.raises(ValueError):
        ra.kv4_append(k.transpose(0, 1), v, slots, a)
    with pytest.raises(ValueError):
        ra.kv4_append(k[:1].expand(T, Hkv, d), v, slots, a)


def test_slots_out_of_range_are_left_out_and_reported(ra):
    from ring_attention_ordered_b200 import _lib
    k, v = vectors(4, 2, 64, torch.bfloat16, 1)
    cache = ra.kv4_cache(3, 2, 64, 16)
    ra.kv4_append(k.cuda(), v.cuda(), i32([0, 48, -2, 2 ** 31 - 1]), cache)
    with pytest.raises(_lib.RingAttnError) as e:
        ra.check_status()
    assert e.value.status == _lib.RA_ERR_INVALID_ARG
    one = ra.kv4_cache(3, 2, 64, 16)
    ra.kv4_append(k[:1].cuda(), v[:1].cuda(), i32([0]), one)
    assert torch.equal(cache, one)
    x, y = ra.kv4_read(cache, i32([48, -7, 0]))
    assert (x[:2] == 0).all() and (y[:2] == 0).all() and (y[2] != 0).any()
    with pytest.raises(_lib.RingAttnError):
        ra.check_status()
    ra.check_status()


# ------------------------------------------------------------------ attention
class Batch:
    """Requests with cached tokens in shuffled pages, and what the oracle
    needs of them: the values that the cache holds."""

    def __init__(self, ra, lens, n, Hq, Hkv, d, page, dtype, seed, k_scale=1.0, spoil=True):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        self.lens, self.n, self.page, self.dtype = lens, n, page, dtype
        pages = [-(-L // page) for L in lens]
        ids = list(range(sum(pages) + 2))
        r.shuffle(ids)
        W = max(pages + [1]) + 1
        self.cache = ra.kv4_cache(len(ids), Hkv, d, page)
        if spoil:   # what no token has written: NaN and infinite parameters
            self.cache.fill_(0xFF)
        table = torch.full((len(lens), W), -1, dtype=torch.int32)
        self.kv = []
        for i, L in enumerate(lens):
            own = [ids.pop() for _ in range(pages[i])]
            table[i, :pages[i]] = torch.tensor(own, dtype=torch.int32)
            k, v = (torch.randn(2, L, Hkv, d, generator=g)).to(dtype)
            k = (k.float() * k_scale).to(dtype)
            if L:
                slots = [own[c // page] * page + c % page for c in range(L)]
                ra.kv4_append(k.cuda(), v.cuda(), i32(slots), self.cache)
            self.kv.append(tuple(oracle_values(x) for x in (k, v)))
        self.table, self.len_t = table.cuda(), i32(lens)
        self.cu = i32([0] + list(np.cumsum(n)))
        self.q = torch.randn(sum(n), Hq, d, generator=g).to(dtype)

    def check(self, out, lse, causal, scale, out_dtype=None):
        """|out - ref| against the half step of the output type plus:
        * the rounding of p * step to fp16, half a step 2^-11 of each term
          w step code, or 2^-25 where it is below fp16's normal range, when
          the reference's key has 2^8 at least: w (15 step) 2^-11 +
          15 max(step) 2^-33 a key;
        * fp32 scores: each of the d + 2 products and sums of a score is off
          by 2^-23 of sum |q| (15 step + |zero|) at most, twice that with the
          exponential's own 2^-22: ds; w ds |v|;
        * the sums over L keys in fp32, in partial sums: 2^-18 w |v|.
        Requests of more than 128 rows (query tokens times the group's heads)
        go to the chunk kernel, which rounds v and p to fp16 instead of
        p * step: half a step of each, 2 * 2^-11 w |v|, or 2^-25 of p below
        fp16's normal range, where the row's largest has 2^5 at least:
        max |v| 2^-30 a key."""
        at = 0
        half = HALF_STEP[out_dtype or self.dtype]
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        worst = 0.0
        for i, L in enumerate(self.lens):
            m = self.n[i]
            (kc, ks, kz), (vc, vs, vz) = self.kv[i]
            k, v = kv4.kv4_values(kc, ks, kz), kv4.kv4_values(vc, vs, vz)
            q = self.q[at:at + m].double().numpy()
            ref, ref_lse, w = kv4.kv4_attention(q, k, v, m, causal, scale)
            Hq, Hkv, d = q.shape[1], k.shape[1], k.shape[2]
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                got = out[at:at + m, h]
                big = 15 * vs[:, kv].astype(np.float64)
                if L == 0:
                    assert (got == 0).all() and np.isneginf(lse[at:at + m, h]).all()
                    continue
                size = np.abs(q[:, h]).sum(-1)[:, None] * (
                    15 * ks[:, kv].astype(np.float64) + np.abs(kz[:, kv].astype(np.float64)))[None]
                ds = 2 * (d + 2) * 2.0 ** -23 * scale * size + 2.0 ** -21
                ds = np.where(w[:, h] > 0, ds, 0)
                av = np.abs(v[:, kv].astype(np.float64))
                if m * (Hq // Hkv) > 128:
                    tol = 2 * 2.0 ** -11 * (w[:, h] @ av) + L * av.max() * 2.0 ** -30
                else:
                    tol = (w[:, h] * big[None]).sum(-1)[:, None] * 2.0 ** -11
                    tol = tol + L * big.max() * 2.0 ** -33
                tol = tol + (w[:, h] * (ds + 2.0 ** -18)) @ av
                tol = tol * (1 + 2 * half) + half * np.abs(ref[:, h]) + 1e-30
                err = np.abs(got - ref[:, h])
                assert (err <= tol).all(), (i, h, float((err / tol).max(initial=0.0)))
                worst = max(worst, float((err / tol).max(initial=0.0)))
                rl, gl = ref_lse[:, h], lse[at:at + m, h]
                none = np.isneginf(rl)
                assert np.array_equal(none, np.isneginf(gl)) and (got[none] == 0).all()
                lt = ds.max(-1) + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl)
                assert (np.abs(gl[~none] - rl[~none]) <= lt[~none]).all()
            at += m
        return worst


def attend(ra, b, causal=True, scale=None, **kw):
    scale = scale if scale is not None else 1 / math.sqrt(b.q.shape[-1])
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, causal=causal,
                          scale=scale, max_q=max(b.n), **kw)
    ra.check_status()
    b.check(out, lse, causal, scale, kw.get("out_dtype"))
    return out, lse


SHAPES = [
    # lens, query tokens, Hq, Hkv, d, page
    ([1], [1], 1, 1, 64, 16),
    ([509], [1], 8, 2, 128, 64),
    ([0, 1, 15, 16, 17, 128, 129, 700], [1] * 8, 8, 2, 128, 16),
    ([300, 0, 77, 64], [1] * 4, 3, 3, 64, 32),
    ([5000, 3, 1200], [1] * 3, 5, 1, 128, 64),
    ([900, 65], [1, 1], 32, 2, 64, 48),                 # groups of 16
    ([1000, 257, 40], [4, 1, 8], 8, 1, 64, 16),         # drafts
    ([130, 3, 0, 513], [9, 5, 2, 16], 4, 2, 128, 128),  # more query tokens than cached ones
    ([200, 333], [200, 70], 4, 2, 128, 64),             # prompts
    ([391, 1, 129], [131, 1, 129], 3, 1, 64, 16),
    ([3000], [700], 4, 1, 128, 64),
    ([257, 1500], [257, 300], 2, 2, 64, 16),
    ([40, 2100, 0, 300, 128], [300, 64, 5, 1, 128], 8, 2, 128, 32),
    ([129], [17], 1, 1, 128, 16),
    ([5000], [3], 8, 1, 64, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(ra, shape, causal, dtype):
    lens, n, Hq, Hkv, d, page = SHAPES[shape]
    attend(ra, Batch(ra, lens, n, Hq, Hkv, d, page, dtype, shape), causal)


def test_attention_without_row_starts_and_in_fp32(ra):
    b = Batch(ra, [70, 0, 300], [1, 1, 1], 4, 2, 64, 16, torch.float16, 3)
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    b.check(out, lse, True, 0.125, torch.float32)
    ref, rl = attend(ra, b, out_dtype=torch.float32)
    assert torch.equal(out, ref) and torch.equal(lse, rl)


@pytest.mark.parametrize("scale,k_scale", [(0.0, 1.0), (1.0, 6.0), (0.125, 40.0)])
def test_attention_flat_and_peaked(ra, scale, k_scale):
    attend(ra, Batch(ra, [600, 33], [3, 1], 4, 2, 64, 16, torch.bfloat16, 11, k_scale), scale=scale)


def test_attention_values_of_very_different_size(ra):
    """A dominant key with tiny values among others with large ones, constant
    value vectors (the smallest step), zeros: the reference follows score and
    step together."""
    b = Batch(ra, [256], [1], 2, 1, 64, 16, torch.bfloat16, 5)
    g = torch.Generator().manual_seed(9)
    k = torch.randn(256, 1, 64, generator=g)
    v = torch.randn(256, 1, 64, generator=g)
    v[::3] *= 1e-6
    v[1::7] = 0.5
    v[5::11] *= 500
    v[40] = 0.0
    k[40] = b.q[0, 0].float() * 2
    k[96] = b.q[0, 1].float() * 2
    v[96] *= 1e-7
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    own = b.table[0].tolist()
    slots = [own[c // 16] * 16 + c % 16 for c in range(256)]
    ra.kv4_append(k.cuda(), v.cuda(), i32(slots), b.cache)
    b.kv = [(oracle_values(k), oracle_values(v))]
    attend(ra, b, scale=0.3)


def test_attention_of_large_and_small_queries(ra):
    b = Batch(ra, [100, 100], [2, 2], 2, 1, 64, 16, torch.bfloat16, 6)
    b.q[0] *= 2.0 ** 40
    b.q[1] = 0
    b.q[2] *= 2.0 ** -60
    b.q[3, 0, 5] = 3e4
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, scale=0.125)
    # row 0's weights sit on one key: compare where scores are of ordinary size
    b2 = Batch(ra, [100, 100], [2, 2], 2, 1, 64, 16, torch.bfloat16, 6)
    b2.q = b.q.clone()
    b2.q[0] = 0
    o2, l2 = attend(ra, b2)
    assert torch.equal(out[1:], o2[1:]) and torch.equal(lse[1:], l2[1:])
    ref, _, w = kv4.kv4_attention(b.q[:2].double().numpy(), kv4.kv4_values(*b.kv[0][0]),
                                  kv4.kv4_values(*b.kv[0][1]), 2, True, 0.125)
    assert (w[0].max(-1) == 1).all()
    err = np.abs(out[0].double().cpu().numpy() - ref[0])
    assert (err <= 2.0 ** -7 * np.abs(ref[0]) + 2.0 ** -9 * np.abs(kv4.kv4_values(*b.kv[0][1])).max()).all()


def test_nan_reaches_only_the_rows_that_see_it_in_a_chunk(ra):
    b = Batch(ra, [300, 40], [200, 30], 2, 1, 128, 16, torch.bfloat16, 7)
    want = attend(ra, b)
    k, v = vectors(1, 1, 128, torch.bfloat16, 3)
    own = b.table[0].tolist()
    slot = i32([own[177 // 16] * 16 + 177 % 16])
    old = ra.kv4_read(b.cache, slot)
    v[0, 0, 3] = math.nan
    ra.kv4_append(old[0], v.cuda(), slot, b.cache)
    # query token t of request 0 sees 101 + t tokens: token 177 from t = 77 on
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, max_q=200)
    assert torch.equal(out[:77], want[0][:77]) and torch.equal(out[200:], want[0][200:])
    assert torch.isnan(out[77:200]).all() and torch.equal(lse, want[1])
    k[0, 0, 0] = math.nan
    ra.kv4_append(k.cuda(), old[1], slot, b.cache)
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, max_q=200)
    assert torch.equal(out[:77], want[0][:77]) and torch.equal(lse[200:], want[1][200:])
    assert torch.isnan(out[77:200]).all() and torch.isnan(lse[77:200]).all()


def test_nan_reaches_only_the_rows_that_see_it(ra):
    b = Batch(ra, [40, 40], [8, 1], 2, 1, 64, 16, torch.bfloat16, 7)
    k, v = vectors(1, 1, 64, torch.bfloat16, 3)
    v[0, 0, 3] = math.nan
    own = b.table[0].tolist()
    ra.kv4_append(k.cuda(), v.cuda(), i32([own[36 // 16] * 16 + 36 % 16]), b.cache)
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu)
    # query token t of request 0 sees 33 + t tokens: token 36 from t = 4 on
    assert not torch.isnan(out[:4]).any() and torch.isnan(out[4:8]).all()
    assert not torch.isnan(out[8]).any() and not torch.isnan(lse).any()
    k[0, 0, 0] = math.nan
    ra.kv4_append(k.cuda(), v.cuda(), i32([own[36 // 16] * 16 + 36 % 16]), b.cache)
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu)
    assert not torch.isnan(out[:4]).any() and torch.isnan(lse[4:8]).all()


def test_rows_behind_the_last_request_are_left(ra):
    b = Batch(ra, [50, 0, 90], [1, 2, 3], 4, 2, 64, 16, torch.bfloat16, 8)
    q = torch.cat([b.q, torch.full((5, 4, 64), math.nan, dtype=torch.bfloat16)]).cuda()
    out = torch.full((11, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((11, 4), 7.0, device="cuda")
    ra.kv4_fwd(q, b.cache, b.table, b.len_t, cu=b.cu, out=out, lse=lse)
    b.check(out[:6], lse[:6], True, 0.125)
    assert (out[6:] == 7).all() and (lse[6:] == 7).all()


@pytest.mark.parametrize("n", [1, 5, 40])
def test_any_split_gives_the_result(ra, n):
    """The same batch on 1, 2, 7 and all CTAs: every result within the
    tolerance, runs of the same split bit for bit alike, the workspace ready
    for the next call."""
    from ring_attention_ordered_b200 import _lib
    b = Batch(ra, [4001, 17, 0, 2500], [n] * 4, 4, 2, 128, 64, torch.bfloat16, 21)
    ws = ra.kv4_workspace()
    try:
        for ctas in (1, 2, 7, 0):
            _lib.ring_attn_set_max_ctas(ctas)
            first = attend(ra, b, workspace=ws)
            for _ in range(3):
                again = attend(ra, b, workspace=ws)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    finally:
        _lib.ring_attn_set_max_ctas(0)


@pytest.mark.parametrize("n", [1, 4, 80])
@pytest.mark.parametrize("d", [64, 128])
def test_the_counters_are_left_zero(ra, n, d):
    """All of the workspace's first KV4_COUNTER_BYTES, by calls whose units cross CTAs,
    the first CTA among them."""
    from ring_attention_ordered_b200 import _lib
    ws = ra.kv4_workspace()
    for lens in ([9000], [9000, 70, 20000]):
        b = Batch(ra, lens, [n] * len(lens), 8, 2, d, 64, torch.bfloat16, 72)
        attend(ra, b, workspace=ws)
        assert not bool(ws[:_lib.KV4_COUNTER_BYTES].any())


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("ctas", [1, 2, 5])
def test_many_short_units_a_cta(ra, ctas, d, dtype):
    """Prompts and chunks whose units, with and without a second row tile, far outnumber
    the places of a CTA's queue; among them single tokens and an empty request."""
    from ring_attention_ordered_b200 import _lib
    n = [70, 33, 1, 129, 40, 257, 64, 0, 65, 35, 100, 160]
    lens = [a + b for a, b in zip(n, [0, 0, 50, 0, 300, 0, 129, 0, 1, 700, 0, 30])]
    b = Batch(ra, lens, n, 8, 2, d, 16, dtype, 71)
    ws = ra.kv4_workspace()
    try:
        _lib.ring_attn_set_max_ctas(ctas)
        first = attend(ra, b, workspace=ws)
        for _ in range(3):
            again = attend(ra, b, workspace=ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert not bool(ws[:_lib.KV4_COUNTER_BYTES].any())
    finally:
        _lib.ring_attn_set_max_ctas(0)


def test_one_long_request(ra):
    """100001 tokens: a stretch of the request on every CTA."""
    b = Batch(ra, [100001], [1], 2, 1, 128, 128, torch.bfloat16, 22)
    attend(ra, b)


def test_pages_out_of_range_are_left_out_and_reported(ra):
    from ring_attention_ordered_b200 import _lib
    b = Batch(ra, [100, 60, 200], [1, 1, 1], 4, 2, 64, 16, torch.bfloat16, 23)
    want = attend(ra, b)
    table = b.table.clone()
    table[1, 1], table[1, 2] = 10 ** 6, -5
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, table, b.len_t, cu=b.cu)
    with pytest.raises(_lib.RingAttnError) as e:
        ra.check_status()
    assert e.value.status == _lib.RA_ERR_INVALID_ARG
    for row in (0, 2):
        assert torch.equal(out[row], want[0][row]) and torch.equal(lse[row], want[1][row])
    # the tokens of the two pages are left out
    (kc, ks, kz), (vc, vs, vz) = b.kv[1]
    keep = [c for c in range(60) if c // 16 not in (1, 2)]
    ref, rl, _ = kv4.kv4_attention(b.q[1:2].double().numpy(), kv4.kv4_values(kc, ks, kz)[keep],
                                   kv4.kv4_values(vc, vs, vz)[keep], 1, False, 0.125)
    assert np.allclose(lse[1].cpu().numpy(), rl[0], atol=1e-4)
    assert np.allclose(out[1].double().cpu().numpy(), ref[0], atol=2e-2)
    # lengths and row starts are cut down to the tensors
    lens, cu = i32([10 ** 9, 60, -3]), i32([0, 1, 2, 99])
    ra.kv4_fwd(b.q.cuda(), b.cache, b.table.clamp(min=0), lens, cu=cu)
    with pytest.raises(_lib.RingAttnError):
        ra.check_status()


@pytest.mark.parametrize("R,n", [(3, 2), (40, 3), (3, 200), (40, 60)])
def test_row_starts_that_fall_are_refused(ra, R, n):
    """Up to 32 requests and more, each kernel: no row is written, the error is
    reported, and the next call with the workspace is right."""
    from ring_attention_ordered_b200 import _lib
    b = Batch(ra, [500 + n] * R, [n] * R, 8, 2, 64, 32, torch.bfloat16, 62)
    ws = ra.kv4_workspace()
    cu = b.cu.clone()
    cu[1::2] = b.q.shape[0]
    out = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
    ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=cu, max_q=n, out=out, lse=lse,
               workspace=ws)
    with pytest.raises(_lib.RingAttnError) as e:
        ra.check_status()
    assert e.value.status == _lib.RA_ERR_INVALID_ARG
    assert bool((out == 7).all()) and bool((lse == 7).all())
    assert not bool(ws[:_lib.KV4_COUNTER_BYTES].any())
    attend(ra, b)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_a_single_request_of_many_rows_without_tokens(ra, d, out_dtype):
    """One request of 70 x 2 rows: the chunk kernel alone serves it, and writes its
    empty rows and reports its numbers itself.  Rows of no request are left."""
    from ring_attention_ordered_b200 import _lib
    n, T = 70, 75
    b = Batch(ra, [160], [n], 4, 2, d, 16, torch.bfloat16, 70)
    q = torch.cat([b.q, torch.full((T - n, 4, d), math.nan, dtype=torch.bfloat16)]).cuda()
    table = b.table[:, :10].contiguous()   # room for 160 tokens
    ws = ra.kv4_workspace()

    def call(length, starts, causal=True, reported=False):
        out = torch.full((T, 4, d), 7.0, dtype=out_dtype, device="cuda")
        lse = torch.full((T, 4), 7.0, device="cuda")
        ra.kv4_fwd(q, b.cache, table, i32([length]), cu=i32(starts), causal=causal, out=out,
                   lse=lse, workspace=ws)
        if reported:
            with pytest.raises(_lib.RingAttnError) as e:
                ra.check_status()
            assert e.value.status == _lib.RA_ERR_INVALID_ARG
        else:
            ra.check_status()
        assert not bool(ws[:_lib.KV4_COUNTER_BYTES].any())
        return out, lse

    def empty(got, first, last):
        out, lse = got
        assert bool((out[first:last] == 0).all()) and bool(torch.isneginf(lse[first:last]).all())
        for x in got:
            assert bool((x[:first] == 7).all()) and bool((x[last:] == 7).all())

    empty(call(0, [0, n]), 0, n)
    empty(call(0, [0, n], causal=False), 0, n)
    empty(call(0, [2, n]), 2, n)
    empty(call(-3, [0, n], reported=True), 0, n)
    empty(call(0, [3, 200], reported=True), 3, T)
    empty(call(0, [-4, n], reported=True), 0, n)
    empty(call(160, [n, 3], reported=True), 0, 0)     # the starts fall: nothing is done
    empty(call(0, [n, 3], reported=True), 0, 0)
    want = call(160, [0, n])
    b.check(want[0][:n], want[1][:n], True, 1 / math.sqrt(d), out_dtype)
    cut = call(10 ** 9, [0, n], reported=True)        # cut down to the table's room
    assert torch.equal(cut[0], want[0]) and torch.equal(cut[1], want[1])
    assert bool((want[0][n:] == 7).all()) and bool((want[1][n:] == 7).all())


@pytest.mark.parametrize("R", [31, 32, 33, 63, 64, 65])
def test_batches_around_the_ways_to_divide_them(ra, R):
    """Empty requests, short ones and a long one, in and out of step with the
    requests a lane takes."""
    lens = [(0, 40, 1, 700, 16, 17)[(r * 5 + R) % 6] for r in range(R)]
    lens[R // 2], lens[-1] = 9001, 33
    attend(ra, Batch(ra, lens, [1 + r % 3 for r in range(R)], 4, 2, 64, 32, torch.bfloat16, 63 + R))


@pytest.mark.parametrize("d", [64, 128])
def test_lse_of_short_requests(ra, d):
    """q . code and zero sum(q) cancel in a score.  Neither, nor a partial sum, is
    above sum|q| (15 step + |zero|) scale; d / 16 instructions and four fp32
    operations each cut off 2^-23 of that at most.  exp, its sum and log add
    2^-20."""
    b = Batch(ra, [1, 2, 3, 5, 2, 1, 4, 7], [1] * 8, 8, 2, d, 16, torch.float16, 64)
    scale = 1 / math.sqrt(d)
    _, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, scale=scale)
    ra.check_status()
    for r in range(8):
        (kc, ks, kz), (vc, vs, vz) = b.kv[r]
        _, ref, _ = kv4.kv4_attention(b.q[r:r + 1].double().numpy(), kv4.kv4_values(kc, ks, kz),
                                      kv4.kv4_values(vc, vs, vz), 1, False, scale)
        got = lse[r].double().cpu().numpy()
        q = b.q[r].double().abs().sum(-1).numpy()
        most = q * scale * (15 * float(np.max(ks)) + float(np.max(np.abs(kz))))
        assert (np.abs(got - ref[0]) <= most * (d / 16 + 4) * 2.0 ** -23 + 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 70])
def test_lse_of_rows_that_see_few_tokens_is_as_of_32_bits(ra, n, d, dtype):
    """Single tokens after 1 to 7 others (the decoding kernel), and the first rows of
    prompts, which see 1 to 8 tokens (the chunk kernel).  The root mean square of the
    error of lse against what 32 bits give: a score is the sum of A = scale ks (q . code)
    and B = scale kz sum(q), in d / 16 sums and four other operations, each off by half
    a place, 2^-24 of the larger of |A| and |B|, at most and one independent of the
    others: 2^-24 max(|A|, |B|) sqrt(d / 16 + 4); exp2 is off by 2^-22 at most, half
    of it taken as its root mean square, and lse is rounded once more.  K codes that
    enter a quarter as large, which loses places as the products are aligned, give 9e-7
    to 1.2e-6 for fp16, where this is 4.9e-7 to 6.7e-7."""
    if n == 1:
        lens, see = [1 + r % 7 for r in range(96)], 1
    else:
        lens, see = [n] * 8, 8
    b = Batch(ra, lens, [n] * len(lens), 8, 2, d, 16, dtype, 90 + d)
    scale = 1 / math.sqrt(d)
    _, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, scale=scale, max_q=n)
    ra.check_status()
    lse = lse.double().cpu().numpy()
    err, most = [], []
    for r, L in enumerate(lens):
        (kc, ks, kz), v = b.kv[r]
        q = b.q[r * n:r * n + see].double().numpy()
        end = L if n == 1 else see
        k, vv = kv4.kv4_values(kc, ks, kz)[:end], kv4.kv4_values(*v)[:end]
        _, ref, w = kv4.kv4_attention(q, k, vv, see, True, scale)
        err.append(lse[r * n:r * n + see] - ref)
        head = np.arange(8) // 4
        A = scale * np.einsum("the,che->thc", q, kc[:end, head].astype(np.float64))
        A = A * ks[:end, head].T.astype(np.float64)
        B = scale * q.sum(-1)[..., None] * kz[:end, head].T.astype(np.float64)
        size = np.maximum(np.abs(A), np.abs(B))
        most.append((w * size ** 2).sum(-1) * 2.0 ** -48 * (d / 16 + 4) + 2.0 ** -46
                    + (2.0 ** -25 * ref) ** 2)
    err, most = (np.sqrt(np.mean(np.square(x))) for x in
                 (np.concatenate(err), np.sqrt(np.concatenate(most))))
    print(f"lse rms error {err:.2e}, 32 bits {most:.2e}")
    assert err <= most


def test_a_table_far_wider_than_the_lengths(ra):
    """2^20 columns of 1024 tokens: the line of work is then counted in groups
    of blocks, so that its longest possible form fits 32 bits."""
    b = Batch(ra, [4000, 17, 0, 1025, 900, 6000, 1, 300], [2] * 8, 16, 8, 64, 1024, torch.bfloat16,
              61)
    wide = torch.full((8, 1 << 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    attend(ra, b)


# ------------------------------------------------------------------ many rows
CHUNKS = [
    # lens, query tokens, Hq, Hkv, d, page
    ([700, 90], [20, 9], 32, 2, 128, 48),               # groups of 16
    ([1000], [33], 5, 1, 64, 4096),                     # one page holds it all
    ([260, 200, 1000], [260, 1, 27], 5, 1, 128, 16),    # a prompt, a token, a chunk
    ([40000], [64], 4, 1, 128, 128),                    # one unit on many CTAs
    ([40001, 9], [40, 1], 8, 1, 64, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", range(len(CHUNKS)))
def test_chunks(ra, shape, dtype):
    lens, n, Hq, Hkv, d, page = CHUNKS[shape]
    b = Batch(ra, lens, n, Hq, Hkv, d, page, dtype, 200 + shape)
    ws = ra.kv4_workspace()
    first = attend(ra, b, out_dtype=torch.float32, workspace=ws)
    again = attend(ra, b, out_dtype=torch.float32, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    attend(ra, b, causal=False, workspace=ws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,k_scale", [(0.0, 1.0), (1.0, 6.0), (0.125, 40.0)])
def test_chunks_flat_and_peaked(ra, scale, k_scale, d):
    """Scores far beyond what the reference in hand allows, of both signs."""
    attend(ra, Batch(ra, [600, 130], [90, 70], 4, 2, d, 16, torch.bfloat16, 210, k_scale),
           scale=scale)


def test_chunk_of_large_and_small_queries(ra):
    """Rows with a scale of their own beside ordinary ones, in the same warp."""
    b = Batch(ra, [200], [100], 2, 1, 64, 16, torch.bfloat16, 211)
    want = attend(ra, b)
    b.q[3] = 0
    b.q[5] *= 2.0 ** -60
    b.q[40, 0, 5] = 3e4
    b.q[41] *= 2.0 ** -11
    got = attend(ra, b)
    for t in (0, 1, 2, 4, 6, 39, 42, 99):
        # a warp with such a row forms its scores in another order: by bf16's step
        assert (got[0][t].float() - want[0][t].float()).abs().max() <= 2.0 ** -6
    b.q[50] *= 2.0 ** 40       # its weights sit on one key
    out, _ = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, max_q=100)
    keys, values = (kv4.kv4_values(*x) for x in b.kv[0])
    s = b.q[50].double().numpy() @ keys[:151, 0].T.astype(np.float64)
    ref = values[s.argmax(-1), 0]
    err = np.abs(out[50].double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * np.abs(ref)).all()


@pytest.mark.parametrize("n", [90, 200])
def test_pages_out_of_range_in_a_chunk(ra, n):
    """A tile with some of its pages missing and one with none of them."""
    from ring_attention_ordered_b200 import _lib
    b = Batch(ra, [700], [n], 4, 2, 64, 16, torch.bfloat16, 212)
    table = b.table.clone()
    gone = [3, 5] + list(range(16, 24)) + [43]
    for i, col in enumerate(gone):
        table[0, col] = (-1, 10 ** 6, -(1 << 31))[i % 3]
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, table, b.len_t, cu=b.cu, causal=False)
    with pytest.raises(_lib.RingAttnError) as e:
        ra.check_status()
    assert e.value.status == _lib.RA_ERR_INVALID_ARG
    keep = [c for c in range(700) if c // 16 not in gone]
    b.kv = [tuple(tuple(x[keep] for x in part) for part in b.kv[0])]
    b.lens = [len(keep)]
    b.check(out, lse, False, 0.125)


@pytest.mark.parametrize("part", ["k", "v"])
def test_nan_in_a_unit_on_many_ctas(ra, part):
    b = Batch(ra, [30000], [64], 4, 1, 128, 64, torch.bfloat16, 213)
    want = attend(ra, b)
    at = 30000 - 20                     # seen by the query tokens from 44 on
    own = b.table[0].tolist()
    slot = i32([own[at // 64] * 64 + at % 64])
    old = dict(zip("kv", ra.kv4_read(b.cache, slot)))
    old[part][0, 0, 3] = math.nan
    ra.kv4_append(old["k"], old["v"], slot, b.cache)
    out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu)
    ra.check_status()
    assert torch.equal(out[:44], want[0][:44]) and torch.equal(lse[:44], want[1][:44])
    assert bool(torch.isnan(out[44:]).all())
    if part == "k":
        assert bool(torch.isnan(lse[44:]).all())
    else:
        assert torch.equal(lse, want[1])


@pytest.mark.parametrize("n,max_q", [(100, 0), (100, 1), (100, 64), (3, 1000), (3, 2 ** 31 - 1)])
def test_max_q_need_not_be_tight(ra, n, max_q):
    """It chooses the kernel: many rows by the decoding kernel, few by the chunk kernel,
    alone and in a batch.  Either kernel's roundings are allowed for: those of p * step
    and of p and v to fp16 (see Batch.check), and of a score, ds: d / 16 instructions
    and four operations that each cut off 2^-23 of sum |q| (15 step + |zero|) at most."""
    for lens in ([300], [300, 40, 170]):
        b = Batch(ra, lens, [n] * len(lens), 4, 2, 64, 16, torch.bfloat16, 214)
        out, lse = ra.kv4_fwd(b.q.cuda(), b.cache, b.table, b.len_t, cu=b.cu, max_q=max_q,
                              out_dtype=torch.float32)
        ra.check_status()
        for i, L in enumerate(lens):
            q = b.q[i * n:i * n + n].double().numpy()
            (kc, ks, kz), (vc, vs, vz) = b.kv[i]
            v = kv4.kv4_values(vc, vs, vz)
            ref, rl, w = kv4.kv4_attention(q, kv4.kv4_values(kc, ks, kz), v, n, True, 0.125)
            none = np.isneginf(rl)
            got, gl = (x[i * n:i * n + n].double().cpu().numpy() for x in (out, lse))
            assert np.array_equal(none, np.isneginf(gl)) and (got[none] == 0).all()
            for h in range(4):
                most = (15 * ks[:, h // 2].astype(np.float64)
                        + np.abs(kz[:, h // 2].astype(np.float64))).max()
                ds = 0.125 * np.abs(q[:, h]).sum(-1) * most * (64 / 16 + 4) * 2.0 ** -23
                ds = ds + 2.0 ** -20
                seen = ~none[:, h]
                assert (np.abs(gl[seen, h] - rl[seen, h]) <= ds[seen]).all()
                big = 15 * vs[:, h // 2].astype(np.float64)
                av = np.abs(v[:, h // 2].astype(np.float64))
                tol = w[:, h] @ ((2.0 ** -10 + 2.0 ** -18) * av + 2.0 ** -11 * big[:, None])
                tol = tol + 2 * ds[:, None] * (w[:, h] @ av)
                tol = tol + L * max(av.max(), big.max()) * 2.0 ** -30
                assert (np.abs(got[:, h] - ref[:, h]) <= tol + 1e-30).all()


@pytest.mark.parametrize("n", [1, 70])
def test_a_cache_of_no_pages(ra, n):
    """Nothing cached: every row is empty; slots and lengths beyond it are reported."""
    from ring_attention_ordered_b200 import _lib
    cache = ra.kv4_cache(0, 2, 64, 16)
    q = torch.randn(2 * n, 4, 64, device="cuda").to(torch.bfloat16)
    none, cu = i32([-1] * (2 * n)), i32([0, n, 2 * n])
    table = i32([[-1, -1]] * 2)
    ra.kv4_append(q[:, :2], q[:, 2:], none, cache)
    assert all(bool((x == 0).all()) for x in ra.kv4_read(cache, none))
    for lens in ([0, 0], [0, 9]):
        out, lse = ra.kv4_fwd(q, cache, table, i32(lens), cu=cu, causal=False)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        if lens[1]:
            with pytest.raises(_lib.RingAttnError):
                ra.check_status()
        ra.check_status()
    ra.kv4_append(q[:, :2], q[:, 2:], i32([0] + [-1] * (2 * n - 1)), cache)
    with pytest.raises(_lib.RingAttnError):
        ra.check_status()


def test_many_requests(ra):
    """More requests than threads, most of them short or empty."""
    r = random.Random(5)
    lens = [r.choice([0, 1, 5, 17, 40]) for _ in range(700)]
    attend(ra, Batch(ra, lens, [1] * 700, 2, 1, 64, 16, torch.bfloat16, 41))
    n = [r.choice([1, 1, 2, 0, 40]) for _ in range(600)]
    attend(ra, Batch(ra, [max(a, b) for a, b in zip(lens, n)], n, 4, 1, 64, 16, torch.float16, 42))


def test_long_sums_keep_their_precision(ra):
    """Weights spread over many tokens: the result is small beside the values,
    and nothing that grows with the number of tokens may show.  Against the
    cached values in 64 bits, as a norm: the output's rounding (rms 2^-11 / sqrt 12
    to twice that) and as much again for rounding p."""
    L, d = 60000, 64
    g = torch.Generator().manual_seed(3)
    k = (0.3 * torch.randn(L, 1, d, generator=g)).to(torch.float16)
    v = torch.randn(L, 1, d, generator=g).to(torch.float16)
    q = torch.randn(1, 8, d, generator=g).to(torch.float16)
    cache = ra.kv4_cache(-(-L // 64), 1, d, 64)
    ra.kv4_append(k.cuda(), v.cuda(), i32(list(range(L))), cache)
    table = i32([list(range(cache.shape[0]))])
    kc, vc = (kv4.kv4_values(*oracle_values(x)) for x in (k, v))
    ref, _, _ = kv4.kv4_attention(q.double().numpy(), kc, vc, 1, True, 0.125)
    out, _ = ra.kv4_fwd(q.cuda(), cache, table, i32([L]))
    err = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err < 2 * 2.0 ** -10 / math.sqrt(12), err


def test_two_graphs_share_a_workspace_one_after_the_other(ra):
    """Two captured calls with one workspace, replayed in turn, and a third
    with its own on another stream at the same time."""
    b = [Batch(ra, lens, [n] * len(lens), 4, 2, 64, 16, torch.bfloat16, 50 + i)
         for i, (lens, n) in enumerate((([3000, 40, 777], 1), ([900, 2000], 60), ([5000], 1)))]
    want = [attend(ra, x) for x in b]
    shared, own = ra.kv4_workspace(), ra.kv4_workspace()
    side = torch.cuda.Stream()
    graphs, outs, qs = [], [], [x.q.cuda() for x in b]
    torch.cuda.synchronize()
    for i, x in enumerate(b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ra.kv4_fwd(qs[i], x.cache, x.table, x.len_t, cu=x.cu, max_q=max(x.n),
                                   workspace=own if i == 2 else shared))
        graphs.append(g)
    for _ in range(5):
        with torch.cuda.stream(side):
            graphs[2].replay()
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    ra.check_status()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_on_another_stream(ra):
    b = Batch(ra, [700, 31], [1, 3], 8, 2, 128, 64, torch.bfloat16, 24)
    s = torch.cuda.Stream()
    want = attend(ra, b)
    q = b.q.cuda()
    torch.cuda.synchronize()
    out, lse = ra.kv4_fwd(q, b.cache, b.table, b.len_t, cu=b.cu, stream=s)
    k, v = ra.kv4_read(b.cache, i32([0, 1]), stream=s)
    ra.check_status(s)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ together
def test_a_sequence_over_two_hosts_merges(ra):
    """The earlier part of a sequence on one cache (no mask), the later one on
    another (causal): ring_attn_merge of the two is attention over both."""
    L0, L1, n, Hq, Hkv, d = 300, 77, 5, 4, 2, 64
    whole = Batch(ra, [L0 + L1], [n], Hq, Hkv, d, 16, torch.bfloat16, 31)
    k, v = ((c[0], c[1], c[2]) for c in whole.kv[0])
    own = whole.table[0].tolist()
    slots = [own[c // 16] * 16 + c % 16 for c in range(L0 + L1)]
    kk, vv = ra.kv4_read(whole.cache, i32(slots), torch.float32)
    assert np.array_equal(kk.cpu().numpy(), kv4.kv4_values(*k))
    # the first 18 pages and 12 tokens, then the rest from a page of its own
    q = whole.q.cuda()
    a = ra.kv4_fwd(q, whole.cache, whole.table, i32([288]), cu=whole.cu, causal=False,
                   out_dtype=torch.float32)
    b = ra.kv4_fwd(q, whole.cache, whole.table[:, 18:].contiguous(), i32([L0 + L1 - 288]),
                   cu=whole.cu, out_dtype=torch.float32)
    out, lse = ra.merge(a[0].view(-1, d), a[1].view(-1), b[0].view(-1, d), b[1].view(-1))
    whole.check(out.view(n, Hq, d), lse.view(n, Hq), True, 0.125, torch.float32)


def serve(ra, captured):
    """A batch from its prompts on: plan, append and attention step by step,
    requests that end and start in between, on one small pool of pages."""
    R, W, page, P, Hq, Hkv, d = 5, 12, 16, 40, 4, 2, 64
    g = torch.Generator().manual_seed(77)
    r = random.Random(77)
    lens, add = i32([0] * R), i32([0] * R)
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    pool, cache, ws = ra.kv4_pool(P), ra.kv4_cache(P, Hkv, d, page), ra.kv4_workspace()
    cap = 64
    cu, slots, short = i32([0] * (R + 1)), i32([0] * cap), i32([0])
    state = (lens, table, pool, cu, slots, short)
    q = torch.zeros(cap, Hq, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(cap, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    out = torch.zeros_like(q)
    lse = torch.zeros(cap, Hq, device="cuda")

    def step():
        ra.kv4_plan(lens, add, table, pool, page, cap, out=state)
        ra.kv4_append(k, v, slots, cache)
        ra.kv4_fwd(q, cache, table, lens, cu=cu, max_q=20, out=out, lse=lse, workspace=ws)

    graph = None
    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    kept = [([], []) for _ in range(R)]
    held = [0] * R
    for i in range(25):
        todo = [20, 3, 17, 1, 9] if i == 0 else [r.choice([1, 1, 1, 1, 0, 2]) for _ in range(R)]
        for j in range(R):
            if i and held[j] and r.random() < 0.08:
                todo[j] = -1
            elif i and not held[j]:
                todo[j] = r.randint(1, 20)
        T = sum(max(a, 0) for a in todo)
        x = torch.randn(3, cap, Hq, d, generator=g).to(torch.bfloat16)
        add.copy_(torch.tensor(todo, dtype=torch.int32))
        q.copy_(x[0])
        k.copy_(x[1, :, :Hkv])
        v.copy_(x[2, :, :Hkv])
        if graph is None:
            step()
        else:
            graph.replay()
        ra.check_status()
        assert short.item() == 0
        assert cu.tolist() == [0] + list(np.cumsum([max(a, 0) for a in todo]))
        at = 0
        for j in range(R):
            m = max(todo[j], 0)
            if todo[j] < 0:
                kept[j], held[j] = ([], []), 0
                continue
            held[j] += m
            kept[j][0].append(kv4.kv4_values(*oracle_values(x[1, at:at + m, :Hkv])))
            kept[j][1].append(kv4.kv4_values(*oracle_values(x[2, at:at + m, :Hkv])))
            if m:
                ref, rl, _ = kv4.kv4_attention(x[0, at:at + m].double().numpy(),
                                               np.concatenate(kept[j][0]),
                                               np.concatenate(kept[j][1]), m, True, 0.125)
                got = out[at:at + m].double().cpu().numpy()
                assert np.abs(lse[at:at + m].cpu().numpy() - rl).max() < 1e-4
                assert np.abs(got - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -9
            at += m
        assert lens.tolist() == held


def test_serving_steps(ra):
    serve(ra, False)


def test_serving_steps_captured_and_replayed(ra):
    serve(ra, True)
