"""Cases, plain forms and 64-bit results of the operators around the paged 4-bit K/V cache.

Four operators belong together: the page plan (block tables and slot maps from request lengths), the
append (quantise new keys and values into the pages), the read (values of given slots) and attention
of query tokens over the cached ones.

The cache is a uint8 tensor [num_pages, Hkv, page / 16, 16 * (d + 8)].  The last axis is one block of
16 tokens of one page and head:
    K codes   16 rows of d / 2 bytes: element 2i in the low nibble of byte i, 2i + 1 in the high one
    K params  16 pairs (step, zero) in float16
    V codes   for keys 8h + 2t + s (h, s < 2, t < 4) and elements g * d/8 + 4w + 2b + n (g < 8,
              w < d/32, b, n < 2): byte [h][g][t][w][s][b], n = 0 in the low nibble
    V params  as K's
and a cached value is step * code + zero.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # every request of a small batch grows by one token: the call before each decoding step
        dict(name="plan_decode_8", op="plan", R=8, page=64, most=9000, prompts=0, done=0, mix=1),
        # a large server: most requests decode, some bring a prompt, some have finished
        dict(name="plan_mixed_1000", op="plan", R=1000, page=16, most=4000, prompts=48, done=37, mix=2),
        # one new token for each of a few dozen requests, written and read back
        dict(name="append_decode_33", op="append", T=33, Hkv=8, d=128, page=64, dtype="bf16", mix=3),
        # a long prompt's keys and values, an odd number of tokens, as they come out of the projection
        dict(name="append_prompt_32749", op="append", T=32749, Hkv=8, d=128, page=64, dtype="bf16", mix=4),
        # a shared prefix taken out of the cache for the bf16 kernels, small heads
        dict(name="read_prefix_4099", op="read", T=4099, Hkv=8, d=64, page=32, dtype="fp16", mix=5),
        # a whole 128K sequence taken out of the cache
        dict(name="read_128k", op="read", T=131072, Hkv=8, d=128, page=128, dtype="bf16", mix=6),
        # one request, short, one token: the smallest decoding call, where latency counts
        dict(name="decode_1x509", op="attn", R=1, lo=509, hi=509, nlo=1, nhi=1, Hq=32, Hkv=8, d=128, page=64,
             causal=True, dtype="bf16", mix=7),
        # a decoding batch of very different lengths, a request without any cached token among them
        dict(name="decode_64_ragged", op="attn", R=64, lo=0, hi=8191, nlo=1, nhi=1, Hq=32, Hkv=8, d=128, page=64,
             causal=True, dtype="bf16", mix=8),
        # one token after a million, two K/V heads
        dict(name="decode_1x1m", op="attn", R=1, lo=1048575, hi=1048575, nlo=1, nhi=1, Hq=8, Hkv=2, d=128, page=128,
             causal=True, dtype="bf16", mix=9),
        # a decoding batch at 32K with a K/V head for every query head
        dict(name="decode_8x32k_mha", op="attn", R=8, lo=30001, hi=32768, nlo=1, nhi=1, Hq=32, Hkv=32, d=128, page=64,
             causal=True, dtype="bf16", mix=10),
        # a few drafted tokens a request, eight query heads to a K/V head, small heads
        dict(name="drafts_16x8", op="attn", R=16, lo=900, hi=16000, nlo=1, nhi=8, Hq=16, Hkv=2, d=64, page=16,
             causal=True, dtype="fp16", mix=11),
        # the next chunk of two long prompts
        dict(name="chunk_2x1024", op="attn", R=2, lo=15001, hi=16384, nlo=999, nhi=1024, Hq=32, Hkv=8, d=128, page=64,
             causal=True, dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        R = _log(rng, 1, 1024)
        return dict(op=op, R=R, page=page, most=_log(rng, 64, 4000), prompts=rng.randint(0, min(R, 40)),
                    done=rng.randint(0, R // 8), mix=mix)
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op != "attn":
        return dict(op=op, T=_log(rng, 1, 32768), Hkv=rng.choice([1, 2, 4, 8]), d=d, page=page, dtype=dtype, mix=mix)
    kind = rng.choice(["decode", "decode", "drafts", "chunk"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    if kind == "decode":
        R = _log(rng, 1, 128)
        hi = _log(rng, 1, min(262144, (1 << 22) // (R * Hkv)))
        nlo = nhi = 1
    elif kind == "drafts":
        R = _log(rng, 1, 32)
        hi = _log(rng, 16, min(65536, (1 << 21) // (R * Hkv)))
        nlo, nhi = 1, rng.randint(2, 16)
    else:
        R = rng.randint(1, 3)
        nhi = _log(rng, 32, 1024)
        nlo = nhi * 3 // 4
        hi = _log(rng, nhi, 8192)
    lo = rng.choice([hi, hi // 2, 0 if kind == "decode" else hi // 4])
    return dict(op=op, R=R, lo=lo, hi=hi, nlo=nlo, nhi=nhi, Hq=G * Hkv, Hkv=Hkv, d=d, page=page,
                causal=kind != "drafts" or rng.random() < 0.7, dtype=dtype, mix=mix)


def _plan_numbers(case):
    """Lengths before the step and tokens to add (-1: the request is done) of a plan case."""
    r = random.Random(case["mix"])
    R = case["R"]
    lens = [_log(r, 1, case["most"]) for _ in range(R)]
    add = [1] * R
    for i in r.sample(range(R), case["prompts"]):
        lens[i], add[i] = 0, _log(r, 16, 2000)
    for i in r.sample(range(R), case["done"]):
        add[i] = -1
    return lens, add


def _attn_numbers(case):
    """Cached tokens and query tokens of each request of an attention case."""
    r = random.Random(case["mix"])
    R, lo, hi = case["R"], case["lo"], case["hi"]
    if lo == 0 and hi > 0:
        lens = [_log(r, 1, hi) for _ in range(R)]
        if R > 1:
            lens[r.randrange(R)] = 0
        lens[r.randrange(R)] = hi
    else:
        lens = [r.randint(lo, hi) for _ in range(R)]
    n = [r.randint(case["nlo"], case["nhi"]) for _ in range(R)]
    return lens, n


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "plan":
        lens, add = _plan_numbers(case)
        R, page, W = len(lens), case["page"], _plan_width(case)
        tokens = sum(max(a, 0) for a in add)
        pool = _plan_pool(case)
        # lengths, additions, table and pool in; lengths, table, pool, starts and slots out
        return {"bytes": 4 * (2 * R + R * W + pool + 1) + 4 * (R + R * W + pool + 1 + R + 1 + tokens) + 4, "flops": tokens}
    d = case["d"]
    packed = d + 8
    if op in ("append", "read"):
        n = case["T"] * case["Hkv"]
        read = n * (packed + 4 * d) + 4 * case["T"]
        return {"bytes": read * (2 if op == "append" else 1), "flops": n * d * (8 if op == "append" else 4)}
    lens, n = _attn_numbers(case)
    T, Hq = sum(n), case["Hq"]
    pairs = 0
    for L, m in zip(lens, n):
        if case["causal"]:
            first = L - m + 1  # keys that the first query token sees
            seen = [max(0, first), max(0, L)]
            rows = min(m, L)
            pairs += rows * (seen[1] + (L - rows + 1)) // 2 if rows > 0 else 0
        else:
            pairs += m * L
    return {"bytes": sum(lens) * case["Hkv"] * packed + T * Hq * (4 * d + 4), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _plan_width(case):
    lens, add = _plan_numbers(case)
    return max(_pages(a + max(b, 0), case["page"]) for a, b in zip(lens, add)) + 3


def _plan_pool(case):
    lens, add = _plan_numbers(case)
    need = sum(_pages(a + max(b, 0), case["page"]) for a, b in zip(lens, add))
    return need + max(8, need // 8)


def _keys_values(g, T, Hkv, d, dtype, first):
    """Keys with a few strong channels and, at a sequence's start, keys that draw attention; plain values."""
    x = torch.randn(2, T, Hkv, d, generator=g, device="cuda")
    x[0] *= 1 + 2 * (torch.rand(Hkv, d, generator=g, device="cuda") > 0.97)
    if first:
        x[0, :4] += 0.5
    return x[0].to(dtype), x[1].to(dtype)


def _blocks(k, v, page):
    """[T, Hkv, d] keys and values as the cache's pages, zeros behind the last token."""
    T, Hkv, d = k.shape
    P = _pages(T, page)
    out = []
    for x, is_v in ((k, False), (v, True)):
        codes, params = _encode(x)
        codes = torch.cat([codes, codes.new_zeros(P * page - T, Hkv, d)])
        params = torch.cat([params, params.new_zeros(P * page - T, Hkv, 2)])
        params = params.view(P, page // 16, 16, Hkv, 2).permute(0, 3, 1, 2, 4).contiguous()
        if is_v:
            # [P, block, h, t, s, Hkv, g, w, b, n] -> [P, Hkv, block, h, g, t, w, s, b, n]
            c = codes.view(P, page // 16, 2, 4, 2, Hkv, 8, d // 32, 2, 2).permute(0, 5, 1, 2, 6, 3, 7, 4, 8, 9)
        else:
            c = codes.view(P, page // 16, 16, Hkv, d // 2, 2).permute(0, 3, 1, 2, 4, 5)
        c = c.reshape(P, Hkv, page // 16, 8 * d, 2)
        out += [c[..., 0] | (c[..., 1] << 4), params.view(torch.uint8).view(P, Hkv, page // 16, 64)]
    return torch.cat(out, -1)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = random.Random(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    page = case["page"]
    if case["op"] == "plan":
        lens, add = _plan_numbers(case)
        W, pool = _plan_width(case), _plan_pool(case)
        ids = list(range(pool))
        r.shuffle(ids)
        table = np.full((len(lens), W), -1, np.int32)
        for i, L in enumerate(lens):
            for j in range(_pages(L, page)):
                table[i, j] = ids.pop()
        free = [len(ids)] + ids + [-1] * (pool - len(ids))
        tokens = sum(max(a, 0) for a in add)
        return dict(case=case, lens=torch.tensor(lens, **i32), add=torch.tensor(add, **i32),
                    table=torch.from_numpy(table).cuda(), pool=torch.tensor(free, **i32), tokens=tokens + 5)
    dtype, Hkv, d = _dtype(case), case["Hkv"], case["d"]
    if case["op"] in ("append", "read"):
        T = case["T"]
        k, v = _keys_values(g, T, Hkv, d, dtype, True)
        P = _pages(T, page) + 3
        if T <= 128:  # a token of its own request each
            P = T + 3
            at = [p * page + r.randrange(page) for p in r.sample(range(P), T)]
        else:  # a prompt over shuffled pages
            order = r.sample(range(P), _pages(T, page))
            at = (torch.tensor(order)[:, None] * page + torch.arange(page)).reshape(-1)[:T].tolist()
        slots = torch.tensor(at, **i32)
        cache = torch.zeros(P, Hkv, page // 16, 16 * (d + 8), dtype=torch.uint8, device="cuda")
        if case["op"] == "append":
            return dict(case=case, cache=cache, slots=slots, k=k, v=v)
        if T <= 128:
            kk = k.new_zeros(P * page, Hkv, d)
            vv = v.new_zeros(P * page, Hkv, d)
            kk[slots.long()], vv[slots.long()] = k, v
            cache = _blocks(kk, vv, page)
        else:
            cache[torch.tensor(order, device="cuda")] = _blocks(k, v, page)
        return dict(case=case, cache=cache, slots=slots)
    lens, n = _attn_numbers(case)
    W = max(1, max(_pages(L, page) for L in lens))
    need = sum(_pages(L, page) for L in lens)
    ids = torch.randperm(need + 2, generator=g, device="cuda")
    cache = torch.zeros(need + 2, Hkv, page // 16, 16 * (d + 8), dtype=torch.uint8, device="cuda")
    table = torch.full((len(lens), W), -1, **i32)
    at = 0
    for i, L in enumerate(lens):
        step = 65536
        for a in range(0, L, step):
            m = min(step, L - a)
            P = _pages(m, page)
            cache[ids[at:at + P]] = _blocks(*_keys_values(g, m, Hkv, d, dtype, a == 0), page)
            table[i, a // page:a // page + P] = ids[at:at + P].to(torch.int32)
            at += P
    T = sum(n)
    q = (1.5 * torch.randn(T, case["Hq"], d, generator=g, device="cuda")).to(dtype)
    state = dict(case=case, q=q, cache=cache, table=table, lens=torch.tensor(lens, **i32), most=max(lens), nmax=max(n),
                 cu=torch.tensor([0] + np.cumsum(n).tolist(), **i32), kept={})
    return state


# ------------------------------------------------------------------ plain forms
def _encode(x):
    """Codes (uint8 [..., d]) and (step, zero) pairs (float16 [..., 2]) of the last axis: zero the smallest
    value, step a fifteenth of the range rounded towards zero, each value to its nearest level, ties to the even code."""
    x = x.float().clamp(-65504.0, 65504.0)
    lo, hi = x.amin(-1), x.amax(-1)
    exact = (hi - lo) / 15
    step = exact.half()
    step = torch.where(step.float() > exact, (step.view(torch.int16) - 1).view(torch.float16), step)
    step = torch.maximum(step, torch.full_like(step, 2.0 ** -24))
    zero = lo.half()
    level = (x.double() - zero.double()[..., None]) / step.double()[..., None]
    codes = level.round().clamp(0, 15).nan_to_num(0).to(torch.uint8)
    return codes, torch.stack([step, zero], -1)


def _places(case, cache, slots):
    """Byte offsets into the flat cache of each slot's K codes, V codes and parameters, [T, Hkv, bytes]."""
    d, page, Hkv = case["d"], case["page"], case["Hkv"]
    dev = slots.device
    s = slots.long()[:, None, None]
    head = torch.arange(Hkv, device=dev)[:, None]
    p, o = s // page, s % page
    base = ((p * Hkv + head) * (page // 16) + o // 16) * (16 * (d + 8))
    i = o % 16
    byte = torch.arange(d // 2, device=dev)
    k = base + i * (d // 2) + byte
    kp = base + 8 * d + 4 * i + torch.arange(4, device=dev)
    pair, b = byte // 2, byte % 2          # 4 elements of one key are 2 bytes
    g, w = pair // (d // 32), pair % (d // 32)
    v = base + 8 * d + 64 + (i // 8) * 4 * d + (g * 4 + (i % 8) // 2) * (d // 8) + w * 4 + (i % 2) * 2 + b
    vp = base + 16 * d + 64 + 4 * i + torch.arange(4, device=dev)
    return k, kp, v, vp


def _values(codes, params):
    """step * code + zero in 32 bits from packed bytes [..., d / 2] and parameter bytes [..., 4]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = params.contiguous().view(torch.float16).float()
    return c * p[..., :1] + p[..., 1:]


def _plain_read(case, cache, slots):
    k, kp, v, vp = _places(case, cache, slots)
    flat = cache.view(-1)
    dtype = _dtype(case)
    return _values(flat[k], flat[kp]).to(dtype), _values(flat[v], flat[vp]).to(dtype)


def _plain_append(case, k, v, slots, cache):
    at = _places(case, cache, slots)
    flat = cache.view(-1)
    kc, kp = _encode(k)
    vc, vp = _encode(v)
    flat[at[0]] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    flat[at[1]] = kp.view(torch.uint8)
    flat[at[2]] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    flat[at[3]] = vp.view(torch.uint8)


def _plain_plan(lens, add, table, pool, page, tokens):
    """Releases first, their pages pushed in table order, then the new pages popped in the requests' order."""
    R, W = table.shape
    dev = lens.device
    L, a = lens.long(), add.long()
    done = a < 0
    new = torch.where(done, torch.zeros_like(L), L + a.clamp(min=0))
    old_pages, new_pages = -(-L // page), -(-new // page)
    col = torch.arange(W, device=dev)
    back = done[:, None] & (col < old_pages[:, None])
    take = ~done[:, None] & (col >= old_pages[:, None]) & (col < new_pages[:, None])
    n = pool[0].long()
    pushed = (back.flatten().cumsum(0)).view(R, W)
    popped = (take.flatten().cumsum(0)).view(R, W)
    size = pool.numel()
    stack = torch.cat([pool, pool.new_zeros(1)])  # the last place takes what is not pushed
    stack = stack.scatter(0, torch.where(back, n + pushed, torch.full_like(pushed, size)).flatten(), table.flatten())
    top = n + back.sum()
    fresh = stack[torch.where(take, top + 1 - popped, torch.zeros_like(popped))]
    table = torch.where(back, torch.full_like(table, -1), torch.where(take, fresh, table))
    count = (top - take.sum()).to(pool.dtype).view(1)
    stack = torch.cat([count, stack[1:size]])
    keep = torch.arange(size, device=dev) <= count
    stack = torch.where(keep, stack, torch.full_like(stack, -1))
    cu = torch.cat([L.new_zeros(1), a.clamp(min=0).cumsum(0)])
    i = torch.arange(tokens, device=dev)
    r = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=R - 1)
    at = (L[r] + i - cu[r]).clamp(min=0)
    slot = table[r, (at // page).clamp(max=W - 1)].long() * page + at % page
    slots = torch.where(i < cu[-1], slot, torch.full_like(slot, -1))
    return [x.to(torch.int32) for x in (new, table, stack, cu, slots)]


def _plain_attention(s):
    case = s["case"]
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    q, lens, cu, n = s["q"], s["lens"].long(), s["cu"].long(), s["nmax"]
    R = lens.numel()
    W = max(1, _pages(s["most"], page))
    b = s["cache"][s["table"][:, :W].clamp(min=0).long()]  # [R, W, Hkv, blocks, bytes]
    b = b.transpose(1, 2).reshape(R, Hkv, W * (page // 16), 16 * (d + 8))
    keys = W * page
    kc, kp, vc, vp = b.split([8 * d, 64, 8 * d, 64], -1)
    k = _values(kc.reshape(R, Hkv, keys, d // 2), kp.reshape(R, Hkv, keys, 4))
    # [.., h, g, t, w, s, b] bytes to [keys = (h, t, s), bytes = (g, w, b)]
    vc = vc.reshape(R, Hkv, -1, 2, 8, 4, d // 32, 2, 2).permute(0, 1, 2, 3, 5, 7, 4, 6, 8).reshape(R, Hkv, keys, d // 2)
    v = _values(vc, vp.reshape(R, Hkv, keys, 4))
    t = torch.arange(n, device=q.device)
    count = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + t).clamp(max=q.shape[0] - 1)
    qq = q[rows].float().view(R, n, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, d)
    x = (qq @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    end = lens[:, None] - count[:, None] + t + 1 if case["causal"] else lens[:, None].expand(R, n)
    end = torch.minimum(end, lens[:, None])
    see = torch.arange(keys, device=q.device) < end[:, :, None]  # [R, n, keys]
    x = x.view(R, Hkv, Hq // Hkv, n, keys).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = (p.view(R, Hkv, -1, keys) @ v).view(R, Hkv, Hq // Hkv, n, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, n, Hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(R, n, Hq)
    row = torch.arange(q.shape[0], device=q.device)
    r = torch.searchsorted(cu, row, right=True) - 1
    return o[r, row - cu[r]].to(q.dtype), lse[r, row - cu[r]]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from ring_attention_ordered_b200 import api
        if op == "plan":
            lens, table, pool, cu, slots, _ = api.kv4_plan(state["lens"], state["add"], state["table"], state["pool"],
                                                           case["page"], state["tokens"])
            return lens, table, pool, cu, slots
        if op == "append":
            api.kv4_append(state["k"], state["v"], state["slots"], state["cache"])
        if op in ("append", "read"):
            return api.kv4_read(state["cache"], state["slots"], _dtype(case))
        if "workspace" not in state["kept"]:
            state["kept"]["workspace"] = api.kv4_workspace(state["q"].device)
        return api.kv4_fwd(state["q"], state["cache"], state["table"], state["lens"], cu=state["cu"], max_q=state["nmax"],
                           causal=case["causal"], workspace=state["kept"]["workspace"])
    if op == "plan":
        return _plain_plan(state["lens"], state["add"], state["table"], state["pool"], case["page"], state["tokens"])
    if op == "append":
        _plain_append(case, state["k"], state["v"], state["slots"], state["cache"])
    if op in ("append", "read"):
        return _plain_read(case, state["cache"], state["slots"])
    return _plain_attention(state)


# ------------------------------------------------------------------ 64 bits
def _exact_cache(cache, d):
    """Every cached key and value in 64 bits: two [num_pages, Hkv, page, d]."""
    P, Hkv, nb, _ = cache.shape
    nibbles = lambda x: torch.stack([x & 15, x >> 4], -1).double()  # noqa: E731
    pairs = lambda x: x.contiguous().view(torch.float16).double().reshape(P, Hkv, nb * 16, 2)  # noqa: E731
    k = nibbles(cache[..., :8 * d]).reshape(P, Hkv, nb * 16, d)
    kp = pairs(cache[..., 8 * d:8 * d + 64])
    v = nibbles(cache[..., 8 * d + 64:16 * d + 64].reshape(P, Hkv, nb, 2, 8, 4, d // 32, 2, 2))
    v = v.permute(0, 1, 2, 3, 5, 7, 4, 6, 8, 9).reshape(P, Hkv, nb * 16, d)
    vp = pairs(cache[..., 16 * d + 64:])
    return kp[..., :1] * k + kp[..., 1:], vp[..., :1] * v + vp[..., 1:]


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    d, page = case["d"], case["page"]
    if case["op"] == "append":
        # the levels of each vector, and the nearest of the sixteen to each value
        found = []
        for x in (s["k"], s["v"]):
            x = x.double().clamp(-65504, 65504)
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            span = (hi.float() - lo.float()) / 15
            step = torch.from_numpy(_toward_zero(span.cpu().numpy())).cuda().double()
            levels = step * torch.arange(16, device="cuda").double() + lo.to(torch.float16).double()
            y = torch.empty_like(x)
            for a in range(0, x.shape[0], 1024):
                far = (x[a:a + 1024, :, :, None] - levels[a:a + 1024, :, None, :]).abs()
                # ties go to the even code: the first of the even ones, unless an odd one is nearer
                even, odd = far[..., 0::2].min(-1), far[..., 1::2].min(-1)
                code = torch.where(even.values <= odd.values, 2 * even.indices, 2 * odd.indices + 1)
                y[a:a + 1024] = torch.gather(levels[a:a + 1024], -1, code)
            found.append(y)
        return tuple(found)
    if case["op"] == "read":
        k, v = _exact_cache(s["cache"], d)
        at = s["slots"].long()
        return k[at // page, :, at % page], v[at // page, :, at % page]
    Hq, Hkv = case["Hq"], case["Hkv"]
    lens, n = _attn_numbers(case)
    T = sum(n)
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for i, (L, m) in enumerate(zip(lens, n)):
        if L:
            pages = s["table"][i, :_pages(L, page)].long()
            for h in range(Hkv):
                k, v = _exact_cache(s["cache"][pages, h:h + 1], d)
                k, v = k.reshape(-1, d)[:L], v.reshape(-1, d)[:L]
                end = torch.tensor([min(L, L - m + t + 1) if case["causal"] else L for t in range(m)], device="cuda")
                hide = torch.arange(L, device="cuda") >= end[:, None]
                for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    x = (s["q"][at:at + m, j].double() @ k.T) / math.sqrt(d)
                    x = x.masked_fill(hide, -math.inf)
                    z = torch.logsumexp(x, -1)
                    lse[at:at + m, j] = z
                    p = torch.where(hide, torch.zeros_like(x), torch.exp(x - z[:, None]))
                    out[at:at + m, j] = p @ v
        at += m
    return out, lse


def _toward_zero(span):
    """float16 steps of float32 spans, rounded towards zero, at least the smallest positive one."""
    h = span.astype(np.float16)
    over = h.astype(np.float32) > span
    h[over] = np.nextafter(h[over], np.float16(0))
    return np.maximum(h, np.float16(2.0 ** -24))
