"""Cases that measure the paged KV cache and the attention operators.

Four operators of a serving step next to the W4A4 linears:

  tables   kv_page_tables    block tables, slots and positions of a step
  write    kv_page_write     new keys and values into the paged cache
  paged    paged_attention   a chunk of new tokens over the paged cache
  prompt   prompt_attention  whole prompts, packed, keys not yet paged

`own` selects the library's kernels; otherwise the same results come from
elementary torch operations in 32 bits, rounded once at the end.  `exact` is
the definition in 64 bits.

Sizes: hidden width 5120 gives 40 heads of 128 or 20 of 256; the 32768 x 1024
KV slab gives 8 key/value heads of 128 or 4 of 256; 32 decode requests and
prompts of up to 32768 tokens are the benchmark's.  The 16 heads of 64 are
generic.
"""
import math
import random

import torch

own = False

_F32, _BF16, _FP8 = "f32", "bf16", "fp8"
_TYPES = {_F32: torch.float32, _BF16: torch.bfloat16}
_HEADS = {64: (16, 16), 128: (40, 8), 256: (20, 4)}     # d: (heads, kv heads)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's bookkeeping: 32 requests, one new token each
        {"name": "tables_decode32", "op": "tables", "requests": 32, "tokens": 32,
         "most": 32768, "page": 16},
        # bookkeeping of a step that admits many prompts at once
        {"name": "tables_admit256", "op": "tables", "requests": 256, "tokens": 32768,
         "most": 4000, "page": 64},
        # 32 decode tokens of one layer into the FP8 cache (launch-bound)
        {"name": "write_decode32_fp8", "op": "write", "tokens": 32, "d": 128, "x": _BF16,
         "cache": _FP8, "page": 16},
        # the 32768-token prompt's keys and values into the FP8 cache
        {"name": "write_prompt32768_fp8", "op": "write", "tokens": 32768, "d": 256,
         "x": _BF16, "cache": _FP8, "page": 64},
        # 1003 tokens in float32 into a bf16 cache with an odd page size
        {"name": "write_1003_f32_bf16", "op": "write", "tokens": 1003, "d": 64, "x": _F32,
         "cache": _BF16, "page": 48},
        # a single user's next token on a short context: latency
        {"name": "paged_one_token_500", "op": "paged", "requests": 1, "new": 1, "chunks": 1,
         "most": 500, "even": True, "d": 128, "cache": _BF16, "page": 16, "window": 0},
        # 32 users at 32k of context, FP8 cache: the bandwidth case
        {"name": "paged_decode32_32768_fp8", "op": "paged", "requests": 32, "new": 1,
         "chunks": 32, "most": 32768, "even": True, "d": 256, "cache": _FP8, "page": 64,
         "window": 0},
        # 64 users of very different lengths, as many kv heads as heads
        {"name": "paged_ragged64_bf16", "op": "paged", "requests": 64, "new": 1, "chunks": 64,
         "most": 16384, "even": False, "d": 64, "cache": _BF16, "page": 32, "window": 0},
        # a 2048-token piece of a long prompt over what is cached of it;
        # pages of 528 tokens, as a hybrid model's state size asks for
        {"name": "paged_chunk2048_32001_fp8", "op": "paged", "requests": 1, "new": 2048,
         "chunks": 1, "most": 32001, "even": True, "d": 128, "cache": _FP8, "page": 528,
         "window": 0},
        # one step of mixed work: 3 chunks and 21 decodes, sliding window
        {"name": "paged_mixed24_window", "op": "paged", "requests": 24, "new": 333,
         "chunks": 3, "most": 9001, "even": False, "d": 256, "cache": _BF16, "page": 16,
         "window": 4096},
        # seven prompts of different lengths packed into one call
        {"name": "prompt_packed7", "op": "prompt", "requests": 7, "most": 2001,
         "even": False, "d": 256, "causal": True, "window": 0},
        # one long prompt: the compute case
        {"name": "prompt_16384", "op": "prompt", "requests": 1, "most": 16384, "even": True,
         "d": 128, "causal": True, "window": 0},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "paged", "paged", "paged", "prompt", "prompt"])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256, 528])
    d = rng.choice([64, 128, 256])
    if op == "tables":
        requests = _log(rng, 1, 512)
        return {"op": op, "requests": requests, "tokens": _log(rng, requests, 32768),
                "most": _log(rng, 1, 32768), "page": page}
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 32768), "d": d,
                "x": rng.choice([_F32, _BF16, _BF16]), "cache": rng.choice([_BF16, _FP8]),
                "page": page}
    if op == "prompt":
        requests = _log(rng, 1, 16)
        causal = rng.random() < 0.8
        pairs = 16384 * 16384 // (1 if causal else 2)       # the largest listed one's
        return {"op": op, "requests": requests,
                "most": _log(rng, 1, math.isqrt(pairs // requests)),
                "even": rng.random() < 0.3, "d": d, "causal": causal,
                "window": rng.choice([0, 0, _log(rng, 1, 4096)])}
    # the padded scores of the plain form are bounded as the listed ones' are
    requests, cache = _log(rng, 1, 64), rng.choice([_BF16, _FP8])
    held = 1 << (20 if cache == _FP8 else 19)       # tokens, as the listed ones' bytes
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
    most = _log(rng, max(1, new), min(32768, held // requests,
                                      (1 << 26) // (new * requests)))
    return {"op": op, "requests": requests, "new": new, "chunks": rng.randint(1, requests),
            "most": most, "even": rng.random() < 0.3, "d": d,
            "cache": cache, "page": page,
            "window": rng.choice([0, 0, 0, _log(rng, 1, 8192)])}


def _lens(case):
    """(new, kv) lengths of the case's requests: part of the case."""
    rng = random.Random("%s %s %s %s" % (case["requests"], case.get("new", 0), case["most"],
                                          case["d"]))
    n, most = case["requests"], case["most"]
    kv = [most if case["even"] or i == 0 else _log(rng, 1, most) for i in range(n)]
    if case["op"] == "prompt":
        return kv, kv
    # chunk lengths vary up to "new"; the other requests decode one token
    new = [min(kv[i], case["new"] if i == 0 or case["even"] else _log(rng, 1, case["new"]))
           if i < case["chunks"] else 1 for i in range(n)]
    return new, kv


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    return {"tables": _prepare_tables, "write": _prepare_write, "paged": _prepare_paged,
            "prompt": _prepare_prompt}[case["op"]](case, gen, rng)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _prepare_tables(case, gen, rng):
    n, tokens, page = case["requests"], case["tokens"], case["page"]
    of_case = random.Random("%s %s %s" % (n, tokens, case["most"]))
    cuts = sorted(of_case.sample(range(1, tokens), n - 1)) if n > 1 else []
    new = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    cached = [_log(of_case, 1, case["most"]) for _ in range(n)]
    cols = -(-(max(new) + max(cached)) // page)     # the same for every seed
    rng.shuffle(new)
    rng.shuffle(cached)
    # most of what is admitted has nothing cached yet
    cached = [0 if new[i] > 1 and rng.random() < 0.7 else cached[i] for i in range(n)]
    ids = torch.randperm(n * cols, generator=gen, device="cuda").to(torch.int32)
    held = _ints([-(-c // page) for c in cached])
    table = torch.where(torch.arange(cols, device="cuda") < held[:, None],
                        ids.view(n, cols), _ints(-1))
    free = ids.view(n, cols)[torch.arange(cols, device="cuda") >= held[:, None]]
    return {"op": "tables", "new": _ints(new), "cached": _ints(cached), "table": table,
            "free": free, "page": page, "tokens": tokens}


def _kv_scale(std):
    """A calibrated decode scale: the largest of many normal values over 448."""
    return torch.full((1,), 4.8 * std / 448.0, device="cuda")


def _pool(gen, kind, pages, heads, page, d, std):
    """Cache pages with values of a running server in them, unused ones too."""
    x = torch.empty(pages, heads, page, d, device="cuda", dtype=torch.bfloat16)
    x.normal_(0.0, std, generator=gen)
    if kind == _BF16:
        return x
    codes = torch.empty(pages, heads, page, d, device="cuda", dtype=torch.uint8)
    scale = float(4.8 * std / 448.0)
    step = max(1, (1 << 27) // (heads * page * d))
    for i in range(0, pages, step):
        codes[i:i + step] = (x[i:i + step].float() / scale).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    return codes


def _prepare_write(case, gen, rng):
    d, page, tokens = case["d"], case["page"], case["tokens"]
    heads, kv_heads = _HEADS[d]
    # keys and values are columns of the fused q|k|v projection's output
    qkv = _normal(gen, tokens, heads + 2 * kv_heads, d).to(_TYPES[case["x"]])
    pages = -(-tokens // page) + 5
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens]
    if tokens >= 4 * page:      # long runs of a prompt's tokens fill whole pages
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(tokens, device="cuda") + rng.randint(0, page - 1)
        slots = order[at // page] * page + at % page
    fp8 = case["cache"] == _FP8
    return {"op": "write", "k": qkv[:, heads:heads + kv_heads], "v": qkv[:, heads + kv_heads:],
            "k_cache": _pool(gen, case["cache"], pages, kv_heads, page, d, 1.0),
            "v_cache": _pool(gen, case["cache"], pages, kv_heads, page, d, 1.0),
            "slots": slots.to(torch.int64), "k_scale": _kv_scale(1.0) if fp8 else None,
            "v_scale": _kv_scale(1.0) if fp8 else None}


def _prepare_paged(case, gen, rng):
    d, page, n = case["d"], case["page"], case["requests"]
    heads, kv_heads = _HEADS[d]
    new, kv = _lens(case)
    cols = -(-max(kv) // page)
    held = [-(-c // page) for c in kv]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = _ints([sum(held[:i]) for i in range(n)])
    at = torch.arange(cols, device="cuda")
    table = torch.where(at < _ints(held)[:, None],
                        order[(first[:, None] + at).clamp(max=pages - 1)], _ints(-1))
    cu = [sum(new[:i]) for i in range(n + 1)]
    fp8 = case["cache"] == _FP8
    # the queries are columns of the fused projection too; the logits'
    # deviation is about 2, so that a few keys of a long context dominate
    qkv = _normal(gen, cu[-1], heads + 2 * kv_heads, d, std=2.0).to(torch.bfloat16)
    return {"op": "paged", "q": qkv[:, :heads],
            "k_cache": _pool(gen, case["cache"], pages, kv_heads, page, d, 1.0),
            "v_cache": _pool(gen, case["cache"], pages, kv_heads, page, d, 1.0),
            "k_scale": _kv_scale(1.0) if fp8 else None,
            "v_scale": _kv_scale(1.0) if fp8 else None, "table": table,
            "cu": _ints(cu), "kv": _ints(kv), "max_new": max(new), "max_kv": max(kv),
            "window": case["window"], "causal": True}


def _prepare_prompt(case, gen, rng):
    d = case["d"]
    heads, kv_heads = _HEADS[d]
    lens, _ = _lens(case)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    qkv = _normal(gen, cu[-1], heads + 2 * kv_heads, d, std=1.4).to(torch.bfloat16)
    return {"op": "prompt", "q": qkv[:, :heads], "k": qkv[:, heads:heads + kv_heads],
            "v": qkv[:, heads + kv_heads:], "cu": _ints(cu), "max_len": max(lens),
            "causal": case["causal"], "window": case["window"]}


# ------------------------------------------------------------------- runs

def run(state):
    op = state["op"]
    if own:
        import nvfp4_w4a4_quantized_03_amd as nv
        if op == "tables":
            got = nv.kv_page_tables(state["new"], state["cached"], state["table"],
                                    state["free"], state["page"], state["tokens"])
            return {"table": state["table"], "cu": got.cu_new, "kv": got.kv_lens,
                    "positions": got.positions, "slots": got.slots, "used": got.pages_used}
        if op == "write":
            nv.kv_page_write(state["k"], state["v"], state["k_cache"], state["v_cache"],
                             state["slots"], state["k_scale"], state["v_scale"])
            return _caches(state)
        if op == "paged":
            return nv.paged_attention(state["q"], state["k_cache"], state["v_cache"],
                                      state["table"], state["cu"], state["kv"],
                                      state["max_new"], state["max_kv"],
                                      causal=state["causal"], window=state["window"],
                                      k_scale=state["k_scale"], v_scale=state["v_scale"])
        return nv.prompt_attention(state["q"], state["k"], state["v"], state["cu"],
                                   state["max_len"], causal=state["causal"],
                                   window=state["window"])
    return {"tables": _plain_tables, "write": _plain_write, "paged": _plain_paged,
            "prompt": _plain_prompt}[op](state)


def _caches(state):
    """The caches as the numbers that they hold (E4M3 codes times 1)."""
    seen = torch.float8_e4m3fn if state["k_cache"].dtype == torch.uint8 else torch.bfloat16
    return {"k_cache": state["k_cache"].view(seen), "v_cache": state["v_cache"].view(seen)}


# ------------------------------------------------------------ plain forms

def _plain_tables(state):
    new, cached, table, free = state["new"], state["cached"], state["table"], state["free"]
    page, cols = state["page"], table.shape[1]
    kv = new + cached
    cu = torch.nn.functional.pad(torch.cumsum(new, 0, dtype=torch.int32), (1, 0))
    held = (cached + page - 1) // page
    need = (((kv + page - 1) // page).clamp(max=cols) - held).clamp(min=0)
    taken = torch.cumsum(need, 0, dtype=torch.int32)
    col = torch.arange(cols, dtype=torch.int32, device=new.device)
    at = col - held[:, None] + (taken - need)[:, None]
    page_id = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, page_id, table)
    t = torch.arange(state["tokens"], dtype=torch.int32, device=new.device)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=new.numel() - 1)
    pos = cached[r] + t - cu[r]
    held_by = table[r, (pos // page).clamp(max=cols - 1)].to(torch.int64)
    real = t < cu[-1]
    slots = torch.where(real & (pos // page < cols) & (held_by >= 0),
                        held_by * page + pos % page, -1)
    return {"table": table, "cu": cu, "kv": kv, "positions": torch.where(real, pos, -1),
            "slots": slots, "used": taken[-1:]}


def _plain_write(state):
    page = state["k_cache"].shape[2]
    at, off = state["slots"] // page, state["slots"] % page
    k, v = state["k"].float(), state["v"].float()
    if state["k_cache"].dtype == torch.uint8:
        state["k_cache"][at, :, off] = (k / state["k_scale"]).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        state["v_cache"][at, :, off] = (v / state["v_scale"]).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    else:
        state["k_cache"][at, :, off] = k.to(torch.bfloat16)
        state["v_cache"][at, :, off] = v.to(torch.bfloat16)
    return _caches(state)


def _plain_pages(cache, table, scale):
    """[requests, kv heads, columns * page, d] in float32."""
    x = cache[table.clamp(min=0).long()]
    x = x.view(torch.float8_e4m3fn).float() * scale if x.dtype == torch.uint8 else x.float()
    b, cols, heads, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, heads, cols * page, d)


def _plain_attention(q, k, v, cu, kv, most, causal, window):
    """Softmax attention of packed queries over padded keys
    [requests, kv heads, length, d]; a row that sees no key gives zeros."""
    tokens, heads, d = q.shape
    b, kv_heads, length, _ = k.shape
    group = heads // kv_heads
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=tokens - 1)
    x = q[rows].float()                                        # [b, most, heads, d]
    x = x.view(b, most, kv_heads, group, d).permute(0, 2, 3, 1, 4).reshape(
        b, kv_heads, group * most, d)
    s = torch.matmul(x, k.transpose(-1, -2)).view(b, kv_heads, group, most, length)
    s.mul_(1.0 / math.sqrt(d))
    j = torch.arange(length, device=q.device)
    pos = (kv - new)[:, None] + i                              # [b, most]
    seen = j < kv[:, None, None]
    if causal:
        seen = seen & (j <= pos[:, :, None])
    if window:
        seen = seen & (j > pos[:, :, None] - window)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    s.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(b, kv_heads, group * most, length), v).view(
        b, kv_heads, group, most, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(
        b, most, heads, d)
    t = torch.arange(tokens, dtype=torch.int32, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    return o[r, t - cu[r]].to(torch.bfloat16)


def _plain_paged(state):
    k = _plain_pages(state["k_cache"], state["table"], state["k_scale"])
    v = _plain_pages(state["v_cache"], state["table"], state["v_scale"])
    # slots past a request's length hold other requests' numbers
    return _plain_attention(state["q"], k, v, state["cu"], state["kv"], state["max_new"],
                            state["causal"], state["window"])


def _plain_prompt(state):
    cu, most = state["cu"], state["max_len"]
    at = (cu[:-1, None] + torch.arange(most, device=cu.device)).clamp(
        max=state["q"].shape[0] - 1)
    k = state["k"][at].float().transpose(1, 2).contiguous()
    v = state["v"][at].float().transpose(1, 2).contiguous()
    return _plain_attention(state["q"], k, v, cu, cu[1:] - cu[:-1], most, state["causal"],
                            state["window"])


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "tables":
        # lengths in; lengths, offsets and each token's position and slot out;
        # each new page's id read and written once
        n, t = case["requests"], case["tokens"]
        return {"bytes": 16 * n + 12 * t + 8 * -(-t // case["page"]), "flops": 0}
    d = case["d"]
    heads, kv_heads = _HEADS[d]
    if op == "write":
        size = 4 if case["x"] == _F32 else 2
        kept = 1 if case["cache"] == _FP8 else 2
        return {"bytes": case["tokens"] * (2 * kv_heads * d * (size + kept) + 8), "flops": 0}
    new, kv = _lens(case)
    size = 1 if case.get("cache") == _FP8 else 2
    window, causal = case["window"], case.get("causal", True)
    moved, pairs = 0, 0
    for a, b in zip(new, kv):
        first = max(0, b - a - window + 1) if window else 0
        moved += (b - first) * 2 * kv_heads * d * size + 2 * a * heads * d * 2
        for_rows = range(b - a, b)
        if causal:
            pairs += sum(min(p + 1, window) if window else p + 1 for p in for_rows)
        else:
            pairs += sum(b - (max(0, p - window + 1) if window else 0) for p in for_rows)
    return {"bytes": moved, "flops": 4 * d * heads * pairs}


# ------------------------------------------------------- 64-bit definition

def _e4m3_grid():
    """The 127 magnitudes of OCP E4M3, from its definition."""
    return torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64,
                        device="cuda")


def _nearest_e4m3(x):
    grid = _e4m3_grid()
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where(up < down, hi, torch.where(up > down, lo, lo + (lo & 1)))
    return torch.where(x < 0, -grid[code], grid[code])


def _held(cache, scale=None):
    """The numbers of cache pages in float64."""
    if cache.dtype != torch.uint8:
        return cache.double()
    code = cache.long()
    val = torch.cat([_e4m3_grid(), torch.full((1,), float("nan"), dtype=torch.float64,
                                              device="cuda")])[code & 127]
    val = torch.where(code >= 128, -val, val)
    return val if scale is None else val * scale.double()


def _exact_rows(q, k, v, first, kv, causal, window):
    """One request: q [new, heads, d], k and v [kv heads, length, d] of the
    positions first, first + 1, ...; its first row stands at kv - new."""
    new, heads, d = q.shape
    group = heads // k.shape[0]
    out = torch.zeros(new, heads, d, dtype=torch.float64, device="cuda")
    j = first + torch.arange(k.shape[1], device="cuda")
    for h in range(heads):
        kt, vh = k[h // group].t().contiguous(), v[h // group]
        for a in range(0, new, 8192):
            p = kv - new + torch.arange(a, min(new, a + 8192), device="cuda")[:, None]
            hide = j >= kv
            if causal:
                hide = hide | (j > p)
            if window:
                hide = hide | (j <= p - window)
            s = (q[a:a + 8192, h].double() @ kt) / math.sqrt(d)
            s = s.masked_fill(hide.expand_as(s), float("-inf"))
            w = torch.softmax(s, -1).nan_to_num(0.0)
            out[a:a + 8192, h] = w @ vh
    return out


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "write":
        page, fp8 = s["k_cache"].shape[2], case["cache"] == _FP8
        got = {}
        for name in ("k", "v"):
            held = _held(s[name + "_cache"])
            x = s[name].double()
            x = _nearest_e4m3(x / s[name + "_scale"].double()) if fp8 else x
            held.permute(0, 2, 1, 3)[s["slots"] // page, s["slots"] % page] = x
            got[name + "_cache"] = held
        return got
    new, kv = _lens(case)
    out = []
    for r in range(case["requests"]):
        at = sum(new[:r])
        q = s["q"][at:at + new[r]]
        if op == "prompt":
            k = s["k"][at:at + kv[r]].double().transpose(0, 1).contiguous()
            v = s["v"][at:at + kv[r]].double().transpose(0, 1).contiguous()
            first = 0
        else:
            page = case["page"]
            first = max(0, kv[r] - new[r] - case["window"] + 1) // page if case["window"] else 0
            ids = s["table"][r, first:-(-kv[r] // page)].long()
            k, v = (_held(s[c + "_cache"][ids], s[c + "_scale"]).transpose(0, 1).reshape(
                _HEADS[case["d"]][1], -1, case["d"]) for c in ("k", "v"))
            first *= page
        out.append(_exact_rows(q, k, v, first, kv[r], case.get("causal", True),
                               case["window"]))
    return torch.cat(out)
