"""Cases that measure the MXFP4 operators and the gated delta rule.

Three operators of a Gated DeltaNet layer in the card's own 4-bit format:

  values  mxfp4_quantize, mxfp4_dequantize   a tensor in MXFP4 and read back
  gemm    mxfp4_gemm                         the product of two MXFP4 tensors
  gdn     gdn_attention                      linear attention with a decay per
                                             head, with or without the delta
                                             rule, over prompts and tokens

`own` selects the library's kernels; otherwise the same results come from
elementary torch operations in 32 bits (logarithms of decays in 64), rounded
once at the end.  `exact` is the definition in 64 bits.

Sizes: hidden width 5120; 12288 in-projection columns are 16 + 16 key heads
and 64 value heads of 128 (64 gate columns each), 10240 the same with 48;
17536 is the fused group; prompts of 32768 tokens and 32 decode requests are
the benchmark's.  The 16 heads of 64 and the odd sizes are generic.
"""
import math
import random

import torch

own = False

_F32, _BF16 = "f32", "bf16"
_TYPES = {_F32: torch.float32, _BF16: torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode batch's activations, fake-quantised: latency
        {"name": "values_32x5120", "op": "values", "rows": 32, "k": 5120, "x": _BF16},
        # the benchmark's prompt, fake-quantised: bandwidth
        {"name": "values_32768x5120", "op": "values", "rows": 32768, "k": 5120, "x": _BF16},
        # a float32 checkpoint tensor of odd sizes (161 blocks a row)
        {"name": "values_1003x5152_f32", "op": "values", "rows": 1003, "k": 5152, "x": _F32},
        # 32 decode tokens through the in-projection: the weight streams
        {"name": "gemm_32x10240x5120", "op": "gemm", "m": 32, "n": 10240, "k": 5120, "y": _BF16},
        # a ragged batch through the fused group, k no multiple of 128
        {"name": "gemm_1003x17536x5152_f32", "op": "gemm", "m": 1003, "n": 17536, "k": 5152,
         "y": _F32},
        # a chunk of a prompt through the in-projection
        {"name": "gemm_4096x12288x5120", "op": "gemm", "m": 4096, "n": 12288, "k": 5120,
         "y": _BF16},
        # the benchmark's long prompt
        {"name": "gemm_32768x10240x5120", "op": "gemm", "m": 32768, "n": 10240, "k": 5120,
         "y": _BF16},
        # a single user's next token: latency
        {"name": "gdn_one_token", "op": "gdn", "requests": 1, "new": 1, "chunks": 0,
         "even": True, "fresh": False, "k_heads": 16, "heads": 48, "dk": 128, "dv": 128,
         "delta": True},
        # 32 users' next tokens: the states are read and written
        {"name": "gdn_decode32", "op": "gdn", "requests": 32, "new": 1, "chunks": 0,
         "even": True, "fresh": False, "k_heads": 16, "heads": 64, "dk": 128, "dv": 128,
         "delta": True},
        # one step of mixed work: 3 chunks of prompts and 21 decodes
        {"name": "gdn_mixed24", "op": "gdn", "requests": 24, "new": 333, "chunks": 3,
         "even": False, "fresh": False, "k_heads": 16, "heads": 48, "dk": 128, "dv": 128,
         "delta": True},
        # seven prompts of different lengths, decay only, as many key heads
        {"name": "gdn_prompts7_decay", "op": "gdn", "requests": 7, "new": 2001, "chunks": 7,
         "even": False, "fresh": True, "k_heads": 16, "heads": 16, "dk": 64, "dv": 64,
         "delta": False},
        # the benchmark's long prompt, from an empty state
        {"name": "gdn_prompt32768", "op": "gdn", "requests": 1, "new": 32768, "chunks": 1,
         "even": True, "fresh": True, "k_heads": 16, "heads": 64, "dk": 128, "dv": 128,
         "delta": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["values", "gemm", "gemm", "gemm", "gdn", "gdn", "gdn", "gdn"])
    k = 32 * (160 if rng.random() < 0.4 else _log(rng, 1, 320))
    if op == "values":
        return {"op": op, "rows": _log(rng, 1, 32768 * 5120 // max(k, 5120)), "k": k,
                "x": rng.choice([_F32, _BF16, _BF16])}
    if op == "gemm":
        n = rng.choice([64, 128, 5120, 10240, 12288, 17536, _log(rng, 1, 17536),
                        _log(rng, 1, 17536)])
        most = 32768 * 10240 * 5120 // (n * k)      # the largest listed one's
        return {"op": op, "m": _log(rng, 1, min(32768, most)), "n": n, "k": k,
                "y": rng.choice([_F32, _BF16, _BF16])}
    k_heads, heads = rng.choice([(16, 64), (16, 48), (16, 16), (4, 12), (1, 3), (8, 8)])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (128, 48)])
    requests = _log(rng, 1, 64)
    kind = rng.choice(["tokens", "drafts", "mixed", "prompts", "prompts"])
    new = {"tokens": 1, "drafts": rng.randint(2, 8)}.get(kind) or \
        _log(rng, 9, 32768 // requests)
    return {"op": op, "requests": requests, "new": new,
            "chunks": {"mixed": rng.randint(1, requests), "prompts": requests}.get(kind, 0),
            "even": kind in ("tokens", "drafts") or rng.random() < 0.3,
            "fresh": kind == "prompts" and rng.random() < 0.5, "k_heads": k_heads,
            "heads": heads, "dk": dk, "dv": dv, "delta": rng.random() < 0.75}


def _lens(case):
    """New tokens of each request: part of the case."""
    n, new = case["requests"], case["new"]
    if case["even"]:
        return [new] * n
    rng = random.Random("%s %s %s" % (n, new, case["chunks"]))
    return [(new if i == 0 else _log(rng, 1, new)) if i < case["chunks"] else 1
            for i in range(n)]


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"values": _prepare_values, "gemm": _prepare_gemm, "gdn": _prepare_gdn}[case["op"]](
        case, gen)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _activations(gen, rows, k):
    """Normal values with one channel in a hundred 60 times as large."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    hot = torch.randperm(k, generator=gen, device="cuda")[:max(1, k // 100)]
    x[:, hot] *= 60.0
    return x


def _prepare_values(case, gen):
    return {"op": "values", "x": _activations(gen, case["rows"], case["k"]).to(_TYPES[case["x"]])}


def _prepare_gemm(case, gen):
    """Activations and weights that a program has quantised before."""
    a = _plain_codes(_activations(gen, case["m"], case["k"]).to(torch.bfloat16))
    w = torch.randn(case["n"], case["k"], generator=gen, device="cuda") * 0.02
    return {"op": "gemm", "a": a, "b": _plain_codes(w), "y": _TYPES[case["y"]]}


def _prepare_gdn(case, gen):
    n, hk, h, dk, dv = (case[s] for s in ("requests", "k_heads", "heads", "dk", "dv"))
    lens = _lens(case)
    cu = [sum(lens[:i]) for i in range(n + 1)]
    tokens = cu[-1]
    # queries, keys and values are columns of the fused projection's output
    # behind its short convolution and SiLU
    x = torch.randn(tokens, 2 * hk * dk + h * dv, generator=gen, device="cuda")
    x = (x * torch.sigmoid(x)).to(torch.bfloat16)
    q, k, v = x.split([hk * dk, hk * dk, h * dv], 1)
    # heads forget between about one and a thousand tokens
    rate = torch.exp(torch.rand(h, generator=gen, device="cuda") * math.log(1000.0)) * 1e-3
    alpha = torch.exp(-rate * torch.exp(
        0.5 * torch.randn(tokens, h, generator=gen, device="cuda")))
    beta = torch.sigmoid(torch.randn(tokens, h, generator=gen, device="cuda"))
    state = torch.randn(n + 3, h, dk, dv, generator=gen, device="cuda") * 0.3
    slots = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
    # decodes continue; of a mixed step's chunks each other one is a first one
    held = [0 if case["fresh"] or (i < case["chunks"] and i % 2 == 0) else 100 + i
            for i in range(n)]
    return {"op": "gdn", "q": q.view(tokens, hk, dk), "k": k.view(tokens, hk, dk),
            "v": v.view(tokens, h, dv), "alpha": alpha,
            "beta": beta if case["delta"] else None, "state": state, "slots": slots,
            "cu": _ints(cu), "held": _ints(held), "max_len": max(lens),
            "normalize": case["delta"]}


# ------------------------------------------------------------------- runs

def run(state):
    op = state["op"]
    if own:
        import nvfp4_w4a4_quantized_03_amd as nv
        if op == "values":
            held = nv.mxfp4_quantize(state["x"])
            return {"values": nv.mxfp4_dequantize(held, state["x"].dtype),
                    "scales": held.scales.view(torch.float8_e8m0fnu)}
        if op == "gemm":
            return nv.mxfp4_gemm(nv.MXFP4(*state["a"]), nv.MXFP4(*state["b"]), state["y"])
        out = nv.gdn_attention(state["q"], state["k"], state["v"], state["alpha"], state["beta"],
                               state["state"], state["cu"], state["max_len"],
                               slots=state["slots"], cached_lens=state["held"],
                               normalize=state["normalize"])
        return {"out": out, "state": state["state"]}
    return {"values": _plain_values, "gemm": _plain_gemm, "gdn": _plain_gdn}[op](state)


# ------------------------------------------------------------ plain forms

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_blocks(x):
    """Element codes (without signs) and scale exponents of x [rows, k]."""
    x = x.float().view(x.shape[0], -1, 32)
    top = x.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    a = (x * torch.exp2(-e.float())[..., None]).abs()
    code = (a > 0.25).to(torch.uint8)
    for mid, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                      (5.0, False)):
        code += (a >= mid) if even else (a > mid)
    return x, code, e


def _plain_values(state):
    x, code, e = _plain_blocks(state["x"])
    grid = torch.tensor(_GRID, device=x.device)
    got = torch.copysign(grid[code.long()], x) * torch.exp2(e.float())[..., None]
    return {"values": got.view(state["x"].shape).to(state["x"].dtype),
            "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _plain_codes(x):
    """(codes, scales) of x as the packed format stores them."""
    v, code, e = _plain_blocks(x)
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = code.view(x.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _plain_read(codes, scales):
    """float32 values of packed codes and scales."""
    grid = torch.tensor(_GRID + tuple(-g for g in _GRID), device=codes.device)
    x = grid[torch.stack((codes & 15, codes >> 4), -1).int()].view(codes.shape[0], -1, 32)
    return (x * torch.exp2(scales.float() - 127.0)[..., None]).view(codes.shape[0], -1)


def _plain_gemm(state):
    a, b = _plain_read(*state["a"]), _plain_read(*state["b"])
    return torch.matmul(a, b.t()).to(state["y"])


def _plain_gdn(s):
    """Chunks of up to 64 tokens: within one by products and the inverse of a
    triangular matrix, from one to the next by the state."""
    cu, most, dev = s["cu"].long(), s["max_len"], s["q"].device
    h, n, hk = s["v"].shape[1], s["slots"].numel(), s["q"].shape[1]
    c = min(64, most)
    chunks = -(-most // c)
    at = torch.arange(chunks * c, device=dev)
    real = at < (cu[1:] - cu[:-1])[:, None]                     # [n, chunks * c]
    rows = torch.where(real, cu[:-1, None] + at, 0)

    def heads(x):                       # [n, heads, chunks, c, ...]; padding is 0
        x = torch.where(real.view(real.shape + (1,) * (x.dim() - 1)), x[rows], 0)
        return x.transpose(1, 2).unflatten(2, (chunks, c))

    q, k, v = (heads(s[name].float()) for name in ("q", "k", "v"))
    if s["normalize"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q = q * s["q"].shape[2] ** -0.5
    log = torch.where(real[..., None], s["alpha"].double()[rows].clamp(min=1e-300).log(), 0.0)
    g = log.transpose(1, 2).unflatten(2, (chunks, c)).cumsum(-1)
    i = torch.arange(c, device=dev)
    decay = torch.where(i[:, None] >= i, g[..., :, None] - g[..., None, :],
                        -math.inf).exp().float()
    kk, qk = (torch.matmul(x, k.transpose(-1, -2)).repeat_interleave(h // hk, 1)
              for x in (k, q))
    k, q = k.repeat_interleave(h // hk, 1), q.repeat_interleave(h // hk, 1)
    qk.mul_(decay)
    delta = s["beta"] is not None
    if delta:
        beta = heads(s["beta"])[..., None]
        a = kk.mul_(decay).mul_(beta).tril_(-1)
        t = torch.eye(c, device=dev).expand_as(a).contiguous()
        for r in range(1, c):           # rows of the inverse of 1 + a
            t[..., r, :r] = -(a[..., r, :r, None] * t[..., :r, :r]).sum(-2)
    g_in, g_out = g.exp().float()[..., None], (g[..., -1:] - g).exp().float()[..., None]
    g_all = g[..., -1].exp().float()[..., None, None]
    k_in, k_out, q_in = k * g_in, (k * g_out).transpose(-1, -2), q * g_in
    held = s["state"][s["slots"].long()]
    held = torch.where((s["held"] > 0)[:, None, None, None], held, 0.0)
    out = torch.empty_like(v)
    for j in range(chunks):
        u = v[:, :, j]
        if delta:
            u = torch.matmul(t[:, :, j], beta[:, :, j] * (u - torch.matmul(k_in[:, :, j], held)))
        out[:, :, j] = torch.matmul(q_in[:, :, j], held) + torch.matmul(qk[:, :, j], u)
        held = g_all[:, :, j] * held + torch.matmul(k_out[:, :, j], u)
    s["state"][s["slots"].long()] = held
    out = out.flatten(2, 3).transpose(1, 2)
    return {"out": out[real].to(torch.bfloat16), "state": s["state"]}


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "values":
        # values in and out, codes and scales written and read back
        size = 2 * (4 if case["x"] == _F32 else 2) + 2 * 17 / 32
        return {"bytes": case["rows"] * case["k"] * size, "flops": 0}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * 17 / 32 + m * n * (4 if case["y"] == _F32 else 2),
                "flops": 2 * m * n * k}
    lens, h, dk, dv = _lens(case), case["heads"], case["dk"], case["dv"]
    tokens = sum(lens)
    first = sum(case["fresh"] or (i < case["chunks"] and i % 2 == 0) for i in range(len(lens)))
    moved = tokens * (4 * case["k_heads"] * dk + 4 * h * dv + (8 if case["delta"] else 4) * h)
    moved += 4 * h * dk * dv * (2 * len(lens) - first)
    return {"bytes": moved, "flops": tokens * h * dk * dv * (6 if case["delta"] else 4)}


# ------------------------------------------------------- 64-bit definition

def _exact_values(x):
    """Nearest values of the format, ties to the even code, from its
    definition; and the scales."""
    x = x.double().view(x.shape[0], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 2)
    # a logarithm next to a power of two may be off by one
    scale = torch.where(scale * 4 > top, scale / 2, torch.where(scale * 8 <= top, scale * 2, scale))
    scale = scale.clamp(min=2.0 ** -127)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    a = (x.abs() / scale).clamp(max=6.0)
    hi = torch.searchsorted(grid, a).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where(up < down, hi, torch.where(up > down, lo, lo + (lo & 1)))
    return torch.copysign(grid[code], x) * scale, scale[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "values":
        parts = [_exact_values(x) for x in s["x"].split(4096)]
        return {"values": torch.cat([p[0] for p in parts]).view(s["x"].shape),
                "scales": torch.cat([p[1] for p in parts])}
    if case["op"] == "gemm":
        return _exact_gemm(s)
    return _exact_gdn(case, s)


def _exact_read(codes, scales):
    half = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    sign, e, m = half >> 3, (half >> 1) & 3, half & 1
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1)).double()
    x = torch.where(sign == 1, -x, x) * torch.exp2(
        scales.double() - 127).repeat_interleave(32, 1)
    return x


def _exact_gemm(s):
    b = _exact_read(*s["b"]).t()
    return torch.cat([_exact_read(c, e) @ b for c, e in
                      zip(s["a"][0].split(4096), s["a"][1].split(4096))])


def _exact_gdn(case, s):
    """Token after token, all requests and heads at once."""
    lens, h = _lens(case), case["heads"]
    if max(lens) * len(lens) * h * case["dk"] * case["dv"] > 2 ** 36:
        return None
    q, k, v, alpha = (s[x].double() for x in ("q", "k", "v", "alpha"))
    beta = s["beta"].double() if case["delta"] else None
    if s["normalize"]:
        q, k = (x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q = q / math.sqrt(case["dk"])
    group = h // case["k_heads"]
    pool = s["state"].double()
    slots = s["slots"].long()
    held = pool[slots] * (s["held"] > 0).double()[:, None, None, None]
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    order = sorted(range(len(lens)), key=lambda r: -lens[r])   # the longest first
    held = held[order]
    starts = s["cu"][:-1].long()[order]
    for t in range(max(lens)):
        live = sum(n > t for n in lens)
        at = starts[:live] + t
        now = held[:live]
        now *= alpha[at][:, :, None, None]
        kt = k[at].repeat_interleave(group, 1)
        u = v[at]
        if beta is not None:
            u = beta[at][..., None] * (u - torch.matmul(kt[:, :, None], now)[:, :, 0])
        now += kt[..., None] * u[:, :, None]
        out[at] = torch.matmul(q[at].repeat_interleave(group, 1)[:, :, None], now)[:, :, 0]
    pool[slots[order]] = held
    return {"out": out, "state": pool}
