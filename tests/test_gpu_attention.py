"""Paged KV cache and attention (through the C ABI) against the float64
oracle.

Tolerance, per output element, from the arithmetic that the header states:
  2^-8 |o|                    the one rounding of the bf16 output: half of
                              the spacing 2^-7 just above a power of two,
  u mean|v|                   the rounding of the weights, u = 2^-8 for bf16
                              and 2^-11 for fp16 weights (half the spacing;
                              fp16 ones are never subnormal where they count),
  2 e mean|v|                 scores off by e in every weight and in the sum:
                              e = (d + 4) 2^-24 reach for d binary32 additions
                              of exact products, with reach = max_j scale
                              sum |q_i k_ij|, plus 2^-24 (reach + 40) log2(e)
                              for the scaling and 2^-22 for the exponential,
  n 2^-23 mean|v|             binary32 sums over n keys.
All are upper bounds of the first order; the sum is taken 1.1 times for the
second.
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _say(*a):
    print("[gpu-attention]", *a, flush=True)


def bf16(x):
    """float64 values of x rounded to bfloat16, and the GPU tensor."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.to(DEV)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def limit(o, mean_abs, reach, d, keys, fp8):
    e = ((d + 4) * reach + 1.45 * (reach + 40.0)) * 2.0 ** -24 + 2.0 ** -22
    u = 2.0 ** -11 if fp8 else 2.0 ** -8
    return 1.1 * (2.0 ** -8 * np.abs(o) + (u + 2 * e[..., None] + keys * 2.0 ** -23) * mean_abs) \
        + 1e-30


def check(got, want, what):
    o, bound = want
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    off = np.abs(got - o)
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    assert np.all(off <= bound), (what, worst, got[worst], o[worst], bound[worst])


def pool(rng, pages, heads, page, d, fp8, layout):
    """A cache full of NaN (codes 0x7F), as [pages, heads, page, d] views of
    memory in the given order."""
    order = {"head": (0, 1, 2, 3), "token": (0, 2, 1, 3), "both": (0, 1, 2, 3)}[layout]
    shape = [pages, heads, page, d]
    if layout == "both":       # K and V interleaved page by page in one pool
        x = torch.empty(pages, 2, heads, page, d, dtype=torch.uint8 if fp8 else torch.bfloat16,
                        device=DEV)
        caches = x[:, 0], x[:, 1]
    else:
        mem = [shape[i] for i in order]
        back = [order.index(i) for i in range(4)]
        caches = tuple(torch.empty(mem, dtype=torch.uint8 if fp8 else torch.bfloat16,
                                   device=DEV).permute(back) for _ in range(2))
    for c in caches:
        c.fill_(0x7F if fp8 else float("nan"))
    return caches


def build(rng, lens, heads, kv_heads, d, page, fp8, layout, spare_cols=2):
    """Requests of (new, kv) lengths: the tensors of a call, written through
    the library's own tables and page writes, and each request's float64
    q, k, v."""
    kv = [b for _, b in lens]
    new = [a for a, _ in lens]
    cols = max(-(-b // page) for b in kv) + spare_cols
    need = sum(-(-b // page) for b in kv)
    pages = need + 3
    k_cache, v_cache = pool(rng, pages, kv_heads, page, d, fp8, layout)
    free = i32(rng.permutation(pages)[:max(need, 1)].tolist())
    table = torch.full((len(lens), cols), -7, dtype=torch.int32, device=DEV)
    total = sum(kv)
    k64, kd = bf16(rng.standard_normal((total, kv_heads, d)))
    v64, vd = bf16(rng.standard_normal((total, kv_heads, d)) + 0.3)
    k_scale = torch.full((1,), 0.011, device=DEV)
    v_scale = torch.full((1,), 0.013, device=DEV)
    if fp8:
        k64 = oracle.kv_decode(oracle.kv_cast(k64.reshape(total, -1), np.float32(0.011)),
                               np.float32(0.011)).reshape(k64.shape)
        v64 = oracle.kv_decode(oracle.kv_cast(v64.reshape(total, -1), np.float32(0.013)),
                               np.float32(0.013)).reshape(v64.shape)
    step = nv.kv_page_tables(i32(kv), i32([0] * len(kv)), table, free, page, total)
    nv.kv_page_write(kd, vd, k_cache, v_cache, step.slots, k_scale if fp8 else None,
                     v_scale if fp8 else None)
    q64, qd = bf16(rng.standard_normal((sum(new), heads, d)) * 1.5)
    cu, at = [0], [0]
    for a, b in lens:
        cu.append(cu[-1] + a)
        at.append(at[-1] + b)
    parts = [(q64[cu[r]:cu[r + 1]], k64[at[r]:at[r + 1]], v64[at[r]:at[r + 1]])
             for r in range(len(lens))]
    kw = dict(k_scale=k_scale, v_scale=v_scale) if fp8 else {}
    return qd, k_cache, v_cache, table, i32(cu), i32(kv), max(new), max(kv), kw, parts


def reference(parts, scale, causal, window, d, fp8):
    o, bound = [], []
    for q, k, v in parts:
        got = oracle.attention(q, k, v, scale, causal, window)
        o.append(got[0])
        bound.append(limit(*got, d, max(len(k), 1), fp8))
    return np.concatenate(o), np.concatenate(bound)


PAGED = [
    # lens, heads, kv_heads, d, page, fp8, layout, causal, window
    ([(1, 1)], 4, 4, 64, 16, False, "head", True, 0),
    ([(1, 17), (1, 16), (1, 15)], 5, 1, 128, 16, True, "head", True, 0),
    ([(1, 700), (1, 3), (1, 129), (1, 64)], 10, 2, 128, 48, False, "head", True, 0),
    ([(1, 333), (1, 1), (1, 528), (1, 529)], 10, 2, 256, 528, True, "head", True, 0),
    ([(1, 1500)], 16, 16, 64, 32, True, "token", True, 0),
    ([(1, 2100)], 5, 1, 256, 16, False, "both", True, 0),
    ([(3, 200), (2, 2), (1, 90)], 10, 2, 128, 16, True, "both", True, 0),
    ([(65, 65), (1, 300), (130, 257)], 6, 2, 64, 64, False, "token", True, 0),
    ([(200, 1000)], 5, 1, 128, 48, True, "head", True, 0),
    ([(70, 300), (33, 33)], 4, 1, 256, 16, False, "head", True, 0),
    ([(70, 300), (1, 200)], 4, 1, 256, 16, True, "token", True, 0),
    ([(40, 300), (1, 500), (7, 7)], 4, 2, 64, 32, False, "head", True, 100),
    ([(150, 400), (1, 400)], 3, 1, 128, 16, True, "head", True, 1),
    ([(50, 170), (20, 20)], 4, 2, 128, 16, False, "head", False, 0),
    ([(60, 200), (1, 77)], 4, 2, 64, 16, True, "head", False, 33),
    # 129 heads on one key/value head: one token is more than a tile of rows
    ([(2, 40), (1, 100)], 129, 1, 64, 16, False, "head", True, 0),
    # more new tokens than keys: the first rows see nothing
    ([(9, 4), (1, 0), (140, 100)], 4, 2, 128, 16, False, "head", True, 0),
    # requests without new tokens between others
    ([(0, 50), (4, 60), (0, 0), (0, 16), (5, 5), (0, 1)], 4, 2, 64, 16, True, "head", True, 0),
]


@pytest.mark.parametrize("lens,heads,kv_heads,d,page,fp8,layout,causal,window", PAGED)
def test_paged(lens, heads, kv_heads, d, page, fp8, layout, causal, window):
    _say("paged", lens, heads, kv_heads, d, page, fp8, layout, causal, window)
    rng = np.random.default_rng(len(lens) * 1000 + d + page)
    # the oracle places a request's queries at the end of its keys
    args = build(rng, lens, heads, kv_heads, d, page, fp8, layout)
    *call, kw, parts = args
    got = nv.paged_attention(*call, causal=causal, window=window, **kw)
    check(got, reference(parts, d ** -0.5, causal, window, d, fp8), "paged")


@pytest.mark.parametrize("n", [1, 63, 64, 65, 300])
def test_paged_many_requests(n):
    """The search for a tile's request over more requests than lanes."""
    _say("many requests", n)
    rng = np.random.default_rng(n)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 4, n), rng.integers(0, 40, n))]
    lens[-1] = (3, 20)
    *call, kw, parts = build(rng, lens, 4, 2, 64, 16, False, "head")
    check(nv.paged_attention(*call, **kw), reference(parts, 0.125, True, 0, 64, False), n)


@pytest.mark.parametrize("n,longest,kv_heads,d,fp8", [
    (2, 5000, 2, 64, False), (64, 3000, 1, 64, True), (70, 4000, 1, 128, False),
    (256, 2500, 1, 64, False), (257, 4500, 1, 64, False)])
def test_paged_pieces_of_many_lengths(n, longest, kv_heads, d, fp8):
    """Keys cut into pieces over requests of very different lengths, among
    them empty ones and chunks that are no single tokens."""
    _say("pieces", n, longest, kv_heads, d, fp8)
    rng = np.random.default_rng(n)
    lens = [(1, int(b)) for b in np.exp(rng.uniform(0, np.log(longest), n)).astype(int)]
    lens[0] = (1, longest)
    if n > 2:
        lens[1], lens[2], lens[n // 2] = (0, 700), (40, 900), (1, 0)
    *call, kw, parts = build(rng, lens, 2 * kv_heads, kv_heads, d, 16, fp8, "head")
    check(nv.paged_attention(*call, **kw), reference(parts, d ** -0.5, True, 0, d, fp8), n)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 2, 40])
def test_paged_split_keys(new, fp8):
    """One request whose keys are cut over many workgroups, with a bound of
    max_kv above the real length."""
    _say("split keys", new, fp8)
    rng = np.random.default_rng(new)
    *call, kw, parts = build(rng, [(new, 5003)], 5, 1, 128, 16, fp8, "head")
    call[-1] = 9000
    check(nv.paged_attention(*call, **kw), reference(parts, 128 ** -0.5, True, 0, 128, fp8), new)


def test_paged_large_scores_and_scale():
    """Scores of several hundred (one key dominates; the bound moves in every
    tile) and a scale of the caller's."""
    _say("large scores")
    rng = np.random.default_rng(5)
    *call, kw, parts = build(rng, [(1, 400), (30, 260)], 4, 2, 128, 16, False, "head")
    got = nv.paged_attention(*call, scale=9.5, **kw)
    check(got, reference(parts, 9.5, True, 0, 128, False), "scale")


def test_paged_offsets_past_32_bits():
    """Pages more than 2^32 bytes and 2^31 elements into the cache."""
    _say("offsets past 32 bits")
    rng = np.random.default_rng(6)
    heads, d, page, pages = 1, 128, 16, 1100000
    k_cache = torch.empty(pages, heads, page, d, dtype=torch.bfloat16, device=DEV)
    v_cache = torch.empty_like(k_cache)
    assert k_cache.numel() > 2 ** 31
    table = torch.full((1, 8), -1, dtype=torch.int32, device=DEV)
    free = i32([pages - 1, 0, pages - 2, 1, pages - 5])
    k64, kd = bf16(rng.standard_normal((75, heads, d)))
    v64, vd = bf16(rng.standard_normal((75, heads, d)))
    q64, qd = bf16(rng.standard_normal((2, 4, d)))
    step = nv.kv_page_tables(i32([75]), i32([0]), table, free, page, 75)
    assert int(step.slots[0]) == (pages - 1) * page
    nv.kv_page_write(kd, vd, k_cache, v_cache, step.slots)
    got = nv.paged_attention(qd, k_cache, v_cache, table, i32([0, 2]), step.kv_lens, 2, 75)
    check(got, reference([(q64, k64, v64)], d ** -0.5, True, 0, d, False), "far pages")


@pytest.mark.parametrize("seed", range(12))
def test_paged_workspace_fits_every_mask(seed):
    """One workspace query serves causal and full masks, windows or none:
    chunks whose keys are cut differently by each."""
    rng = np.random.default_rng(100 + seed)
    new = int(rng.integers(20, 400))
    lens = [(new, new + int(rng.integers(0, 1500)))]
    if seed % 2:
        lens.append((1, int(rng.integers(1, 2500))))
    d, window = (64, 128, 256)[seed % 3], (0, 300, 900)[seed // 3 % 3]
    fp8, causal = bool(seed & 1), seed % 4 != 3
    _say("workspace", lens, d, window, fp8, causal)
    *call, kw, parts = build(rng, lens, 2, 1, d, 16, fp8, "head")
    check(nv.paged_attention(*call, causal=causal, window=window, **kw),
          reference(parts, d ** -0.5, causal, window, d, fp8), seed)


def test_nothing_to_attend_to():
    """Tokens that belong to no request, bounds of zero: nothing is written."""
    _say("bounds of zero")
    q = torch.zeros(3, 34, 64, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    table = i32([[0]])
    for heads in (34, 2):
        out = torch.full((3, heads, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        nv.paged_attention(q[:, :heads], cache, cache, table, i32([0, 0]), i32([0]), 0, 0, out=out)
        nv.prompt_attention(q[:, :heads], q[:, :2], q[:, :2], i32([0, 0]), 0, out=out)
        assert (out == 7).all()
    many = i32([0] * 301)
    out = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    nv.paged_attention(q[:, :2], cache, cache, i32([[0]] * 300), many, many[:300], 0, 0, out=out)
    assert (out == 7).all()
    out = nv.paged_attention(q[:, :2], cache, cache, table, i32([0, 3]), i32([0]), 3, 0)
    assert not out.any()
    empty = nv.paged_attention(q[:0, :2], cache, cache, table, i32([0, 0]), i32([0]), 0, 0)
    assert empty.shape == (0, 2, 64)


def test_paged_page_out_of_range_reads_zeros():
    _say("page out of range")
    rng = np.random.default_rng(7)
    *call, kw, parts = build(rng, [(1, 64)], 4, 2, 64, 16, False, "head")
    call[3][0, 1] = -1
    call[3][0, 2] = 10 ** 6
    q, k, v = parts[0]
    k[16:48] = 0
    v[16:48] = 0
    check(nv.paged_attention(*call, **kw), reference([(q, k, v)], 0.125, True, 0, 64, False), "")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv,window", [(1, 300, 64), (3, 1200, 700), (40, 300, 64)])
def test_paged_before_the_window_is_unused(new, kv, window, fp8):
    """Keys that no row of the call sees may be anything, their pages gone."""
    _say("before the window", new, kv, window, fp8)
    rng = np.random.default_rng(window)
    qd, kc, vc, table, cu, lens, mn, mk, kw, parts = build(rng, [(new, kv)], 4, 2, 128, 16, fp8,
                                                           "head")
    first = kv - new - window + 1
    bad = 0x7F if fp8 else float("nan")
    for p in range(first % 16):
        for c in (kc, vc):
            c[int(table[0, first // 16]), :, p] = bad
    table[0, :first // 16] = -1
    got = nv.paged_attention(qd, kc, vc, table, cu, lens, mn, mk, window=window, **kw)
    check(got, reference(parts, 128 ** -0.5, True, window, 128, fp8), window)


def test_paged_zero_scales():
    """A K scale of zero makes every weight equal, a V scale of zero every
    output."""
    _say("zero scales")
    rng = np.random.default_rng(8)
    *call, kw, parts = build(rng, [(3, 50)], 4, 2, 64, 16, True, "head")
    zero = torch.zeros(1, device=DEV)
    q, k, v = parts[0]
    got = nv.paged_attention(*call, k_scale=zero, v_scale=kw["v_scale"])
    check(got, reference([(q, k * 0, v)], 0.125, True, 0, 64, True), "k")
    assert not nv.paged_attention(*call, k_scale=kw["k_scale"], v_scale=zero).any()


PROMPT = [
    # lens, heads, kv_heads, d, causal, window
    ([1], 4, 4, 64, True, 0),
    ([127, 128, 129, 1, 0, 2], 2, 2, 64, True, 0),
    ([700], 5, 1, 128, True, 0),
    ([300, 33, 64], 4, 2, 256, True, 0),
    ([500, 100], 4, 2, 128, True, 150),
    ([200, 31], 3, 1, 64, False, 0),
    ([150], 2, 1, 256, False, 40),
    ([0, 0, 5], 8, 2, 128, True, 3),
]


@pytest.mark.parametrize("lens,heads,kv_heads,d,causal,window", PROMPT)
def test_prompt(lens, heads, kv_heads, d, causal, window):
    """Columns of a fused projection's output in, a strided output."""
    _say("prompt", lens, heads, kv_heads, d, causal, window)
    rng = np.random.default_rng(sum(lens) + d)
    x64, x = bf16(rng.standard_normal((sum(lens), heads + 2 * kv_heads, d)))
    big = torch.full((sum(lens), heads + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    got = nv.prompt_attention(x[:, :heads], x[:, heads:heads + kv_heads],
                              x[:, heads + kv_heads:], i32(cu), max(lens), causal=causal,
                              window=window, out=big[:, 1:heads + 1])
    parts = [(x64[a:b, :heads], x64[a:b, heads:heads + kv_heads], x64[a:b, heads + kv_heads:])
             for a, b in zip(cu, cu[1:])]
    check(got, reference(parts, d ** -0.5, causal, window, d, False), "prompt")
    assert (big[:, 0] == 7).all() and (big[:, heads + 1:] == 7).all()


@pytest.mark.parametrize("n", [70, 256, 257])
def test_prompt_many_of_several_tiles(n):
    """The order of the tiles over more prompts than lanes, and over more than
    are ordered."""
    _say("many prompts", n)
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 150, n).tolist()
    lens[3] = 400
    x64, x = bf16(rng.standard_normal((sum(lens), 4, 64)))
    cu = [0]
    for a in lens:
        cu.append(cu[-1] + a)
    got = nv.prompt_attention(x[:, :2], x[:, 2:3], x[:, 3:], i32(cu), 400, window=90)
    parts = [(x64[a:b, :2], x64[a:b, 2:3], x64[a:b, 3:]) for a, b in zip(cu, cu[1:])]
    check(got, reference(parts, 0.125, True, 90, 64, False), n)


def test_prompt_agrees_with_chunks():
    """A prompt at once and in three chunks over the cache: the same rows
    within both tolerances."""
    _say("prompt against chunks")
    rng = np.random.default_rng(9)
    n, heads, kv_heads, d, page = 391, 10, 2, 128, 48
    x64, x = bf16(rng.standard_normal((n, heads + 2 * kv_heads, d)))
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    want = reference([(x64[:, :heads], x64[:, heads:heads + kv_heads],
                       x64[:, heads + kv_heads:])], d ** -0.5, True, 0, d, False)
    check(nv.prompt_attention(q, k, v, i32([0, n]), n), want, "whole")
    k_cache, v_cache = pool(rng, 12, kv_heads, page, d, False, "head")
    table = torch.full((1, 9), -1, dtype=torch.int32, device=DEV)
    free, out = i32(list(range(12))), []
    for a, b in ((0, 100), (100, 101), (101, n)):
        step = nv.kv_page_tables(i32([b - a]), i32([a]), table, free, page, b - a)
        free = free[int(step.pages_used):]
        nv.kv_page_write(k[a:b], v[a:b], k_cache, v_cache, step.slots)
        out.append(nv.paged_attention(q[a:b], k_cache, v_cache, table, step.cu_new,
                                      step.kv_lens, b - a, b))
    check(torch.cat(out), want, "chunks")


def test_repeatable_and_on_another_stream():
    """The same call gives the same bits again, also on a stream of its own."""
    _say("repeatable")
    rng = np.random.default_rng(10)
    *call, kw, _ = build(rng, [(1, 3000), (5, 900), (140, 200)], 10, 2, 128, 16, True, "head")
    first = nv.paged_attention(*call, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = nv.paged_attention(*call, **kw)
    side.synchronize()
    assert torch.equal(first.view(torch.int16), second.view(torch.int16))


def test_graph_replays():
    """A decode step captured once and replayed on growing lengths, the
    program's own eager work in between."""
    _say("graph")
    rng = np.random.default_rng(11)
    lens = [(1, 200), (1, 1000)]
    qd, kc, vc, table, cu, kv, max_new, max_kv, kw, parts = build(
        rng, lens, 10, 2, 128, 16, True, "head", spare_cols=4)
    cached = kv - 1
    free = i32([])
    new = i32([1, 1])
    out = torch.empty_like(qd)

    def step():
        s = nv.kv_page_tables(new, cached, table, free, 16, 2)
        nv.paged_attention(qd, kc, vc, table, s.cu_new, s.kv_lens, 1, 1000, out=out, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shorter in (0, 3, 100, 0):
        cached.copy_(kv - 1 - shorter)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(got, out)
        cut = [(q, k[:len(k) - shorter], v[:len(v) - shorter]) for q, k, v in parts]
        check(got, reference(cut, 128 ** -0.5, True, 0, 128, True), shorter)


def wide_pool(pages, kv_heads, page, d, fp8, stride):
    """A cache whose tokens are `stride` elements apart, K and V columns of
    one buffer full of NaN."""
    mem = torch.empty(pages * page, stride, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    mem.fill_(0x7F if fp8 else float("nan"))
    return tuple(mem.as_strided((pages, kv_heads, page, d), (page * stride, d, stride, 1),
                                i * kv_heads * d) for i in range(2))


@pytest.mark.parametrize("d,fp8,stride", [
    # the widest accepted token strides: the last multiple of 16 bytes below 2^26
    (64, False, (1 << 25) - 8), (128, False, (1 << 25) - 8), (256, False, (1 << 25) - 8),
    (64, True, (1 << 26) - 16), (128, True, (1 << 26) - 16), (256, True, (1 << 26) - 16)])
def test_paged_widest_token_stride(d, fp8, stride):
    """Keys times token stride past 2^31 and 2^32 bytes, for a chunk (tiles of
    rows), a decode and a windowed chunk: the bits of the same cache packed."""
    _say("widest token stride", d, fp8, stride)
    rng = np.random.default_rng(d)
    lens, heads, kv_heads, page = [(50, 100), (1, 39), (17, 34)], 4, 2, 16
    size = 1 if fp8 else 2
    assert 33 * stride * size > 2 ** 31 and 65 * stride * size > 2 ** 32
    qd, kc, vc, table, cu, kv, mn, mk, kw, parts = build(rng, lens, heads, kv_heads, d, page, fp8,
                                                         "head")
    wide = wide_pool(kc.shape[0], kv_heads, page, d, fp8, stride)
    for w, c in zip(wide, (kc, vc)):
        w.copy_(c)
    for causal, window in ((True, 0), (True, 21), (False, 0)):
        packed = nv.paged_attention(qd, kc, vc, table, cu, kv, mn, mk, causal=causal,
                                    window=window, **kw)
        check(packed, reference(parts, d ** -0.5, causal, window, d, fp8), (causal, window))
        got = nv.paged_attention(qd, *wide, table, cu, kv, mn, mk, causal=causal, window=window,
                                 **kw)
        assert torch.equal(got.view(torch.int16), packed.view(torch.int16)), (causal, window)


def test_write_widest_token_stride():
    """The page write into such a cache."""
    _say("write, widest token stride")
    rng = np.random.default_rng(12)
    wide = wide_pool(3, 2, 16, 64, True, (1 << 26) - 16)
    kd, vd = (bf16(rng.standard_normal((40, 2, 64)))[1] for _ in range(2))
    packed = tuple(torch.full((3, 2, 16, 64), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    scale = torch.full((1,), 0.01, device=DEV)
    slots = torch.from_numpy(rng.permutation(48)[:40]).to(DEV)
    for cache in (wide, packed):
        nv.kv_page_write(kd, vd, *cache, slots, scale, scale)
    assert torch.equal(wide[0], packed[0]) and torch.equal(wide[1], packed[1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_widest_token_stride(d):
    """Rows of keys and values as far apart as the prompt form takes them."""
    _say("prompt, widest token stride", d)
    rng = np.random.default_rng(d + 1)
    lens, heads, kv_heads, stride = [80, 3, 17], 4, 2, (1 << 25) - 8
    n = sum(lens)
    x64, x = bf16(rng.standard_normal((n, heads + 2 * kv_heads, d)))
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    mem = torch.full((n, stride), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide = tuple(mem.as_strided((n, kv_heads, d), (stride, d, 1), i * kv_heads * d)
                 for i in range(2))
    wide[0].copy_(k)
    wide[1].copy_(v)
    cu = [0]
    for a in lens:
        cu.append(cu[-1] + a)
    for causal, window in ((True, 0), (True, 21), (False, 0)):
        packed = nv.prompt_attention(q, k, v, i32(cu), max(lens), causal=causal, window=window)
        parts = [(x64[a:b, :heads], x64[a:b, heads:heads + kv_heads], x64[a:b, heads + kv_heads:])
                 for a, b in zip(cu, cu[1:])]
        check(packed, reference(parts, d ** -0.5, causal, window, d, False), (causal, window))
        got = nv.prompt_attention(q, *wide, i32(cu), max(lens), causal=causal, window=window)
        assert torch.equal(got.view(torch.int16), packed.view(torch.int16)), (causal, window)


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_chunk_offsets_past_32_bits(fp8):
    """Pages more than 2^32 bytes into the cache, read by tiles of rows."""
    _say("chunk, offsets past 32 bits", fp8)
    rng = np.random.default_rng(13)
    kv_heads, d, page, pages = 1, 128, 16, 2200000
    *call, kw, parts = build(rng, [(20, 75)], 4, kv_heads, d, page, fp8, "head")
    qd, kc, vc, table, cu, kv, mn, mk = call
    far = tuple(torch.empty(pages, kv_heads, page, d, dtype=kc.dtype, device=DEV) for _ in range(2))
    assert far[0].numel() * far[0].element_size() > 2 ** 32
    ids = [pages - 1, 0, pages - 2, 1, pages - 5]
    for b, p in enumerate(ids):
        for f, c in zip(far, (kc, vc)):
            f[p] = c[int(table[0, b])]
    table[0, :5] = i32(ids)
    got = nv.paged_attention(qd, *far, table, cu, kv, mn, mk, **kw)
    check(got, reference(parts, d ** -0.5, True, 0, d, fp8), "far pages")


@pytest.mark.parametrize("n,kv_heads,d,fp8", [(300, 2, 64, True), (1100, 4, 64, False),
                                              (2100, 4, 128, True)])
def test_paged_more_requests_than_planned(n, kv_heads, d, fp8):
    """Requests cut by the bound of their lengths, far above the lengths
    themselves, and so many that none is cut."""
    _say("more requests than planned", n, kv_heads, d, fp8)
    rng = np.random.default_rng(n)
    lens = [(1, int(b)) for b in rng.integers(1, 40, n)]
    lens[1], lens[n // 2], lens[n - 1] = (0, 30), (1, 2500), (2, 700)
    *call, kw, parts = build(rng, lens, 2 * kv_heads, kv_heads, d, 16, fp8, "head")
    call[-1] = 150000
    check(nv.paged_attention(*call, **kw), reference(parts, d ** -0.5, True, 0, d, fp8), n)


@pytest.mark.parametrize("n,heads,kv_heads,new", [(5, 6, 6, 1), (3, 6, 6, 5), (40, 6, 2, 1),
                                                  (2, 16, 1, 1), (1, 7, 7, 2), (270, 3, 1, 2)])
def test_paged_places_of_few_rows(n, heads, kv_heads, new):
    """Cut keys of requests of 1 to 16 rows: each piece's sums in places of
    their own, none past the workspace (the bytes behind it stay)."""
    _say("places of few rows", n, heads, kv_heads, new)
    rng = np.random.default_rng(n + heads)
    lens = [(int(a), int(b)) for a, b in zip(rng.integers(1, new + 1, n), rng.integers(1, 50, n))]
    lens[0], lens[n - 1] = (new, 4400), (new, 3000)
    qd, kc, vc, table, cu, kv, mn, mk, kw, parts = build(rng, lens, heads, kv_heads, 64, 16, False,
                                                         "head")
    want = reference(parts, 0.125, True, 0, 64, False)
    tokens, lib = qd.shape[0], nv.library()
    size = lib.kv_paged_attention_workspace(tokens, heads, kv_heads, 64, n, mn, mk, 0)
    assert size > 0
    work = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(qd)
    torch.cuda.synchronize()
    p = [t.data_ptr() for t in (qd, kc, vc, table, cu, kv, out, work)]
    rc = lib.kv_paged_attention(
        p[0], qd.stride(0), qd.stride(1), tokens, heads, p[1], p[2], nv.DTYPE_BF16, kc.shape[0], 16,
        kv_heads, 64, kc.stride(0), kc.stride(1), kc.stride(2), None, None, p[3], table.shape[1],
        table.stride(0), p[4], p[5], n, mn, mk, 0.125, 1, 0, p[6], out.stride(0), out.stride(1),
        p[7], size, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    check(out, want, n)
    assert (work[size:] == 0xA5).all()


@pytest.mark.parametrize("n", [3, 300])
def test_offsets_that_begin_past_zero(n):
    """Some of a step's requests: offsets that do not begin at row 0 nor end
    at the last one; the rows of the others are not written."""
    _say("offsets past zero", n)
    rng = np.random.default_rng(n + 1)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 12, n), rng.integers(0, 40, n))]
    lens[0], lens[n - 1] = (20, 33), (140, 150)
    qd, kc, vc, table, cu, kv, mn, mk, kw, parts = build(rng, lens, 4, 2, 64, 16, False, "head")
    before, after = 700, 300
    q = torch.full((before + qd.shape[0] + after, 4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[before:-after] = qd
    out = torch.full_like(q, 7.0)
    nv.paged_attention(q, kc, vc, table, cu + before, kv, mn, mk, out=out, **kw)
    check(out[before:-after], reference(parts, 0.125, True, 0, 64, False), "paged")
    assert (out[:before] == 7).all() and (out[-after:] == 7).all()
    x64, x = bf16(rng.standard_normal((q.shape[0], 8, 64)))
    out.fill_(7.0)
    nv.prompt_attention(x[:, :4], x[:, 4:6], x[:, 6:], cu + before, mn, out=out)
    at = (cu + before).tolist()
    parts = [(x64[a:b, :4], x64[a:b, 4:6], x64[a:b, 6:]) for a, b in zip(at, at[1:])]
    check(out[before:-after], reference(parts, 0.125, True, 0, 64, False), "prompt")
    assert (out[:before] == 7).all() and (out[-after:] == 7).all()


@pytest.mark.parametrize("new,kv,window,fp8", [
    (1, 70001, 0, False), (1, 70001, 50003, True), (3, 66000, 0, True), (3, 66000, 40001, False),
    (60, 40007, 0, False), (60, 40007, 30001, True), (200, 33333, 0, True),
    (200, 33333, 20011, False)])
def test_masks_to_the_key(new, kv, window, fp8):
    """Long contexts, queries of zero, so that every visible key weighs exactly
    the same, and values of zero but for 64 marks of 1 at an edge of the mask,
    each in an element of its own: a row gives 1 / (keys it sees) at the marks
    it sees, within the bf16 rounding (2^-8, and 2^-22 for the division), and
    zero at the others."""
    _say("masks to the key", new, kv, window, fp8)
    d, page, kv_heads, heads = 64, 16, 2, 4
    rng = np.random.default_rng(new + kv)
    cols = -(-kv // page)
    k_cache, v_cache = pool(rng, cols + 2, kv_heads, page, d, fp8, "head")
    table = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
    step = nv.kv_page_tables(i32([kv]), i32([0]), table, i32(rng.permutation(cols + 2).tolist()),
                             page, kv)
    one = torch.ones(1, device=DEV) if fp8 else None
    q = torch.zeros(new, heads, d, dtype=torch.bfloat16, device=DEV)
    k = torch.randn(kv, kv_heads, d, device=DEV).to(torch.bfloat16)
    rows = np.arange(kv - new, kv)
    first = np.maximum(rows - window + 1, 0) if window else np.zeros_like(rows)
    edges = [kv - 64, min(kv - new - 32, kv - 64)] + ([int(first[0]) - 32, int(first[-1]) - 32] if window
                                                 else [0])
    for edge in edges:
        v = torch.zeros(kv, kv_heads, d, dtype=torch.bfloat16, device=DEV)
        for e in range(64):
            v[edge + e, :, e] = 1.0
        nv.kv_page_write(k, v, k_cache, v_cache, step.slots, one, one)
        got = nv.paged_attention(q, k_cache, v_cache, table, i32([0, new]), step.kv_lens, new, kv,
                                 window=window, k_scale=one, v_scale=one).double().cpu().numpy()
        at = edge + np.arange(64)
        sees = (at[None] <= rows[:, None]) & (at[None] >= first[:, None])
        want = np.where(sees, 1.0 / (rows - first + 1)[:, None], 0.0)[:, None]
        assert np.all(np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -22)), edge
        assert np.all(got[np.broadcast_to(~sees[:, None], got.shape)] == 0.0), edge


@pytest.mark.parametrize("n,causal,window", [(9000, True, 0), (9000, True, 5003), (5000, False, 0),
                                             (5000, False, 1777)])
def test_prompt_masks_to_the_key(n, causal, window):
    """The same in a prompt, with marks at four places."""
    _say("prompt masks to the key", n, causal, window)
    d, heads, kv_heads = 64, 2, 1
    q = torch.zeros(n, heads, d, dtype=torch.bfloat16, device=DEV)
    k = torch.randn(n, kv_heads, d, device=DEV).to(torch.bfloat16)
    rows = np.arange(n)
    first = np.maximum(rows - window + 1, 0) if window else np.zeros_like(rows)
    last = rows if causal else np.full(n, n - 1)
    for edge in (0, 1000, n // 2 + 1, n - 64):
        v = torch.zeros(n, kv_heads, d, dtype=torch.bfloat16, device=DEV)
        for e in range(64):
            v[edge + e, :, e] = 1.0
        got = nv.prompt_attention(q, k, v, i32([0, n]), n, causal=causal,
                                  window=window).double().cpu().numpy()
        at = edge + np.arange(64)
        sees = (at[None] <= last[:, None]) & (at[None] >= first[:, None])
        want = np.where(sees, 1.0 / (last - first + 1)[:, None], 0.0)[:, None]
        assert np.all(np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -22)), edge
        assert np.all(got[np.broadcast_to(~sees[:, None], got.shape)] == 0.0), edge
