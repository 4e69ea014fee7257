"""The paged-cache and attention calls refuse bad arguments before any device
work: the C ABI with fake addresses that are never touched, the binding with
stand-ins for GPU tensors.  Runs on the CPU.  The oracle's own definition is
pinned against brute force."""
import os

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        pytest.fail("library not built: run __graft_entry__.build()")
    return nv.library()


def at(i):
    return P + i * 0x10000000


def tables(lib, **kw):
    a = dict(new=at(0), cached=at(1), n=4, table=at(2), cols=8, ld=8, free=at(3), n_free=9,
             page=16, tokens=5, cu=at(4), kv=at(5), pos=at(6), slots=at(7), used=at(8))
    a.update(kw)
    return lib.kv_page_tables(*a.values(), None)


def test_tables_validation(lib):
    for kw in ("new", "cached", "table", "free", "cu", "kv", "pos", "slots", "used"):
        assert tables(lib, **{kw: None}) == INVALID, kw
    assert tables(lib, n=0) == INVALID
    assert tables(lib, cols=0) == INVALID
    assert tables(lib, ld=7) == INVALID
    assert tables(lib, n_free=-1) == INVALID
    assert tables(lib, page=0) == INVALID
    assert tables(lib, page=1 << 25) == INVALID
    assert tables(lib, tokens=-1) == INVALID
    assert tables(lib, page=24) == UNSUPPORTED
    assert tables(lib, slots=at(7) + 4) == MISALIGNED
    assert tables(lib, cu=at(4) + 2) == MISALIGNED
    assert tables(lib, slots=at(6)) == INVALID             # outputs overlap
    assert tables(lib, kv=at(0) + 8) == INVALID            # an output on an input


def write(lib, **kw):
    a = dict(k=at(0), kt=256, kh=64, v=at(1), vt=256, vh=64, dt=1, tokens=3, kc=at(2), vc=at(3),
             ct=1, pages=4, page=16, heads=2, d=64, ps=2048, hs=1024, ts=64, ks=at(4), vs=at(5),
             slots=at(6))
    a.update(kw)
    return lib.kv_page_write(*a.values(), None)


def test_write_validation(lib):
    for kw in ("k", "v", "kc", "vc", "slots"):
        assert write(lib, **{kw: None}) == INVALID, kw
    for kw in ("ks", "vs"):
        assert write(lib, ct=2, **{kw: None}) == INVALID, kw
    for kw in ("tokens", "kt", "kh", "vt", "vh", "ps", "hs", "ts"):
        assert write(lib, **{kw: -16}) == INVALID, kw
    for kw in ("pages", "page", "heads", "d"):
        assert write(lib, **{kw: 0}) == INVALID, kw
    assert write(lib, kh=0) == INVALID                     # heads on top of each other
    assert write(lib, tokens=1 << 40) == INVALID
    assert write(lib, dt=2) == UNSUPPORTED
    assert write(lib, ct=0) == UNSUPPORTED
    assert write(lib, page=24) == UNSUPPORTED
    assert write(lib, d=24) == UNSUPPORTED
    assert write(lib, d=2048, kh=2048, vh=2048, kt=4096, vt=4096, ts=2048, hs=32768,
                 ps=65536) == UNSUPPORTED
    assert write(lib, k=at(0) + 8) == MISALIGNED
    assert write(lib, kt=260) == MISALIGNED
    assert write(lib, ts=68) == MISALIGNED
    assert write(lib, ct=2, ts=72) == MISALIGNED           # E4M3 rows of 72 bytes
    assert write(lib, slots=at(6) + 4) == MISALIGNED
    assert write(lib, kc=at(0) + 64) == INVALID            # the cache on the input
    assert write(lib, tokens=0) == OK                      # nothing to do


def paged(lib, **kw):
    a = dict(q=at(0), qt=256, qh=64, tokens=3, heads=4, kc=at(1), vc=at(2), ct=1, pages=4,
             page=16, kv_heads=2, d=64, ps=2048, hs=1024, ts=64, ks=at(3), vs=at(4),
             table=at(5), cols=4, ld=4, cu=at(6), kv=at(7), n=2, max_new=2, max_kv=64,
             scale=0.125, causal=1, window=0, out=at(8), ot=256, oh=64, ws=at(9),
             wn=1 << 26)
    a.update(kw)
    return lib.kv_paged_attention(*a.values(), None)


def test_paged_validation(lib):
    for kw in ("q", "kc", "vc", "table", "cu", "kv", "out"):
        assert paged(lib, **{kw: None}) == INVALID, kw
    assert paged(lib, ct=2, ks=None) == INVALID
    for kw in ("tokens", "max_new", "max_kv", "window", "cols", "scale"):
        assert paged(lib, **{kw: -1}) == INVALID, kw
    for kw in ("heads", "kv_heads", "n", "pages", "page"):
        assert paged(lib, **{kw: 0}) == INVALID, kw
    assert paged(lib, heads=5) == INVALID                  # not a multiple of kv_heads
    assert paged(lib, scale=0.0) == INVALID
    assert paged(lib, scale=float("nan")) == INVALID
    assert paged(lib, scale=float("inf")) == INVALID
    assert paged(lib, tokens=1 << 31) == INVALID
    assert paged(lib, n=1 << 25) == INVALID
    assert paged(lib, max_kv=1 << 31) == INVALID
    assert paged(lib, ld=3) == INVALID
    assert paged(lib, qh=32) == INVALID
    assert paged(lib, ts=1 << 26) == INVALID
    assert paged(lib, d=96, qh=96, oh=96, ts=96) == UNSUPPORTED
    assert paged(lib, ct=0) == UNSUPPORTED
    assert paged(lib, page=40) == UNSUPPORTED
    assert paged(lib, q=at(0) + 8) == MISALIGNED
    assert paged(lib, qt=260) == MISALIGNED
    assert paged(lib, out=at(8) + 4) == MISALIGNED
    assert paged(lib, table=at(5) + 2) == MISALIGNED
    assert paged(lib, out=at(0) + 64) == INVALID           # the output on the queries
    assert paged(lib, out=at(1) + 4096) == INVALID         # the output on the cache
    assert paged(lib, tokens=0) == OK


def test_paged_workspace(lib):
    """A call that needs a workspace is refused without it, with a small one,
    a misaligned one and one that lies on another buffer."""
    sizes = dict(tokens=1, heads=4, kv_heads=2, d=64, n=1, max_new=1, max_kv=100000)
    need = lib.kv_paged_attention_workspace(1, 4, 2, 64, 1, 1, 100000, 0)
    assert need > 0
    big = dict(sizes, cols=8000, ld=8000)
    assert paged(lib, ws=None, wn=need, **big) == INVALID
    assert paged(lib, wn=need - 1, **big) == INVALID
    assert paged(lib, ws=at(9) + 8, wn=need, **big) == MISALIGNED
    assert paged(lib, ws=at(0), wn=need, **big) == INVALID
    assert paged(lib, ws=at(8), wn=need, **big) == INVALID
    assert lib.kv_paged_attention_workspace(1, 4, 3, 64, 1, 1, 100, 0) == -1
    assert lib.kv_paged_attention_workspace(1, 4, 2, 65, 1, 1, 100, 0) == -1
    assert lib.prompt_attention_workspace(1, 4, 2, 64, 0, 1, 0) == -1
    assert lib.prompt_attention_workspace(1 << 20, 16, 8, 128, 4, 1 << 18, 0) == 0


def prompt(lib, **kw):
    a = dict(q=at(0), qt=256, qh=64, k=at(1), kt=128, kh=64, v=at(2), vt=128, vh=64, tokens=9,
             heads=4, kv_heads=2, d=64, cu=at(3), n=2, most=5, scale=0.125, causal=1, window=0,
             out=at(4), ot=256, oh=64, ws=at(5), wn=1 << 26)
    a.update(kw)
    return lib.prompt_attention(*a.values(), None)


def test_prompt_validation(lib):
    for kw in ("q", "k", "v", "cu", "out"):
        assert prompt(lib, **{kw: None}) == INVALID, kw
    for kw in ("tokens", "most", "window", "scale", "n", "kt", "vh", "ot"):
        assert prompt(lib, **{kw: -8}) == INVALID, kw
    assert prompt(lib, heads=3) == INVALID
    assert prompt(lib, kt=1 << 25) == INVALID
    assert prompt(lib, d=32) == UNSUPPORTED
    assert prompt(lib, v=at(2) + 2) == MISALIGNED
    assert prompt(lib, vt=132) == MISALIGNED
    assert prompt(lib, oh=66) == MISALIGNED
    assert prompt(lib, cu=at(3) + 1) == MISALIGNED
    assert prompt(lib, out=at(2)) == INVALID
    assert prompt(lib, tokens=0) == OK


# ---------------------------------------------------------------- binding

class _OnGpu(torch.Tensor):
    """A host tensor that claims to live on cuda:0 (never dereferenced)."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda:0")


def gpu(*shape, dtype=torch.bfloat16):
    return torch.Tensor._make_subclass(_OnGpu, torch.zeros(*shape, dtype=dtype))


@pytest.fixture
def no_library(monkeypatch):
    def reached():
        raise AssertionError("the library was called with unchecked buffers")
    monkeypatch.setattr(nv, "library", reached)


def ints(*shape, dtype=torch.int32):
    return gpu(*shape, dtype=dtype)


def test_binding_refuses_tables(no_library):
    good = dict(new_lens=ints(3), cached_lens=ints(3), block_table=ints(3, 4),
                free_pages=ints(5), page_size=16, n_tokens=2)
    bad = [("new_lens", torch.zeros(3, dtype=torch.int32)), ("new_lens", ints(3, dtype=torch.int64)),
           ("cached_lens", ints(4)), ("block_table", ints(2, 4)), ("block_table", ints(3, 0)),
           ("block_table", ints(4, 3).t()), ("free_pages", ints(5, dtype=torch.int64)),
           ("free_pages", ints(2, 2)), ("n_tokens", -1),
           ("out", nv.KVPages(ints(4), ints(3), ints(2), ints(2), ints(1)))]
    for name, value in bad:
        with pytest.raises(ValueError):
            nv.kv_page_tables(**dict(good, **{name: value}))


def test_binding_refuses_write(no_library):
    cache = gpu(4, 2, 16, 64)
    good = dict(k=gpu(3, 2, 64), v=gpu(3, 2, 64), k_cache=cache, v_cache=cache,
                slots=ints(3, dtype=torch.int64))
    bad = [("k", torch.zeros(3, 2, 64)), ("k", gpu(3, 2, 64, dtype=torch.float16)), ("k", gpu(3, 128)),
           ("v", gpu(3, 2, 64, dtype=torch.float32)), ("v", gpu(4, 2, 64)),
           ("v", gpu(3, 64, 2).transpose(1, 2)), ("k_cache", gpu(4, 2, 16, 128)),
           ("v_cache", gpu(4, 16, 2, 64).transpose(1, 2)),
           ("k_cache", gpu(4, 2, 16, 64, dtype=torch.uint8)), ("slots", ints(3)),
           ("slots", ints(2, dtype=torch.int64))]
    for name, value in bad:
        with pytest.raises(ValueError):
            nv.kv_page_write(**dict(good, **{name: value}))
    codes = gpu(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):                        # E4M3 without scales
        nv.kv_page_write(**dict(good, k_cache=codes, v_cache=codes))
    with pytest.raises(ValueError):                        # caches of float16
        half = gpu(4, 2, 16, 64, dtype=torch.float16)
        nv.kv_page_write(**dict(good, k_cache=half, v_cache=half))


def test_binding_refuses_attention(no_library):
    cache = gpu(4, 2, 16, 64)
    good = dict(q=gpu(3, 4, 64), k_cache=cache, v_cache=cache, block_table=ints(2, 3),
                cu_new=ints(3), kv_lens=ints(2), max_new=2, max_kv=40)
    bad = [("q", gpu(3, 4, 64, dtype=torch.float32)), ("q", gpu(3, 256)), ("q", gpu(3, 4, 128)),
           ("q", gpu(3, 5, 64)), ("q", torch.zeros(3, 4, 64, dtype=torch.bfloat16)),
           ("cu_new", ints(2)), ("kv_lens", ints(2, dtype=torch.int64)),
           ("block_table", ints(3, 3)), ("block_table", ints(2, 3, dtype=torch.int64)),
           ("out", gpu(3, 4, 64, dtype=torch.float32)), ("out", gpu(2, 4, 64))]
    for name, value in bad:
        with pytest.raises(ValueError):
            nv.paged_attention(**dict(good, **{name: value}))
    good = dict(q=gpu(5, 4, 64), k=gpu(5, 2, 64), v=gpu(5, 2, 64), cu_lens=ints(3), max_len=3)
    bad = [("q", gpu(5, 4, 64, dtype=torch.float32)), ("k", gpu(4, 2, 64)), ("k", gpu(5, 3, 64)),
           ("v", gpu(5, 1, 64)), ("v", gpu(5, 2, 64, dtype=torch.float16)),
           ("cu_lens", ints(3, dtype=torch.int64)), ("out", gpu(5, 4, 32))]
    for name, value in bad:
        with pytest.raises(ValueError):
            nv.prompt_attention(**dict(good, **{name: value}))


# ----------------------------------------------------------------- oracle

def test_oracle_attention_brute_force():
    """The oracle against sums written out key by key with math.exp."""
    import math
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 8), (7, 2, 8), (7, 2, 8)))
    for causal, window in ((True, 0), (True, 2), (False, 0), (False, 3)):
        o, _, _ = oracle.attention(q, k, v, 0.3, causal, window)
        for i in range(5):
            for h in range(4):
                p, top, bottom = 2 + i, np.zeros(8), 0.0
                for j in range(7):
                    if (causal and j > p) or (window and j <= p - window):
                        continue
                    w = math.exp(0.3 * sum(q[i, h, e] * k[j, h // 2, e] for e in range(8)))
                    top += w * v[j, h // 2]
                    bottom += w
                assert np.allclose(o[i, h], top / bottom, rtol=1e-12, atol=1e-12)


def test_oracle_attention_empty_rows():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((4, 1, 8)), rng.standard_normal((2, 1, 8))
    o, _, _ = oracle.attention(q, k, k, 1.0)
    assert not o[:2].any() and np.allclose(o[2, 0], k[0, 0])
    o, _, _ = oracle.attention(q, k[:0], k[:0], 1.0)
    assert not o.any()


def test_oracle_tables_by_hand():
    """Two requests of 16-token pages: 20 cached and 14 new fill the second
    page and open a third; 0 cached and 3 new open one."""
    t, cu, kv, pos, slots, used = oracle.page_tables([14, 3], [20, 0], [[4, 9, -1], [-1, -1, -1]],
                                                     [7, 2, 5], 16, 18)
    assert t.tolist() == [[4, 9, 7], [2, -1, -1]] and cu.tolist() == [0, 14, 17]
    assert kv.tolist() == [34, 3] and used == 2
    assert pos.tolist() == list(range(20, 34)) + [0, 1, 2, -1]
    assert slots.tolist() == [9 * 16 + i for i in range(4, 16)] + [112, 113] + [32, 33, 34, -1]


@pytest.mark.parametrize("heads,kv_heads,d", [(40, 8, 128), (20, 4, 256), (16, 16, 64),
                                              (40, 40, 128), (8, 1, 64), (16, 1, 256)])
@pytest.mark.parametrize("most", [600, 32768, 131072, 1 << 20])
def test_decode_workspace_is_bounded(lib, heads, kv_heads, d, most):
    """The sums of cut decodes take no more places, whatever the number of
    requests and the bound of their lengths, than 8192 pieces of 16 rows, or
    where the kernel cuts by the lengths (256 requests) than those pieces; and
    a 257th request does not multiply them."""
    def need(n):
        return lib.kv_paged_attention_workspace(n, heads, kv_heads, d, n, 1, most, 0)
    row = (d + 2) * 4
    for n in (257, 300, 512, 1000, 2048, 4096, 10000):
        assert need(n) <= 8192 * 16 * row, n
        assert need(n) <= 4 * max(need(256), 1 << 20), n
    for n in (2, 5, 32, 100, 255, 256):
        assert need(n) <= (n * kv_heads + 2048 + 2 * kv_heads) * 16 * row, n


@pytest.mark.parametrize("heads,kv_heads,d,new", [
    (40, 40, 128, 1), (40, 40, 128, 3), (40, 40, 128, 16), (40, 8, 128, 1), (40, 8, 128, 3),
    (16, 16, 64, 1), (16, 16, 64, 16), (16, 1, 256, 1)])
def test_decode_workspace_holds_rows_that_exist(lib, heads, kv_heads, d, new):
    """A piece has places for the rows that its request can have, not for the
    most that the kernel takes at once."""
    rows = new * heads // kv_heads
    for n in (1, 2, 100, 256, 257):
        pieces = max(n * kv_heads + 2048 + 2 * kv_heads, 8192 if n > 256 else 0)
        assert lib.kv_paged_attention_workspace(n * new, heads, kv_heads, d, n, new, 131072, 0) <= \
            pieces * rows * (d + 2) * 4, n


@pytest.mark.parametrize("heads,kv_heads,d", [(40, 8, 128), (20, 4, 256), (16, 16, 64), (64, 1, 128)])
@pytest.mark.parametrize("most", [32768, 131072, 1 << 20])
def test_chunk_workspace_is_bounded(lib, heads, kv_heads, d, most):
    """The sums of cut chunks take the rows of seven rounds of 512 tiles at
    most, whatever the number of new tokens and the length of the context."""
    for new in (17, 64, 300, 700, 1500, 2048, 3000, 3500, 4096, 6000, 7000, 8192, 10000, 13000, 16384):
        need = lib.kv_paged_attention_workspace(new, heads, kv_heads, d, 1, new, most, 0)
        assert 0 <= need <= 7 * 512 * 128 * (d + 2) * 4, new
