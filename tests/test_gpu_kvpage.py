"""Block tables, slots and page writes (through the C ABI) against the
oracle: whole numbers and cache bytes exactly."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _say(*a):
    print("[gpu-kvpage]", *a, flush=True)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


TABLES = [
    # requests, largest new, largest cached, page, spare columns, free pages short by, padding
    (1, 1, 0, 16, 0, 0, 0),
    (1, 0, 40, 16, 0, 0, 0),
    (3, 100, 100, 48, 3, 0, 5),
    (257, 9, 500, 16, 1, 0, 0),
    (600, 70, 0, 32, 0, 0, 700),
    (40, 300, 90, 16, 0, 37, 3),
    (40, 300, 90, 16, -3, 0, 0),
    (5, 2000, 3000, 528, 0, 0, 0),
]


@pytest.mark.parametrize("n,new_most,cached_most,page,spare,short,pad", TABLES)
def test_tables(n, new_most, cached_most, page, spare, short, pad):
    _say("tables", n, new_most, cached_most, page, spare, short, pad)
    rng = np.random.default_rng(n + page)
    new = rng.integers(0, new_most + 1, n)
    cached = rng.integers(0, cached_most + 1, n)
    if n > 10:
        new[rng.integers(0, n, n // 4)] = 0
        cached[rng.integers(0, n, n // 4)] = 0
    cols = max(int(max(-(-(a + b) // page) for a, b in zip(new, cached))) + spare, 1)
    table = rng.integers(0, 10 ** 6, (n, cols))
    need = sum(max(0, min(-(-(a + b) // page), cols) - -(-b // page)) for a, b in zip(new, cached))
    free = rng.permutation(10 ** 6)[:max(0, need + (4 if not short else -short))]
    total = int(new.sum()) + pad
    want = oracle.page_tables(new, cached, table, free, page, total)
    # a table of more columns than are handed over
    wide = torch.full((n, cols + 3), -5, dtype=torch.int32, device=DEV)
    wide[:, :cols] = i32(table.tolist())
    got = nv.kv_page_tables(i32(new.tolist()), i32(cached.tolist()), wide[:, :cols],
                            i32(free.tolist()), page, total)
    again = nv.kv_page_tables(i32(new.tolist()), i32(cached.tolist()), wide[:, :cols],
                              i32(free.tolist()), page, total, out=got)
    assert again is got
    for name, a, b in (("table", wide[:, :cols], want[0]), ("cu", got.cu_new, want[1]),
                       ("kv", got.kv_lens, want[2]), ("positions", got.positions, want[3]),
                       ("slots", got.slots, want[4])):
        assert np.array_equal(a.cpu().numpy().astype(np.int64), b), name
    assert int(got.pages_used) == want[5]
    assert (wide[:, cols:] == -5).all()


def test_tables_negative_lengths_and_padding_only():
    _say("tables, no tokens")
    table = torch.full((2, 2), -1, dtype=torch.int32, device=DEV)
    got = nv.kv_page_tables(i32([-3, 0]), i32([-1, 20]), table, i32([]), 16, 0)
    assert got.cu_new.tolist() == [0, 0, 0] and got.kv_lens.tolist() == [0, 20]
    assert got.pages_used.tolist() == [0] and got.slots.numel() == 0
    got = nv.kv_page_tables(i32([0]), i32([0]), table[:1], i32([]), 16, 300)
    assert (got.slots == -1).all() and (got.positions == -1).all()


WRITE = [
    # tokens, heads, d, page, x, fp8, layout
    (1, 1, 64, 16, "bf16", True, "head"),
    (33, 8, 128, 16, "bf16", True, "token"),
    (100, 2, 256, 48, "f32", True, "head"),
    (257, 4, 64, 528, "f32", False, "token"),
    (70, 3, 80, 32, "bf16", False, "head"),
    (64, 5, 16, 16, "f32", True, "both"),
]


@pytest.mark.parametrize("tokens,heads,d,page,x,fp8,layout", WRITE)
def test_write(tokens, heads, d, page, x, fp8, layout):
    """Every byte of the caches: the written slots and the others."""
    _say("write", tokens, heads, d, page, x, fp8, layout)
    rng = np.random.default_rng(tokens + d)
    pages = -(-tokens // page) + 2
    dt = torch.float32 if x == "f32" else torch.bfloat16
    wide = torch.from_numpy((rng.standard_normal((tokens, 3 * heads, d)) * 2).astype(np.float32))
    wide = wide.to(dt).to(DEV)
    k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
    ct = torch.uint8 if fp8 else torch.bfloat16
    if layout == "both":
        both = torch.empty(pages, 2, heads, page, d, dtype=ct, device=DEV)
        k_cache, v_cache = both[:, 0], both[:, 1]
    elif layout == "token":
        k_cache, v_cache = (torch.empty(pages, page, heads, d, dtype=ct, device=DEV).transpose(1, 2)
                            for _ in range(2))
    else:
        k_cache, v_cache = (torch.empty(pages, heads, page, d, dtype=ct, device=DEV)
                            for _ in range(2))
    for c in (k_cache, v_cache):
        c.fill_(0x5A if fp8 else 5.0)
    slots = rng.permutation(pages * page)[:tokens]
    skip = rng.random(tokens) < 0.2
    given = np.where(skip, rng.choice([-1, pages * page, -(2 ** 40), 2 ** 40], tokens), slots)
    ks, vs = np.float32(0.013), np.float32(0.02)
    scales = (torch.tensor([ks], device=DEV), torch.tensor([vs], device=DEV)) if fp8 else ()
    nv.kv_page_write(k, v, k_cache, v_cache, torch.from_numpy(given).to(DEV), *scales)
    for src, cache, s in ((k, k_cache, ks), (v, v_cache, vs)):
        flat = src.float().cpu().numpy().reshape(tokens, -1)
        if fp8:
            want = np.full((pages, heads, page, d), 0x5A, dtype=np.uint8)
            rows = oracle.kv_cast(flat, s).reshape(tokens, heads, d)
            have = cache.contiguous().cpu().numpy()
        else:
            want = torch.full((pages, heads, page, d), 5.0, dtype=torch.bfloat16).view(torch.int16).numpy()
            rows = src.to(torch.bfloat16).cpu().contiguous().view(torch.int16).numpy()
            have = cache.contiguous().cpu().view(torch.int16).numpy()
        for t in range(tokens):
            if not skip[t]:
                want[slots[t] // page, :, slots[t] % page] = rows[t]
        assert np.array_equal(have, want)


def test_write_equals_dense_cast():
    """The codes of a page write are those of the dense cast, extreme scales
    included."""
    _say("write against cast")
    rng = np.random.default_rng(4)
    x = torch.from_numpy((rng.standard_normal((64, 4, 64)) * 3).astype(np.float32)).to(DEV)
    for s in (0.0, 2.0 ** -120, 0.01, 2.0 ** 110):
        scale = torch.tensor([s], dtype=torch.float32, device=DEV)
        cache = torch.zeros(4, 4, 16, 64, dtype=torch.uint8, device=DEV)
        other = torch.zeros_like(cache)
        nv.kv_page_write(x, x, cache, other, torch.arange(64, device=DEV), scale, scale)
        dense = nv.fp8_kv_cast(x.view(64, 256), scale).view(4, 16, 4, 64).transpose(1, 2)
        assert torch.equal(cache, dense) and torch.equal(other, dense)


def test_write_no_tokens():
    _say("write nothing")
    cache = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(0, 1, 64, device=DEV)
    nv.kv_page_write(x, x, cache, cache.clone(), torch.empty(0, dtype=torch.int64, device=DEV))
