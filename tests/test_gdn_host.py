"""gdn_attention on the CPU: the oracle against other forms of the same
recurrence, the C ABI's and the binding's refusals.  Nothing is launched."""
import os

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle
from test_attention_host import at, gpu, ints, no_library  # noqa: F401

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        pytest.fail("library not built: run __graft_entry__.build()")
    return nv.library()


# ------------------------------------------------------------------ oracle

def case(rng, tokens, k_heads, heads, dk, dv):
    q, k = rng.standard_normal((2, tokens, k_heads, dk)) * 0.4
    v = rng.standard_normal((tokens, heads, dv))
    alpha = rng.uniform(0.5, 1.0, (tokens, heads))
    beta = rng.uniform(0.0, 1.0, (tokens, heads))
    return q, k, v, alpha, beta, rng.standard_normal((heads, dk, dv))


def test_plain_rule_is_weighted_sums():
    """Without beta: o_t = scale (prod alpha S0^T q_t + sum_j prod alpha_{j+1..t}
    (k_j.q_t) v_j)."""
    q, k, v, alpha, _, s0 = case(np.random.default_rng(1), 9, 2, 4, 6, 5)
    o, s, _, _ = oracle.gdn(q, k, v, alpha, None, s0, 0.3)
    for h in range(4):
        for t in range(9):
            want = alpha[:t + 1, h].prod() * s0[h].T @ q[t, h // 2]
            for j in range(t + 1):
                want = want + alpha[j + 1:t + 1, h].prod() * (k[j, h // 2] @ q[t, h // 2]) * v[j, h]
            assert np.allclose(o[t, h], 0.3 * want, rtol=1e-12, atol=1e-12)
        last = alpha[:, h].prod() * s0[h] + sum(
            alpha[j + 1:, h].prod() * np.outer(k[j, h // 2], v[j, h]) for j in range(9))
        assert np.allclose(s[h], last, rtol=1e-12, atol=1e-12)


def test_delta_rule_is_a_product_of_reflections():
    """S_t = alpha (I - beta k k^T) S_{t-1} + beta k v^T."""
    q, k, v, alpha, beta, s0 = case(np.random.default_rng(2), 11, 1, 3, 7, 4)
    o, s, _, _ = oracle.gdn(q, k, v, alpha, beta, s0, 1.0)
    for h in range(3):
        S = s0[h].copy()
        for t in range(11):
            S = alpha[t, h] * (np.eye(7) - beta[t, h] * np.outer(k[t, 0], k[t, 0])) @ S + \
                beta[t, h] * np.outer(k[t, 0], v[t, h])
            assert np.allclose(o[t, h], S.T @ q[t, 0], rtol=1e-11, atol=1e-11)
        assert np.allclose(s[h], S, rtol=1e-11, atol=1e-11)


def test_delta_rule_recalls():
    """beta = 1, alpha = 1 and unit keys: reading with the key just written
    returns its value, whatever was there."""
    rng = np.random.default_rng(3)
    q, k, v, _, _, s0 = case(rng, 6, 2, 2, 8, 3)
    one = np.ones((6, 2))
    k = k / np.sqrt((k * k).sum(-1, keepdims=True))
    o, _, _, _ = oracle.gdn(k, k, v, one, one, s0, 1.0)
    assert np.allclose(o, v, rtol=1e-12, atol=1e-12)


def test_normalize_divides_by_norms():
    q, k, v, alpha, beta, s0 = case(np.random.default_rng(4), 5, 2, 2, 8, 3)
    a = oracle.gdn(q, k, v, alpha, beta, s0, 1.0, True)
    n = [x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k)]
    b = oracle.gdn(*n, v, alpha, beta, s0, 1.0)
    assert np.allclose(a[0], b[0], rtol=1e-13) and np.allclose(a[1], b[1], rtol=1e-13)


def test_bounds_hold_the_values():
    """size bounds the outputs and the last n the state, by Cauchy-Schwarz."""
    q, k, v, alpha, beta, s0 = case(np.random.default_rng(5), 20, 2, 4, 8, 6)
    o, s, size, (reach, w, n) = oracle.gdn(q, k, v, alpha, beta, s0, 0.5, True)
    assert (np.abs(o) <= size * (1 + 1e-12)).all() and (size <= reach * (1 + 1e-12)).all()
    assert (np.sqrt((s * s).sum(1)) <= n * (1 + 1e-12)).all() and (n <= w).all()


# ---------------------------------------------------------------- refusals

def call(lib, **kw):
    a = dict(q=at(0), qt=128, qh=64, k=at(1), kt=128, kh=64, v=at(2), vt=128, vh=32, tokens=5,
             k_heads=2, heads=4, dk=64, dv=32, alpha=at(3), lda=4, beta=at(4), ldb=4,
             state=at(5), n_slots=3, ss=8192, slots=at(6), cu=at(7), cached=at(8), n=2, most=4,
             scale=0.125, norm=1, out=at(9), ot=128, oh=32, ws=at(10), wn=1 << 26)
    a.update(kw)
    return lib.gdn_attention(*a.values(), None)


def test_validation(lib):
    for kw in ("q", "k", "v", "alpha", "state", "cu", "out"):
        assert call(lib, **{kw: None}) == INVALID, kw
    for kw in ("tokens", "most", "scale", "lda", "ldb", "qt", "kh", "vt", "ot", "ss"):
        assert call(lib, **{kw: -8}) == INVALID, kw
    for kw in ("k_heads", "heads", "n", "n_slots", "dk", "dv"):
        assert call(lib, **{kw: 0}) == INVALID, kw
    assert call(lib, heads=3) == INVALID                   # not a multiple of k_heads
    assert call(lib, lda=3) == INVALID
    assert call(lib, ldb=3) == INVALID
    assert call(lib, ss=8188) == INVALID
    assert call(lib, slots=None, n=4) == INVALID           # more requests than slots
    assert call(lib, n=1 << 20) == INVALID
    assert call(lib, tokens=1 << 26) == INVALID
    assert call(lib, most=1 << 31) == INVALID
    for bad in (0.0, float("nan"), float("inf")):
        assert call(lib, scale=bad) == INVALID
    for dk in (32, 96, 256):
        assert call(lib, dk=dk, qh=dk, kh=dk, qt=2 * dk, kt=2 * dk, ss=1 << 20) == UNSUPPORTED
    for dv in (8, 24, 528):
        assert call(lib, dv=dv, vh=528, vt=2112, oh=528, ot=2112, ss=1 << 20) == UNSUPPORTED
    assert call(lib, q=at(0) + 8) == MISALIGNED
    assert call(lib, kt=132) == MISALIGNED
    for kw in ("qt", "kt", "vt", "ot"):
        assert call(lib, **{kw: 1 << 24}) == INVALID, kw
    assert call(lib, v=at(2) + 4) == MISALIGNED
    assert call(lib, out=at(9) + 4) == MISALIGNED
    assert call(lib, state=at(5) + 8) == MISALIGNED
    assert call(lib, ss=8194) == MISALIGNED
    for kw in ("alpha", "beta", "slots", "cu", "cached"):
        assert call(lib, **{kw: at(11) + 2}) == MISALIGNED, kw
    for on in range(9):
        assert call(lib, out=at(on)) == INVALID, on
        if on != 5:
            assert call(lib, state=at(on)) == INVALID, on
    assert call(lib, tokens=0) == OK                       # nothing to do


def test_workspace(lib):
    f = lib.gdn_attention_workspace
    assert f(5, 2, 4, 64, 32, 2, 1, 1) == 0                # single tokens need none
    need = f(100, 2, 4, 64, 32, 2, 90, 1)
    assert need > f(100, 2, 4, 64, 32, 2, 90, 0) > 0       # the plain rule needs less
    big = dict(tokens=100, most=90)
    assert call(lib, ws=None, wn=need, **big) == INVALID
    assert call(lib, wn=need - 1, **big) == INVALID
    assert call(lib, ws=at(10) + 8, wn=need, **big) == MISALIGNED
    for on in range(10):
        assert call(lib, ws=at(on), wn=need, **big) == INVALID, on
    assert f(5, 2, 3, 64, 32, 2, 4, 1) == -1
    assert f(5, 2, 4, 65, 32, 2, 4, 1) == -1
    assert f(5, 2, 4, 64, 33, 2, 4, 1) == -1
    assert f(-1, 2, 4, 64, 32, 2, 4, 1) == -1
    assert f(1 << 26, 2, 4, 64, 32, 2, 4, 1) == -1


def test_binding_refuses(no_library):  # noqa: F811
    f32 = torch.float32
    good = dict(q=gpu(5, 2, 64), k=gpu(5, 2, 64), v=gpu(5, 4, 32), alpha=gpu(5, 4, dtype=f32),
                beta=gpu(5, 4, dtype=f32), state=gpu(3, 4, 64, 32, dtype=f32),
                cu_lens=ints(3), max_len=3, slots=ints(2), cached_lens=ints(2))
    bad = dict(q=[torch.zeros(5, 2, 64, dtype=torch.bfloat16), gpu(5, 2, 64, dtype=f32),
                  gpu(4, 2, 64), gpu(5, 3, 64), gpu(5, 128), gpu(5, 0, 64)],
               k=[gpu(5, 2, 32), gpu(5, 1, 64), gpu(5, 2, 64, dtype=torch.float16)],
               v=[gpu(4, 4, 32), gpu(5, 3, 32), gpu(5, 4, 32, dtype=f32),
                  gpu(5, 4, 64)[:, :, ::2]],
               alpha=[None, gpu(5, 4), gpu(5, 3, dtype=f32), gpu(4, 5, dtype=f32).t(),
                      gpu(20, dtype=f32)],
               beta=[gpu(5, 4), gpu(4, 4, dtype=f32)],
               state=[gpu(3, 4, 64, 32), gpu(3, 4, 32, 64, dtype=f32), gpu(4, 64, 32, dtype=f32),
                      gpu(3, 4, 64, 64, dtype=f32)[..., :32]],
               cu_lens=[gpu(3, dtype=f32), ints(2, 2)],
               slots=[ints(3), gpu(2, dtype=torch.int64)], cached_lens=[ints(1)],
               out=[gpu(5, 4, 32, dtype=f32), gpu(5, 4, 16)])
    for name, values in bad.items():
        for v in values:
            with pytest.raises((ValueError, AttributeError)):
                nv.gdn_attention(**dict(good, **{name: v}))
