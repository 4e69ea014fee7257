"""gdn_attention (through the C ABI) against the float64 oracle.

Tolerances, from norms that the oracle sums without cancellation (its
docstring): n bounds a state column's norm, w sums what each token rounds, both
carried by alpha (with unit keys and 0 <= beta <= 1 the delta rule's I - beta k
k^T does not lengthen an error, so errors are carried by alpha alone).

  state   A token's sums of dk products in binary32 are off by (dk/16 + 6)
          2^-24 |k| n at most, its products and additions by a few 2^-24 of n
          and |k| |u|, its normalisation by 8 2^-24: 40 2^-24 (n + |k| |beta
          v|) a token in all, 40 2^-24 w over the tokens.
  out     2^-8 |o| for its own rounding; scale |q| times the state's error;
          40 2^-24 scale |q| n for its own sum.

Requests of more than 20 tokens go in chunks, whose products take binary32
operands as sums of bf16 numbers:

  out     the state and the scores enter as one bf16 number each, 2^-8: with
          |q| the state's column norm for the one and the sum of |scores| |u|
          for the other, together 2^-8 scale |q| n at most; 2^-14 of the same
          covers the binary32 and two-number roundings.
  state   two numbers leave 2^-17 of an operand at most, of either sign from
          element to element: the state in K S and the triangular matrix, two
          sources whose squares add.  Held to sqrt(3) 2^-17 < 2^-16 of the
          columns' norms n, in the 2-norm over a request's state, which leaves
          as much for the rest.
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[gpu-gdn]", *a, flush=True)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def build(rng, lens, k_heads, heads, dk, dv, delta=True, spare=2, decay="mixed", pad=0):
    """Tensors of a call: q, k, v as columns of one projection, slots in a
    random order, spare slots and padding rows filled with NaN."""
    n, tokens = len(lens), sum(lens) + pad
    x = rng.standard_normal((tokens, 2 * k_heads * dk + heads * dv))
    x[:, :2 * k_heads * dk] += 0.3                         # keys that resemble each other
    x[sum(lens):] = np.nan
    x = torch.from_numpy(x).to(BF16).to(DEV)
    q, k, v = x.split([k_heads * dk, k_heads * dk, heads * dv], 1)
    rate = {"mixed": np.exp(rng.uniform(np.log(1e-3), np.log(2.0), (1, heads))),
            "slow": np.full((1, heads), 1e-4), "fast": np.full((1, heads), 8.0),
            "none": np.zeros((1, heads))}[decay]
    alpha = np.exp(-rate * np.exp(0.5 * rng.standard_normal((tokens, heads))))
    if decay == "fast":
        alpha[rng.random((tokens, heads)) < 0.2] = 0.0     # underflown gates
    beta = 1 / (1 + np.exp(-2 * rng.standard_normal((tokens, heads))))
    beta[rng.random((tokens, heads)) < 0.05] = 1.0
    beta[rng.random((tokens, heads)) < 0.05] = 0.0
    alpha, beta = (torch.from_numpy(g).to(F32).to(DEV) for g in (alpha, beta))
    state = torch.full((n + spare, heads, dk, dv), float("nan"), device=DEV)
    slots = rng.permutation(n + spare)[:n]
    state[torch.from_numpy(slots).to(DEV)] = torch.from_numpy(
        rng.standard_normal((n, heads, dk, dv))).to(F32).to(DEV)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return dict(q=q.view(tokens, k_heads, dk), k=k.view(tokens, k_heads, dk),
                v=v.view(tokens, heads, dv), alpha=alpha, beta=beta if delta else None,
                state=state, cu_lens=i32(cu), max_len=max(lens), slots=i32(slots),
                normalize=delta)


def reference(c, held=None, scale=None):
    """The oracle's answer for every request: [(o, S, size, reach, w)]."""
    q, k, v, alpha = (c[x].double().cpu().numpy() for x in ("q", "k", "v", "alpha"))
    beta = None if c["beta"] is None else c["beta"].double().cpu().numpy()
    state = c["state"].double().cpu().numpy()
    cu, slots = c["cu_lens"].cpu().numpy(), c["slots"].cpu().numpy()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    got = []
    for r in range(len(cu) - 1):
        a, b = cu[r], cu[r + 1]
        s0 = state[slots[r]] if held is None or held[r] > 0 else np.zeros(state.shape[1:])
        o, s, size, (reach, w, n) = oracle.gdn(q[a:b], k[a:b], v[a:b], alpha[a:b],
                                            None if beta is None else beta[a:b], s0, scale,
                                            c["normalize"])
        got.append((o, s, size, reach, w, n))
    return got


def compare(got_o, got_s, ref, what, chunked=None):
    """One request's outputs and state within what the header derives."""
    o, s, size, reach, w, n = ref
    chunked = len(o) > 20 if chunked is None else chunked
    assert np.isfinite(got_o).all() and np.isfinite(got_s).all(), what
    e = 40 * 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(o) + ((2.0 ** -8 + 2.0 ** -14) * size if chunked
                                   else e * (reach + size))
    off, tol = np.abs(got_o - o), 1.1 * tol + 1e-30
    worst = np.unravel_index(np.argmax(off - tol), off.shape)
    assert (off <= tol).all(), (what, "out", worst, got_o[worst], o[worst], tol[worst])
    off = np.abs(got_s - s)
    if chunked:
        norm = np.linalg.norm(off), 2.0 ** -16 * np.linalg.norm(n)
        assert norm[0] <= norm[1], (what, "state", norm)
    else:
        tol = np.broadcast_to(1.1 * e * w[:, None] + 1e-30, off.shape)
        worst = np.unravel_index(np.argmax(off - tol), off.shape)
        assert (off <= tol).all(), (what, "state", worst, got_s[worst], s[worst], tol[worst])


def check(c, out, before, want, what):
    """Outputs and states of a call; slots and rows of no request stay."""
    cu, slots = c["cu_lens"].cpu().numpy(), c["slots"].cpu().numpy()
    got, state = out.double().cpu().numpy(), c["state"].double().cpu().numpy()
    for r, ref in enumerate(want):
        if cu[r + 1] == cu[r]:
            kept = (t[slots[r]].view(torch.int32) for t in (c["state"], before))  # NaN too
            assert torch.equal(*kept), (what, r)
        else:
            compare(got[cu[r]:cu[r + 1]], state[slots[r]], ref, (what, r))
    rest = np.setdiff1d(np.arange(len(state)), slots)
    assert np.isnan(state[rest]).all(), what


def run(c, held=None, scale=None, what="", **kw):
    want = reference(c, held, scale)
    before = c["state"].clone()
    if held is not None:
        # what the slot of a first request holds is never read
        for r, h in enumerate(held):
            if h <= 0 and int(c["cu_lens"][r + 1]) > int(c["cu_lens"][r]):
                c["state"][int(c["slots"][r])] = float("nan")
    out = nv.gdn_attention(**c, cached_lens=None if held is None else i32(held), scale=scale, **kw)
    check(c, out, before, want, what)
    return out


@pytest.mark.parametrize("k_heads,heads,dk,dv", [(1, 1, 64, 16), (2, 4, 128, 128), (1, 3, 64, 128),
                                                 (2, 2, 128, 64), (1, 2, 128, 48), (3, 6, 64, 272)])
@pytest.mark.parametrize("delta", [True, False])
def test_single_tokens(k_heads, heads, dk, dv, delta):
    _say("single", k_heads, heads, dk, dv, delta)
    rng = np.random.default_rng(heads * dk + dv)
    run(build(rng, [1] * 5, k_heads, heads, dk, dv, delta))


@pytest.mark.parametrize("lens", [[2], [3, 1, 8], [5, 0, 1, 7, 0], [0, 0, 4]])
@pytest.mark.parametrize("delta", [True, False])
def test_few_tokens(lens, delta):
    _say("few", lens, delta)
    rng = np.random.default_rng(sum(lens))
    run(build(rng, lens, 2, 4, 128, 64, delta))


LENS = [[63], [64], [65], [128], [129, 1, 64], [17, 200, 0, 31, 300], [9, 10, 16, 33]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 48)])
def test_prompts(lens, delta, dk, dv):
    _say("prompts", lens, delta, dk, dv)
    rng = np.random.default_rng(sum(lens) + dk)
    held = [int(rng.integers(0, 2)) for _ in lens]
    run(build(rng, lens, 1, 3, dk, dv, delta), held=held)


@pytest.mark.parametrize("decay", ["slow", "fast", "none", "mixed"])
@pytest.mark.parametrize("delta", [True, False])
def test_decays(decay, delta):
    """From gates that never forget to gates that underflow to zero."""
    _say("decay", decay, delta)
    rng = np.random.default_rng(7)
    run(build(rng, [150, 1, 70], 2, 4, 128, 64, delta, decay=decay))


@pytest.mark.parametrize("delta", [True, False])
def test_long_prompt(delta):
    _say("long", delta)
    rng = np.random.default_rng(11)
    run(build(rng, [2500], 1, 2, 128, 32, delta, decay="slow"), held=[0])


@pytest.mark.parametrize("lens", [[1, 1], [100, 3]])
def test_first_requests_do_not_read_their_slot(lens):
    rng = np.random.default_rng(5)
    run(build(rng, lens, 2, 2, 64, 64), held=[0, 1])
    run(build(rng, lens, 2, 2, 64, 64), held=[0, 0])


@pytest.mark.parametrize("lens", [[1, 1, 1], [90, 1, 30]])
def test_left_out_and_padding(lens):
    """Requests whose slot is out of range, and rows behind the last request,
    are neither read nor written."""
    rng = np.random.default_rng(6)
    c = build(rng, lens, 2, 4, 128, 64, pad=5)
    c["slots"][1] = -1
    out = torch.full_like(c["v"], 3.0)
    before = c["state"].clone()
    want = reference(dict(c, slots=c["slots"].clamp(min=0)))
    nv.gdn_attention(**c, out=out)
    cu = c["cu_lens"].tolist()
    assert bool((out[cu[1]:cu[2]] == 3).all()) and bool((out[cu[3]:] == 3).all())
    got, state = out.double().cpu().numpy(), c["state"].double().cpu().numpy()
    for r in (0, 2):
        compare(got[cu[r]:cu[r + 1]], state[int(c["slots"][r])], want[r], r)
    used = [int(c["slots"][r]) for r in (0, 2)]
    for i in range(len(state)):
        if i not in used:
            assert torch.equal(c["state"][i].isnan(), before[i].isnan()), i
    c["slots"][0] = len(state)
    again = torch.full_like(out, 3.0)
    nv.gdn_attention(**c, out=again)
    assert bool((again[:cu[1]] == 3).all())


@pytest.mark.parametrize("lens", [[1, 1], [3, 130]])
def test_strides(lens):
    """Slots inside a larger pool, strided outputs and gates, default slots."""
    rng = np.random.default_rng(8)
    c = build(rng, lens, 1, 2, 64, 32)
    n = len(lens)
    pool = torch.full((n + 2, 2 * 64 * 32 + 100), float("nan"), device=DEV)
    held = c["state"][c["slots"].long()].clone()
    view = pool[:, :2 * 64 * 32].view(n + 2, 2, 64, 32)
    view[:n] = held
    gates = torch.zeros(c["alpha"].shape[0], 9, device=DEV)
    gates[:, 1:3], gates[:, 4:6] = c["alpha"], c["beta"]
    out = torch.full((c["v"].shape[0], 3, 40), 9.0, dtype=BF16, device=DEV)
    c.update(state=view, slots=i32(list(range(n))), alpha=gates[:, 1:3], beta=gates[:, 4:6])
    want = reference(c)
    c2 = dict(c)
    del c2["slots"]
    nv.gdn_attention(**c2, out=out[:, :2, 4:36])
    cu = c["cu_lens"].tolist()
    for r in range(n):
        compare(out[cu[r]:cu[r + 1], :2, 4:36].double().cpu().numpy(),
                view[r].double().cpu().numpy(), want[r], r)
    out[:, :2, 4:36] = 9.0
    assert bool((out == 9).all())
    assert bool(pool[n:].isnan().all()) and bool(pool[:, 2 * 64 * 32:].isnan().all())


def test_chunks_continue_the_state():
    """A prompt in pieces of every kind equals the whole prompt, within the
    tolerances of the oracle's run."""
    rng = np.random.default_rng(12)
    c = build(rng, [333], 2, 4, 128, 64)
    want = reference(c, held=[0])
    whole = c["state"].clone()
    out, at = [], 0
    for piece in (100, 1, 64, 5, 1, 130, 32):
        part = {x: c[x][at:at + piece] for x in ("q", "k", "v", "alpha", "beta")}
        out.append(nv.gdn_attention(state=whole, cu_lens=i32([0, piece]), max_len=piece,
                                    slots=c["slots"], cached_lens=i32([at]),
                                    normalize=True, **part))
        at += piece
    assert at == 333
    compare(torch.cat(out).double().cpu().numpy(),
            whole[int(c["slots"][0])].double().cpu().numpy(), want[0], "pieces", True)


@pytest.mark.parametrize("lens", [[1] * 7, [70, 200, 1]])
def test_repeats_bit_for_bit(lens):
    rng = np.random.default_rng(13)
    c = build(rng, lens, 2, 4, 128, 128)
    first = c["state"].clone()
    out = nv.gdn_attention(**c)
    for _ in range(3):
        again = dict(c, state=first.clone())
        assert torch.equal(nv.gdn_attention(**again), out)
        assert torch.equal(again["state"][c["slots"].long()], c["state"][c["slots"].long()])


def test_scale_and_no_normalisation():
    rng = np.random.default_rng(14)
    for lens in ([1, 1], [80]):
        c = build(rng, lens, 1, 2, 64, 32)
        c["k"] = (c["k"].float() / 12).to(BF16)           # |k| < 1 without the division
        c["normalize"] = False
        run(c, scale=0.7)


@pytest.mark.parametrize("k_heads,heads,dk,dv", [(3, 3, 128, 16), (3, 3, 64, 32), (2, 4, 128, 80),
                                                 (2, 4, 64, 64), (1, 4, 64, 16), (2, 10, 128, 64),
                                                 (1, 8, 128, 32), (1, 9, 64, 48), (9, 9, 64, 64),
                                                 (1, 1, 128, 512), (2, 2, 64, 272)])
@pytest.mark.parametrize("delta", [True, False])
def test_heads_of_prompts(k_heads, heads, dk, dv, delta):
    _say("heads", k_heads, heads, dk, dv, delta)
    rng = np.random.default_rng(heads * dk + dv)
    run(build(rng, [90, 2, 64, 17], k_heads, heads, dk, dv, delta), held=[1, 1, 0, 1])


@pytest.mark.parametrize("every", [1, 97])
def test_many_requests(every):
    """Of 600 requests every one or some are long: the scan finds each of them."""
    rng = np.random.default_rng(every)
    lens = [int(rng.integers(17, 40)) if i % every == 0 else int(rng.integers(0, 3))
            for i in range(600)]
    run(build(rng, lens, 1, 1, 64, 16), held=[int(rng.integers(0, 2)) for _ in lens])


def test_more_units_than_workgroups():
    """Records and columns that a workgroup takes after its first ones."""
    rng = np.random.default_rng(21)
    lens = [100] * 36 + [3] * 4 + [20] * 20
    run(build(rng, lens, 8, 32, 64, 48))


@pytest.mark.parametrize("lens,max_len", [([40, 3, 70], 16), ([40, 3, 70], 0), ([40, 3, 200], 17)])
def test_longer_than_max_len(lens, max_len):
    """max_len chooses kernels only."""
    rng = np.random.default_rng(22)
    c = build(rng, lens, 1, 3, 64, 48)
    want, before = reference(c), c["state"].clone()
    out = nv.gdn_attention(**dict(c, max_len=max_len))
    cu, got, state = c["cu_lens"].tolist(), out.double().cpu().numpy(), c["state"].double().cpu().numpy()
    for r, ref in enumerate(want):
        compare(got[cu[r]:cu[r + 1]], state[int(c["slots"][r])], ref, (lens, max_len, r),
                chunked=None if max_len > 16 else False)


@pytest.mark.parametrize("pad", [0, 3])
def test_no_tokens(pad):
    rng = np.random.default_rng(23)
    c = build(rng, [0, 0], 1, 2, 64, 32, pad=pad)
    before = c["state"].clone()
    out = torch.full((pad, 2, 32), 5.0, dtype=BF16, device=DEV)
    for max_len in (0, 1, 100):
        nv.gdn_attention(**dict(c, max_len=max_len), out=out)
        assert bool((out == 5).all())
        assert torch.equal(c["state"].view(torch.int32), before.view(torch.int32))


@pytest.mark.parametrize("lens", [[1, 1, 1], [60, 70, 100]])
def test_what_is_not_finite_stays_with_its_request(lens):
    """NaN and infinities of one request's inputs leave the others alone."""
    rng = np.random.default_rng(24)
    c = build(rng, lens, 2, 4, 128, 64)
    clean = dict(c, state=c["state"].clone())
    want = nv.gdn_attention(**clean)
    lo, hi = int(c["cu_lens"][1]), int(c["cu_lens"][2])
    bad = dict(c, **{x: c[x].clone() for x in ("q", "k", "v", "alpha", "beta")})
    bad["q"][lo:hi], bad["k"][hi - 1] = float("inf"), float("nan")
    bad["v"][lo], bad["alpha"][lo:hi, 1], bad["beta"][lo] = float("-inf"), float("nan"), float("nan")
    out = nv.gdn_attention(**bad)
    assert bool(out[lo:hi].isnan().any())
    for rows in (slice(0, lo), slice(hi, None)):
        assert torch.equal(out[rows], want[rows])
    for r in (0, 2):
        s = int(c["slots"][r])
        assert torch.equal(bad["state"][s], clean["state"][s])
