"""gdn_attention on each of its paths, at the borders between them, against the
oracle (tolerances: test_gpu_gdn.py) or exactly.

Whether a call goes token after token or in chunks is the library's choice; the
tests take the border from it (a call in chunks wants a workspace).
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle
import test_gpu_gdn as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[gpu-gdn-paths]", *a, flush=True)


def in_chunks(max_len):
    return nv.library().gdn_attention_workspace(max_len, 1, 1, 64, 16, 1, max_len, 1) > 0


def few():
    """The longest max_len that goes token after token."""
    return next(n for n in range(1, 4096) if not in_chunks(n) and in_chunks(n + 1))


def run(c, max_len, held=None, what=""):
    """A call with this max_len; each request held to the tolerance of its path."""
    want, before = gdn.reference(c, held), c["state"].clone()
    if held is not None:
        for r, h in enumerate(held):
            if h <= 0 and int(c["cu_lens"][r + 1]) > int(c["cu_lens"][r]):
                c["state"][int(c["slots"][r])] = float("nan")
    out = nv.gdn_attention(**dict(c, max_len=max_len), cached_lens=None if held is None else
                           gdn.i32(held))
    cu, got = c["cu_lens"].tolist(), out.double().cpu().numpy()
    state = c["state"].double().cpu().numpy()
    for r, ref in enumerate(want):
        s, n = int(c["slots"][r]), cu[r + 1] - cu[r]
        if n == 0:
            assert torch.equal(c["state"][s].view(torch.int32), before[s].view(torch.int32))
        else:
            gdn.compare(got[cu[r]:cu[r + 1]], state[s], ref, (what, r),
                        chunked=in_chunks(max_len) and n > few())


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("over", [0, 1])
def test_border_of_chunks(delta, over):
    """Requests of the last length token after token, the first in chunks, and
    longer than max_len on either path."""
    n = few()
    _say("border", n, delta, over)
    lens = [n, n + 1, n - 1, 200, 64, n, 1, 129]
    c = gdn.build(np.random.default_rng(over), lens, 2, 4, 64, 48, delta)
    run(c, n + over, held=[1, 0, 0, 1, 1, 1, 0, 1])


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 48), (64, 64), (64, 272)])
@pytest.mark.parametrize("length", [1, 20])
@pytest.mark.parametrize("delta", [True, False])
def test_many_states(dk, dv, length, delta):
    """Decodes and drafts whose states fill the card (wide waves), ragged."""
    _say("many", dk, dv, length, delta)
    assert not in_chunks(length)
    rng = np.random.default_rng(dk + dv + length)
    lens = [length] + [int(rng.integers(0, length + 1)) for _ in range(31)]
    c = gdn.build(rng, lens, 4, 16, dk, dv, delta)
    run(c, length, held=[int(rng.integers(0, 2)) for _ in lens])


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("k_heads,heads,dk,dv", [(1, 2, 128, 32), (1, 1, 64, 64)])
def test_more_chunks_than_lanes(delta, k_heads, heads, dk, dv):
    """A request of 130 chunks and a rest, whose decays differ from chunk to chunk:
    the oracle's, and the bits of calls of one chunk each."""
    _say("chunks", delta, dk, dv)
    tokens = 130 * 64 + 41
    rng = np.random.default_rng(dk)
    c = gdn.build(rng, [tokens], k_heads, heads, dk, dv, delta)
    rate = np.exp(rng.uniform(np.log(1e-5), np.log(0.2), (tokens // 64 + 1, heads)))
    c["alpha"].copy_(torch.from_numpy(np.exp(-np.repeat(rate, 64, 0)[:tokens])))
    alone, s = c["state"].clone(), int(c["slots"][0])
    out = []
    for at in range(0, tokens, 64):
        part = {x: None if c[x] is None else c[x][at:at + 64] for x in
                ("q", "k", "v", "alpha", "beta")}
        n = part["q"].shape[0]
        out.append(nv.gdn_attention(state=alone, cu_lens=gdn.i32([0, n]), max_len=64,
                                    slots=c["slots"], normalize=c["normalize"], **part))
    state = c["state"].clone()
    assert torch.equal(nv.gdn_attention(**dict(c, state=state)), torch.cat(out))
    assert torch.equal(state[s], alone[s])
    run(c, tokens, what="oracle")


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("dk,dv,group", [(128, 48, 3), (128, 64, 4), (128, 32, 1), (128, 48, 2),
                                         (64, 80, 4)])
def test_more_work_than_workgroups(dk, dv, group, delta):
    """Units of the preparation and items of the scan that a workgroup takes after its
    first ones, next to requests of few tokens."""
    _say("work", dk, dv, group, delta)
    lens = [21, 22, 40, 66, 2] * 14
    k_heads = 8
    c = gdn.build(np.random.default_rng(dk + group), lens, k_heads, k_heads * group, dk, dv, delta)
    # preparation: 512 workgroups; scan: 256, of 32 columns each
    long = [n for n in lens if n > 20]
    assert sum(-(-n // 64) for n in long) * k_heads > 512 or group < 3
    assert len(long) * k_heads * group * -(-dv // 32) > 256
    run(c, max(lens))


@pytest.mark.parametrize("i,j", [(0, 1), (3, 40), (10, 30), (17, 63), (31, 32), (47, 49)])
@pytest.mark.parametrize("dk", [64, 128])
def test_state_keeps_24_bits_within_a_chunk(i, j, dk):
    """Two tokens with one key, everything else without effect: the state's row is
    s + u_i + u_j, u_i = b_i (v_i - s), u_j = b_j (v_j - s - u_i).  All numbers are
    multiples of 2^-21 below 4, so binary32 holds them and the result is exact, if the
    operands' parts are: s takes two bf16 numbers, v - s three, b_i b_j two (the products
    of both of its parts with all three), u three into the state."""
    _say("bits", i, j, dk)
    tokens, heads, dv = 64, 3, 128
    rng = np.random.default_rng(i + j)
    k = torch.zeros(tokens, 1, dk)
    k[[i, j], 0, 5] = 1
    beta = torch.zeros(tokens, heads)
    beta[i], beta[j] = torch.tensor([1, 1 + 2.0 ** -9, 0.5 + 2.0 ** -9]), torch.tensor([0.5, 0.5, 1])
    v = torch.from_numpy(rng.integers(-128, 129, (tokens, heads, dv)) / 128)
    s = np.zeros((heads, dv))
    # two bf16 numbers, of multiples of 2^-11 and of 2^-20, which v - s takes three for;
    # multiples of 2^-10 under a gate of two
    s[0] = rng.integers(64, 128, dv) / 2.0 ** 11 + rng.integers(-127, 128, dv) / 2.0 ** 20
    s[1:] = rng.integers(-1024, 1025, (2, dv)) / 2.0 ** 10
    state = torch.zeros(1, heads, dk, dv)
    state[0, :, 5] = torch.from_numpy(s)
    assert torch.equal(state[0, :, 5].double(), torch.from_numpy(s))
    c = dict(q=k, k=k, v=v, alpha=torch.ones(tokens, heads), beta=beta)
    want = oracle.gdn(*(c[x].double().numpy() for x in ("q", "k", "v", "alpha", "beta")),
                      state[0].double().numpy(), 1.0)[1]
    assert np.array_equal(want, want.astype(np.float32))
    c = {x: t.to(F32 if x in ("alpha", "beta") else BF16).to(DEV) for x, t in c.items()}
    got = state.to(DEV)
    nv.gdn_attention(**c, state=got, cu_lens=gdn.i32([0, tokens]), max_len=tokens, scale=1.0)
    assert np.array_equal(got[0].double().cpu().numpy(), want)


@pytest.mark.parametrize("which", ["q", "k", "v", "alpha", "beta"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_what_is_not_finite_stays_behind_its_chunk(which, value):
    """A non-finite input of one token: token after token, earlier rows stay; in
    chunks, those of earlier chunks (a query's reaches its own row only)."""
    _say("finite", which, value)
    n, at = 200, 150
    c = gdn.build(np.random.default_rng(3), [n], 2, 4, 128, 64)
    clean, first = nv.gdn_attention(**dict(c, state=c["state"].clone())), c["state"].clone()
    bad = dict(c, state=first.clone())
    bad[which] = c[which].clone()
    bad[which][at, 1] = float(value)
    out = nv.gdn_attention(**bad)
    assert torch.equal(out[:at // 64 * 64], clean[:at // 64 * 64])
    if which == "q":
        others = [t for t in range(n) if t != at]
        assert torch.equal(out[others], clean[others])
        assert torch.equal(bad["state"][int(c["slots"][0])], nv_state(c))
    else:
        assert not bool(out[at:].isfinite().all())
    # the same tokens before it in calls of few tokens
    m = few()
    head = {x: c[x][:m] for x in ("q", "k", "v", "alpha", "beta")}
    tail = dict(head, **{which: head[which].clone()})
    tail[which][m - 3, 1] = float(value)
    outs = [nv.gdn_attention(state=first.clone(), cu_lens=gdn.i32([0, m]), max_len=m,
                             slots=c["slots"], normalize=True, **x) for x in (head, tail)]
    assert torch.equal(outs[0][:m - 3], outs[1][:m - 3])


def nv_state(c):
    state = c["state"].clone()
    nv.gdn_attention(**dict(c, state=state))
    return state[int(c["slots"][0])]
