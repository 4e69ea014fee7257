"""The scan of gdn_attention over many chunks, against itself and the oracle.

A prompt cut at multiples of the 64 tokens of a chunk has the same chunks as the
whole, and the state passes between calls in binary32, so a call over the whole
prompt has to give the bits that calls of one chunk each give.  Those hold
nothing in LDS from one chunk to the next: a read that a later chunk's load
overtakes, a buffer taken for another's or a decay of the wrong chunk shows as a
difference.

Outputs in chunks take no binary32 operand as one bf16 number.  Two numbers leave
(2^-8)^2 = 2^-16 of an operand at most; with d what an output is off before its own
rounding to bf16, size = scale |q| n and n the oracle's bound on the state's column
(its docstring):

  the state in Q S    2^-16 scale |q| |S|           the scores P    2^-16 sum |P| |U|
    (together 2^-16 size, since n bounds alpha |S| + sum |k| |u|)
  U, and the product of both second parts, each 2^-16 sum |P| |U| <= 2^-16 size
  what U itself is off: the state in K S, T, and the product of R's and T's second
    parts: 3 2^-16 n
  binary32 sums       128 2^-24 size at most, half of 2^-16

  |d| <= 6.5 2^-16 size < 2^-13 size.

The nearest bf16 number to o + d is no farther from o than half a step of o and |d|.
Of either sign from element to element, errors of six sources add by their squares,
and a sum of dk of them against a query of any direction is 1 / sqrt(dk) of the norms'
product: in the 2-norm sqrt(6.5) 2^-16 size / sqrt(dk).  With r what rounding the exact
outputs leaves, |got - o| <= |r| + 2 |d| for each (got is nearer to o + d than bf16(o)
is), which the 2-norm keeps.
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import test_gpu_gdn as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[gpu-gdn-scan]", *a, flush=True)


def in_pieces(c, state, piece):
    """Outputs of one request taken `piece` tokens a call; state is updated."""
    tokens, out = c["q"].shape[0], []
    for at in range(0, tokens, piece):
        n = min(piece, tokens - at)
        part = {x: None if c[x] is None else c[x][at:at + n] for x in
                ("q", "k", "v", "alpha", "beta")}
        out.append(nv.gdn_attention(state=state, cu_lens=gdn.i32([0, n]), max_len=64,
                                    slots=c["slots"], normalize=c["normalize"], **part))
    return torch.cat(out)


@pytest.mark.parametrize("k_heads,heads,dk,dv", [(1, 2, 128, 64), (2, 2, 64, 48), (1, 5, 128, 128),
                                                 (4, 64, 128, 128)])
@pytest.mark.parametrize("delta", [True, False])
def test_chunks_alone(k_heads, heads, dk, dv, delta):
    """30 chunks and a rest at once and one by one."""
    _say("alone", k_heads, heads, dk, dv, delta)
    c = gdn.build(np.random.default_rng(heads * dk + dv), [30 * 64 + 37], k_heads, heads, dk, dv,
                  delta, decay="slow")
    c["normalize"] = True
    alone = c["state"].clone()
    want = in_pieces(c, alone, 64)
    for _ in range(5):
        state = c["state"].clone()
        assert torch.equal(nv.gdn_attention(**dict(c, state=state)), want)
        s = int(c["slots"][0])
        assert torch.equal(state[s], alone[s])


def half_step(o):
    """Half the distance of bf16 numbers at o."""
    return np.ldexp(1.0, np.frexp(o)[1] - 1 - 8)


@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 48)])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("decay", ["fast", "mixed"])
def test_outputs_round_once(dk, dv, delta, decay):
    _say("round", dk, dv, delta, decay)
    c = gdn.build(np.random.default_rng(dk), [8 * 64, 29, 1, 70], 2, 4, dk, dv, delta, decay=decay)
    c["normalize"] = True
    want = gdn.reference(c)
    got, cu = nv.gdn_attention(**c).double().cpu().numpy(), c["cu_lens"].tolist()
    for r, (o, _, size, *_) in enumerate(want):
        off = got[cu[r]:cu[r + 1]] - o
        assert (np.abs(off) <= half_step(o) + 2.0 ** -13 * size).all(), r
        once = np.linalg.norm(torch.from_numpy(o).to(BF16).double().numpy() - o)
        assert np.linalg.norm(off) <= once + 2 * 6.5 ** 0.5 * 2.0 ** -16 * np.linalg.norm(size) / dk ** 0.5, r


@pytest.mark.parametrize("which", ["state", "scores"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("delta", [True, False])
def test_operands_between_bf16_numbers(which, dk, delta):
    """States, or scores, all a little less than half a step from the bf16 number
    below: as one number each, outputs would be off by 2^-8 of themselves besides
    their own rounding.  The scales put the outputs over a whole step."""
    _say("between", which, dk, delta)
    tokens, dv, x = 64, 16, 1 + 2.0 ** -8 - 2.0 ** -20
    keys, gates = torch.zeros(tokens, 1, dk, dtype=BF16, device=DEV), torch.ones(tokens, 1, device=DEV)
    for step in range(16):
        if which == "state":
            # nothing is written: the outputs are scale dk x
            state, scale = torch.full((1, 1, dk, dv), x, device=DEV), (1 + step * 2.0 ** -11) * 1.5 / dk
            q, k, v = keys + 1, keys, torch.zeros(tokens, 1, dv, dtype=BF16, device=DEV)
            alpha, beta = gates, 0 * gates
        else:
            # nothing is kept, keys and queries of one element: the outputs are x v
            state, scale = torch.zeros(1, 1, dk, dv, device=DEV), x
            q = k = torch.eye(tokens, dk, dtype=BF16, device=DEV)[:, None]
            v = torch.full((tokens, 1, dv), 1 + step * 2.0 ** -4, dtype=BF16, device=DEV)
            alpha, beta = 0 * gates, gates
        c = dict(q=q, k=k, v=v, alpha=alpha, beta=beta if delta else None, state=state,
                 cu_lens=gdn.i32([0, tokens]), slots=gdn.i32([0]), normalize=False)
        scale = float(np.float32(scale))
        (o, _, size, *_), = gdn.reference(c, scale=scale)
        got = nv.gdn_attention(max_len=tokens, scale=scale, **c).double().cpu().numpy()
        off = np.abs(got - o)
        assert (off <= half_step(o) + 2.0 ** -13 * size).all(), (step, off.max(), o[0, 0, 0])
