"""The scan of gdn_attention over many chunks, against itself and the oracle.

A prompt cut at multiples of the 64 tokens of a chunk has the same chunks as the
whole, and the state passes between calls in binary32, so a call over the whole
prompt has to give the bits that calls of one chunk each give.  Those hold
nothing in LDS from one chunk to the next: a read that a later chunk's load
overtakes, a buffer taken for another's or a decay of the wrong chunk shows as a
difference.
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import test_gpu_gdn as gdn

pytestmark = pytest.mark.gpu


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
