"""Linear attention with a decay per head, in float64, token after token.
TEST INFRASTRUCTURE ONLY (see oracle/__init__.py for the page key).

The recurrence of a Gated DeltaNet layer ([P3] 前提2): the state forgets by
alpha, the delta rule writes beta times what the value differs from what the
state holds for the key; without beta the value itself is written.
"""
import numpy as np


def gdn(q, k, v, alpha, beta, state, scale, normalize=False):
    """One request: q, k [tokens, k_heads, dk], v [tokens, heads, dv], alpha and
    beta [tokens, heads] (beta None: plain rule), state [heads, dk, dv].

    Returns (o, S, size, reach): outputs, the last state, and what bounds their
    roundings, each a sum of norms without cancellation.  Per head and column,
    n_t = alpha n_{t-1} + |k_t| |u_t| bounds the state's column norm, w_t =
    alpha w_{t-1} + n_t + |k_t| |beta v_t| sums what every step rounds; size =
    scale |q_t| n_t [tokens, heads, dv], reach = (scale |q_t| w_t, the last w,
    the last n)."""
    q, k, v, alpha, S = (np.array(t, dtype=np.float64) for t in (q, k, v, alpha, state))
    tokens, heads, dv = v.shape
    group = heads // k.shape[1]
    if normalize:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    o, size, reach = np.zeros(v.shape), np.zeros(v.shape), np.zeros(v.shape)
    n = np.sqrt((S * S).sum(1))
    w = n.copy()
    for t in range(tokens):
        kt, qt = np.repeat(k[t], group, 0), np.repeat(q[t], group, 0)
        a = alpha[t][:, None]
        S *= a[:, :, None]
        u = v[t].copy()
        wrote = np.abs(u)
        if beta is not None:
            b = np.asarray(beta[t], dtype=np.float64)[:, None]
            wrote = np.abs(b * u)
            u = b * (u - (kt[:, None, :] @ S)[:, 0])
        S += kt[:, :, None] * u[:, None, :]
        o[t] = scale * (qt[:, None, :] @ S)[:, 0]
        kn, qn = (np.sqrt((x * x).sum(-1))[:, None] for x in (kt, qt))
        n = a * n + kn * np.abs(u)
        w = a * w + n + kn * wrote
        size[t], reach[t] = scale * qn * n, scale * qn * w
    return o, S, size, (reach, w, n)
