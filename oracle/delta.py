"""fp64 oracle of the gated delta rule, token by token (test infrastructure only)."""

from __future__ import annotations

import numpy as np


def run(S, q, k, v, g, beta, scale: float):
    """S [Hv, dk, dv]; q, k [n, Hk, dk]; v [n, Hv, dv]; g, beta [n, Hv], all fp64.  Returns outputs [n, Hv, dv], the new
    state, and for tolerances the sums |S| |q| scale."""
    S = S.copy()
    rep = S.shape[0] // q.shape[1]
    out, mag = np.zeros_like(v), np.zeros_like(v)
    for t in range(q.shape[0]):
        for h in range(S.shape[0]):
            kt, qt = k[t, h // rep], q[t, h // rep]
            S[h] *= np.exp(g[t, h])
            S[h] += np.outer(kt, beta[t, h] * (v[t, h] - S[h].T @ kt))
            out[t, h] = scale * (S[h].T @ qt)
            mag[t, h] = scale * (np.abs(S[h]).T @ np.abs(qt))
    return out, S, mag
