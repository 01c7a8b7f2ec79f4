"""The gated delta rule and the gated norm in fp64 on the CPU, from their definitions, and the
inputs that their GPU tests share (imported by tests only)."""
from __future__ import annotations

import numpy as np

K = 128


def delta_ref(cu, slot, q, k, v, a, beta, S, normalize=False, scale=1.0):
    """Token by token in fp64.  q, k [N][Hqk][K], v [N][H][V], a, beta [N][H], S [B][H][K][V];
    returns (y, S, touched) with y zero where no sequence lies."""
    q, k, v, a, beta = (np.asarray(x, np.float64) for x in (q, k, v, a, beta))
    S = np.array(S, np.float64)
    r = v.shape[1] // q.shape[1]
    if normalize:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    q, k = np.repeat(q * scale, r, 1), np.repeat(k, r, 1)
    y, touched = np.zeros(v.shape), np.zeros(v.shape[0], bool)
    for i, s in enumerate(slot):
        if s < 0:
            continue
        for t in range(cu[i], cu[i + 1]):
            M = S[s]
            u = beta[t][:, None] * (v[t] - a[t][:, None] * np.einsum("hkv,hk->hv", M, k[t]))
            S[s] = a[t][:, None, None] * M + k[t][..., None] * u[:, None, :]
            y[t] = np.einsum("hkv,hk->hv", S[s], q[t])
            touched[t] = True
    return y, S, touched


def draw(seed, n, B, H, Hqk, V, unit=True):
    """fp32 inputs: unit (or standard normal) q and k, values N(0, 1), decays near 1, states 0.1 N(0, 1)."""
    g = np.random.default_rng(seed)
    q, k = (g.standard_normal((n, Hqk, K)) for _ in range(2))
    if unit:
        q, k = q / np.linalg.norm(q, axis=-1, keepdims=True), k / np.linalg.norm(k, axis=-1, keepdims=True)
    v = g.standard_normal((n, H, V))
    a = np.exp(-0.05 * np.log1p(np.exp(g.standard_normal((n, H)))))
    beta = 1 / (1 + np.exp(-g.standard_normal((n, H))))
    S = 0.1 * g.standard_normal((B, H, K, V))
    return {x: y.astype(np.float32) for x, y in dict(q=q, k=k, v=v, a=a, beta=beta, S=S).items()}


def state_tol(longest):
    """Bound of the state's error relative to the largest column norm of the states.

    A token's u comes from a product of length 128 of the state: summed in fp32 (at most 24
    roundings on any term's way, or splits of 2^-22 per factor) that is off by at most
    24 * 2^-24 |k| |S_column| with |k| <= 1.  The step a (I - beta k k^T) shrinks what is off
    already, with a geometric sum of at most about 1 / (1 - a) tokens for the decays of draw()
    (mean a = 0.96); so after n tokens it is at most min(n + 1, 64) such errors."""
    return 24 * 2.0 ** -24 * min(longest + 1, 64)


def norm_ref(x, z, w, eps, activation, gate_first):
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    act = 1.0
    if z is not None:
        z = np.asarray(z, np.float64)
        act = 1 / (1 + np.exp(-z))
        if activation == "silu":
            act = act * z
    u = x * act if gate_first else x
    u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * w
    return u if gate_first else u * act
