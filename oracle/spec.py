"""fp64 CPU oracle for speculative decoding on the recurrent state: tree decode,
draft verification, state advance and the packed state pool. TEST
INFRASTRUCTURE (same rules as the rest of ``oracle``).

Every function is a definition written out token by token. The tree and advance
functions also return a *scale* per value: the sum of the magnitudes of the
terms that the value is a sum of (for the delta rule, with the terms of the
increments it rests on). A computation whose every product, sum and rounding is
off by a relative g is then off by at most about g times that scale.
"""

import numpy as np

from .la_oracle import _as64, phi_elu1


def path_of(parent, i):
    """The nodes from the top down to i, by one tree's parents (values that are
    not an earlier node: a child of the committed state)."""
    path = []
    while i >= 0:
        path.append(i)
        p = int(parent[i])
        i = p if 0 <= p < i else -1
    return path[::-1]


def decode_tree(S, z, q, k, v, parent, alpha=None, count=None, eps=1e-6):
    """Every node's output: the recurrence along its own path. S [B,H,dk,dv],
    z [B,H,dk], q, k [B,H,T,dk], v [B,H,T,dv], parent [B,T], alpha [H], count
    [B]. Returns (out, scale); rows behind a tree's last node are NaN in both."""
    S, z, q, k, v = _as64(S, z, q, k, v)
    B, H, T, _ = q.shape
    a = np.ones(H) if alpha is None else np.asarray(alpha, np.float64)
    out = np.full(v.shape, np.nan)
    scale = np.full(v.shape, np.nan)
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        for i in range(n):
            Si, zi, Ai = S[b], z[b], np.abs(S[b])
            for j in path_of(parent[b], i):
                f = phi_elu1(k[b, :, j])
                Si = a[:, None, None] * Si + f[:, :, None] * v[b, :, j, None, :]
                Ai = np.abs(a)[:, None, None] * Ai + f[:, :, None] * np.abs(v[b, :, j, None, :])
                zi = a[:, None] * zi + f
            f = phi_elu1(q[b, :, i])
            den = np.einsum("hk,hk->h", f, zi) + eps
            out[b, :, i] = np.einsum("hk,hkv->hv", f, Si) / den[:, None]
            scale[b, :, i] = np.einsum("hk,hkv->hv", f, Ai) / np.abs(den)[:, None]
    return out, scale


def decode_tree_delta(S, q, k, v, parent, count=None):
    """The delta rule along every node's path; returns (out, scale)."""
    S, q, k, v = _as64(S, q, k, v)
    B, H, T, _ = q.shape
    out = np.full(v.shape, np.nan)
    scale = np.full(v.shape, np.nan)
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        for i in range(n):
            Si, Ai = S[b], np.abs(S[b])
            for j in path_of(parent[b], i):
                kj = k[b, :, j]
                u = v[b, :, j] - np.einsum("hkv,hk->hv", Si, kj)
                au = np.abs(v[b, :, j]) + np.einsum("hkv,hk->hv", Ai, np.abs(kj))
                Si = Si + kj[:, :, None] * u[:, None, :]
                Ai = Ai + np.abs(kj)[:, :, None] * au[:, None, :]
            out[b, :, i] = np.einsum("hkv,hk->hv", Si, q[b, :, i])
            scale[b, :, i] = np.einsum("hkv,hk->hv", Ai, np.abs(q[b, :, i]))
    return out, scale


def advance(S, z, k, v, path=None, accepted=None, alpha=None):
    """State after each sequence's accepted rows; returns (S, z, scale of S)."""
    S, z, k, v = (x.copy() for x in _as64(S, z, k, v))
    A = np.abs(S)
    B, H, T, _ = k.shape
    a = np.ones(H) if alpha is None else np.asarray(alpha, np.float64)
    for b in range(B):
        for j in _rows(path, accepted, b, T):
            f = phi_elu1(k[b, :, j])
            S[b] = a[:, None, None] * S[b] + f[:, :, None] * v[b, :, j, None, :]
            A[b] = np.abs(a)[:, None, None] * A[b] + f[:, :, None] * np.abs(v[b, :, j, None, :])
            z[b] = a[:, None] * z[b] + f
    return S, z, A


def advance_delta(S, k, v, path=None, accepted=None):
    """State after each sequence's accepted rows by the delta rule; (S, scale)."""
    S, k, v = (x.copy() for x in _as64(S, k, v))
    A = np.abs(S)
    B, _, T, _ = k.shape
    for b in range(B):
        for j in _rows(path, accepted, b, T):
            kj = k[b, :, j]
            u = v[b, :, j] - np.einsum("hkv,hk->hv", S[b], kj)
            au = np.abs(v[b, :, j]) + np.einsum("hkv,hk->hv", A[b], np.abs(kj))
            S[b] = S[b] + kj[:, :, None] * u[:, None, :]
            A[b] = A[b] + np.abs(kj)[:, :, None] * au[:, None, :]
    return S, A


def _rows(path, accepted, b, T):
    n = T if accepted is None else min(max(int(accepted[b]), 0), T)
    rows = []
    for t in range(n):
        j = t if path is None else int(path[b][t])
        if j < 0 or j >= T:
            break
        rows.append(j)
    return rows


def draw(w, u):
    """The smallest t with w_0 + .. + w_t > u * (all of them); weights that are
    not above zero are zero. -1 where none is positive."""
    w = np.asarray(w, np.float64)
    w = np.where(w > 0, w, 0.0)
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    past = np.nonzero(c > np.float64(u) * c[-1])[0]
    return int(past[0]) if past.size else int(np.nonzero(w)[0][-1])


def verify_chain(target, draft, tokens, uniform, count=None):
    """(accepted [B], next [B]) of drafted chains."""
    target, draft, uniform = _as64(target, draft, uniform)
    B, T = target.shape[0], target.shape[1] - 1
    V = target.shape[2]
    accepted, nxt = np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        all_ = T if count is None else min(max(int(count[b]), 0), T)
        n = 0
        while n < all_:
            x = int(tokens[b][n])
            if not (0 <= x < V and uniform[b, n] * draft[b, n, x] < target[b, n, x]):
                break
            n += 1
        w = target[b, n]
        if n < all_:
            with np.errstate(invalid="ignore"):
                d = w - draft[b, n]
            if np.any(d > 0):
                w = d
        accepted[b], nxt[b] = n, draw(w, uniform[b, T])
    return accepted, nxt


def verify_tree(target, tokens, parent, uniform, count=None):
    """(path [B,T], accepted [B], next [B]) of drafted trees."""
    target, uniform = _as64(target, uniform)
    B, T = target.shape[0], target.shape[1] - 1
    path, accepted, nxt = np.full((B, T), -1), np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        all_ = T if count is None else min(max(int(count[b]), 0), T)
        par = [int(p) if 0 <= int(p) < i else -1 for i, p in enumerate(parent[b][:all_])]
        at, n = -1, 0
        while True:
            x = draw(target[b, at + 1], uniform[b, at + 1])
            hit = [i for i in range(all_) if par[i] == at and int(tokens[b][i]) == x and x >= 0]
            if not hit:
                break
            at = hit[0]
            path[b, n] = at
            n += 1
        accepted[b], nxt[b] = n, x
    return path, accepted, nxt


# The 127 finite non-negative e4m3 values, in code order (code 127: NaN).
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]


def to_e4m3(y):
    """Codes of the nearest e4m3 values (ties to the even code, infinities and
    everything beyond to the largest), NaN to 0x7f."""
    y = np.asarray(y, np.float64)
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(E4M3[hi] - a), np.abs(a - E4M3[lo])
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(a >= E4M3[126], 126, pick)
    return np.where(np.isnan(y), 0x7f, pick | (np.signbit(y) * 128)).astype(np.uint8)


def pack(S):
    """(codes like S, scales [..., dv / min(32, dv)]) uint8 of fp32 states."""
    S = np.asarray(S, np.float32).astype(np.float64)
    w = min(32, S.shape[-1])
    x = S.reshape(S.shape[:-1] + (-1, w))
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -127)
    while np.any(top > 448.0 * 2.0 ** e):
        e = np.where(top > 448.0 * 2.0 ** e, e + 1, e)
    y = x / 2.0 ** e[..., None]
    # 256 * 2^120 is beyond fp32: blocks with that scale stop at 240
    y = np.where((e[..., None] == 120) & (np.abs(y) > 240), np.copysign(240.0, y), y)
    return to_e4m3(y).reshape(S.shape), (e + 127).astype(np.uint8)


def unpack(codes, scales):
    """fp32 states of codes and scales."""
    codes = np.asarray(codes)
    m = codes & 127
    x = np.where(m == 127, np.nan, np.append(E4M3, 0.0)[m]) * np.where(codes >= 128, -1.0, 1.0)
    w = codes.shape[-1] // scales.shape[-1]
    return (x * np.repeat(2.0 ** (scales.astype(np.float64) - 127), w, axis=-1)).astype(np.float32)
