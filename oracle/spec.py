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


def decode_tree_delta_bound(S, q, k, v, parent, count=None, parts=False):
    """How far a delta-rule tree decode may be off before its result is rounded,
    [B,H,T,dv]. Where ``scale`` of decode_tree_delta adds up magnitudes along a
    path and grows with every token, this takes the increments themselves:

    With A_jl = k_j.k_l and W_ij = q_i.k_j along the paths, M = (I + A)^-1 and
    R = v - S^T k, the increments are U = M R and out = S^T q + W U. If U_hat
    solves (I + A) U_hat = R + rho, it is off by at most |M| |rho|. Let u = 2^-24.

    parts=False: fp32 throughout. A sum of m products is off by (m + 4) u of its
    terms' magnitudes, so that rho has (dk + 4) u |S|^T |k|, 2 u (|v| + |S|^T |k|)
    for the difference, (dk + 4) u |k_j|.|k_l| |U_l| for the key products and
    (T + 4) u |A| |U| for the substitution.

    parts=True: fp32 operands as two bf16 parts, x = hi + lo up to 2^-17 of x, and
    products of two of them without lo lo: up to 2^-15 of the term. A sum of m
    terms on the tensor cores is off by 4 m u: three products a term and sums
    that truncate. The solve goes block by block of 16 nodes, U_b = X_b R'_b with
    X_b the inverse of the block's own triangle L_b (the same block of M) and R'_b
    = L_b U_b what the earlier blocks leave, so that an error of the product with
    X_b counts as L_b times it in rho; X_b itself, by substitution, is off by
    32 u |X| |L| |X| and by its triangle's errors.

    Errors of second order are allowed for by 5 %."""
    S, q, k, v = _as64(S, q, k, v)
    B, H, T, dk = q.shape
    bound = np.full(v.shape, np.nan)
    u = 2.0 ** -24
    split, pair = (2.0 ** -17, 2.0 ** -15) if parts else (0.0, 0.0)
    acc = (lambda m: 4 * m * u) if parts else (lambda m: (m + 4) * u)
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        on = np.zeros((n, n), bool)
        for i in range(n):
            on[i, path_of(parent[b], i)] = True
        below = on & ~np.eye(n, dtype=bool)
        block = np.arange(n) // 16
        same = block[:, None] == block[None]
        for h in range(H):
            S_, q_, k_, v_ = S[b, h], q[b, h, :n], k[b, h, :n], v[b, h, :n]
            A, W = np.where(below, k_ @ k_.T, 0.0), np.where(on, q_ @ k_.T, 0.0)
            kk, qk = np.where(below, np.abs(k_) @ np.abs(k_).T, 0.0), np.where(on, np.abs(q_) @ np.abs(k_).T, 0.0)
            M = np.linalg.inv(np.eye(n) + A)
            U = M @ (v_ - k_ @ S_)
            aU, read = np.abs(U), np.abs(k_) @ np.abs(S_)
            rho = (split + acc(dk)) * read + 2 * u * (np.abs(v_) + read)
            if parts:
                L, X = np.eye(n) + np.where(same, A, 0.0), np.abs(np.where(same, M, 0.0))
                rho += (pair + acc(64)) * np.where(same, 0.0, np.abs(A)) @ aU + acc(dk) * np.where(same, 0.0, kk) @ aU
                XR = X @ np.abs(L @ U)
                own = (pair + acc(48)) * XR + X @ (acc(dk) * np.where(same, kk, 0.0) + 32 * u * np.abs(L)) @ XR
                rho += np.abs(L) @ own
            else:
                rho += acc(T) * np.abs(A) @ aU + acc(dk) * kk @ aU
            off = (split + acc(dk)) * (np.abs(q_) @ np.abs(S_)) + acc(dk) * qk @ aU + (pair + acc(64)) * np.abs(W) @ aU
            bound[b, h, :n] = 1.05 * (off + np.abs(W) @ (np.abs(M) @ rho))
    return bound


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


def advance_delta_bound(S, k, v, path=None, accepted=None):
    """How far an fp32 state advance by the delta rule may be off, like S. A step
    takes an error E of the state to (I - k k^T) E, whose columns grow by at most
    max(1, | |k|^2 - 1 |) in the 2-norm, and adds its own: (dk + 4) u of |S|^T |k| in
    u = S^T k and 2 u of |v| + |S|^T |k| in v - u, times |k|, and u of the new state
    (u = 2^-24). Every value of a column is off by at most the column's norm; 5 %
    for errors of second order."""
    S, k, v = (x.copy() for x in _as64(S, k, v))
    B, _, T, dk = k.shape
    u, err = 2.0 ** -24, np.zeros((S.shape[0], S.shape[1], S.shape[3]))
    for b in range(B):
        for j in _rows(path, accepted, b, T):
            kj, vj = k[b, :, j], v[b, :, j]
            size = np.einsum("hkv,hk->hv", np.abs(S[b]), np.abs(kj))
            off = (dk + 4) * u * size + 2 * u * (np.abs(vj) + size)
            S[b] = S[b] + kj[:, :, None] * (vj - np.einsum("hkv,hk->hv", S[b], kj))[:, None, :]
            norm = np.linalg.norm(kj, axis=-1)[:, None]
            err[b] = err[b] * np.maximum(1.0, np.abs(norm ** 2 - 1)) + norm * off + u * np.linalg.norm(S[b], axis=1)
    return np.broadcast_to(1.05 * err[:, :, None, :], S.shape)


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
