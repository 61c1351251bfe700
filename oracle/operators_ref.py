"""fp64 definitions of the operators around the expert layer (numpy, TEST INFRASTRUCTURE ONLY).

Each follows its contract in include/moe_lora.h with plain loops and no rounding; arrays are
fp64 (bf16 inputs decoded by the caller).  Shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np

from .moe_lora_ref import e4m3_to_f64


# ---------------------------------------------------------------- general routing
def _scores(l: np.ndarray, score: str) -> np.ndarray:
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        p = np.exp(l - np.where(m == -np.inf, 0.0, m))
        s = p.sum(1, keepdims=True)
        return p / np.where(s == 0, 1.0, s)


def route_scored(l, top_k, score="softmax", renormalize=True, n_group=1, topk_group=1, group_score=1,
                 scale=1.0, bias=None):
    """ids [T, k] and weights [T, k].  Choice: sorts of explicit (key descending, index) lists."""
    T, E = l.shape
    per = E // n_group
    p = _scores(l, score)
    key = l if bias is None else p + np.asarray(bias, dtype=np.float64)
    basis = p if (bias is None and group_score == 2) else key
    ids = np.empty((T, top_k), np.int32)

    def order(v, cand):  # NaN first, then descending, ties to the lower index
        return sorted(cand, key=lambda i: (0 if np.isnan(v[i]) else 1, -v[i] if not np.isnan(v[i]) else 0.0, i))

    for t in range(T):
        cand = range(E)
        if n_group > 1:
            gs = []
            for g in range(n_group):
                b = [basis[t, i] for i in order(basis[t], range(g * per, (g + 1) * per))[:group_score]]
                gs.append(sum(b))
            kept = sorted(order(np.array(gs), range(n_group))[:topk_group])
            cand = [e for g in kept for e in range(g * per, (g + 1) * per)]
        ids[t] = order(key[t], cand)[:top_k]
    return ids, scale * chosen_weights(l, ids, score, renormalize)


def chosen_weights(l, ids, score, renormalize):
    x = np.take_along_axis(l, ids.astype(np.int64), 1)
    if not renormalize:
        return np.take_along_axis(_scores(l, score), ids.astype(np.int64), 1)
    with np.errstate(over="ignore", invalid="ignore"):
        z = x if score == "softmax" else np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
        m = z.max(1, keepdims=True)
        q = np.exp(z - np.where(m == -np.inf, 0.0, m))
        s = q.sum(1, keepdims=True)
        return q / np.where(s == 0, 1.0, s)


def route_scored_backward(l, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """d_logits [T, E]: the formulas of the weights' derivatives, one chosen expert at a time.
    Ids outside [0, E) take no part; equal ids of a token add up."""
    T, E = l.shape
    out = np.zeros((T, E))
    p = _scores(l, score)
    for t in range(T):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not js:
            continue
        es, g = [int(ids[t, j]) for j in js], np.array([dw[t, j] for j in js])
        if score == "softmax" and not renormalize:
            dot = sum(gj * p[t, e] for gj, e in zip(g, es))
            out[t] = -p[t] * dot
            for gj, e in zip(g, es):
                out[t, e] += p[t, e] * gj
        else:
            with np.errstate(over="ignore"):
                rest = 1.0 / (1.0 + np.exp(l[t, es])) if score == "sigmoid" else np.ones(len(es))
            if renormalize:
                q = chosen_weights(l[t:t + 1], np.array([es]), score, True)[0]
                d = q * (g - (q * g).sum()) * rest
            else:
                d = p[t, es] * rest * g
            for dj, e in zip(d, es):
                out[t, e] += dj
    return scale * out


def expert_pack(ids, E):
    """expert_offsets, expanded_to_permuted, permuted_to_expanded of a choice [T, k]."""
    flat = ids.reshape(-1)
    p2e = np.argsort(flat, kind="stable").astype(np.int32)
    e2p = np.empty_like(p2e)
    e2p[p2e] = np.arange(flat.size, dtype=np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
    return off, e2p, p2e


# ---------------------------------------------------------------- 8-bit checkpoints
CKPT_BLOCK = 32
CKPT_MIN_EXP = -117  # of a block, so that every decoded value is a normal bf16


def checkpoint_exponent(amax: float) -> int:
    """Smallest e >= CKPT_MIN_EXP with amax <= 448 * 2^e."""
    e = CKPT_MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


_E4M3 = e4m3_to_f64(np.arange(127, dtype=np.uint8))  # the finite magnitudes, ascending


def checkpoint_pack(x: np.ndarray):
    """codes uint8 [M, H] and biased exponents uint8 [M, ceil(H / 32)] of bf16 values x (fp64).
    Not-finite values become the code 0x7f (NaN) and take no part in the exponent."""
    M, H = x.shape
    nb = -(-H // CKPT_BLOCK)
    codes, exps = np.zeros((M, H), np.uint8), np.zeros((M, nb), np.uint8)
    for i in range(M):
        for b in range(nb):
            v = x[i, b * CKPT_BLOCK:(b + 1) * CKPT_BLOCK]
            fin = np.isfinite(v)
            e = checkpoint_exponent(float(np.abs(v[fin]).max(initial=0.0)))
            # a value that would round up to 2^128 is held as the largest below
            limit = 240.0 if e == 120 else 448.0
            for j, val in enumerate(v):
                if not np.isfinite(val):
                    codes[i, b * CKPT_BLOCK + j] = 0x7F
                    continue
                a = min(abs(val) / 2.0 ** e, limit)
                d = np.abs(_E4M3 - a)
                near = np.flatnonzero(d == d.min())
                c = int(near[0]) if len(near) == 1 or near[0] % 2 == 0 else int(near[1])
                codes[i, b * CKPT_BLOCK + j] = c | (0x80 if np.signbit(val) else 0)
            exps[i, b] = e + 127
    return codes, exps


def checkpoint_unpack(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    cols = np.arange(codes.shape[1]) // CKPT_BLOCK
    return e4m3_to_f64(codes) * np.ldexp(1.0, exps.astype(np.int64) - 127)[:, cols]


# ---------------------------------------------------------------- finalize, backward
def finalize_backward(d_out, y_perm, w, e2p):
    """d_y_perm [R, H] and d_weights [T, k] of out[t] = sum_j w[t, j] y_perm[e2p[t k + j]]."""
    T, k = w.shape
    dy, dw = np.zeros_like(y_perm), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = e2p[t * k + j]
            dy[p] = w[t, j] * d_out[t]
            dw[t, j] = d_out[t] @ y_perm[p]
    return dy, dw


# ---------------------------------------------------------------- projection with pooled adapters
def _adapter_rows(slot, rank, S, R):
    for s in range(S):
        rows, r = np.flatnonzero(slot == s), int(min(max(rank[s], 0), R))
        if len(rows) and r:
            yield s, rows, r


def project(x, w, slot, rank, scaling, a, b):
    """y = W x + s_a B_a (A_a x) [T, N] and v = A_a x [T, R] (zero past a row's rank)."""
    S, R = a.shape[:2]
    y, v = x @ w.T, np.zeros((x.shape[0], R))
    for s, rows, r in _adapter_rows(slot, rank, S, R):
        v[rows, :r] = x[rows] @ a[s, :r].T
        y[rows] += float(scaling[s]) * (v[rows, :r] @ b[s, :, :r].T)
    return y, v


def project_backward(dy, x, w, slot, rank, scaling, a, b, v):
    """dx [T, K], da [S, R, K], db [S, N, R]."""
    S, R = a.shape[:2]
    dx, da, db = dy @ w, np.zeros_like(a), np.zeros_like(b)
    for s, rows, r in _adapter_rows(slot, rank, S, R):
        u = float(scaling[s]) * (dy[rows] @ b[s, :, :r])
        dx[rows] += u @ a[s, :r]
        da[s, :r] = u.T @ x[rows]
        db[s, :, :r] = float(scaling[s]) * (dy[rows].T @ v[rows, :r])
    return dx, da, db
