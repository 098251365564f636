"""fp64 oracle of the windowed attention with sinks and of the paged cache.

The definitions of include/infllmv2.h in plain numpy, one sequence at a time:
    keys(t) = { c <= t : window == 0 or c > t - window or c < n_sink }.
Beside each result stands what its rounding error scales with, so that the
tests can bound the error of a kernel element by element.
"""
import math

import numpy as np


def visible(pos, n_keys, window, n_sink):
    """[len(pos), n_keys] truth values: key c is visible to position t."""
    t = np.asarray(pos)[:, None]
    c = np.arange(n_keys)[None, :]
    return (c <= t) & ((window == 0) | (c > t - window) | (c < n_sink))


def _head(q, k, v, see, scale):
    """One head: q [r, d] over k, v [n, d] with see [r, n] -> (P, O, lse)."""
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(axis=1, keepdims=True)
    P = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, np.where(np.isfinite(m), m, 0.0) + np.log(l), -np.inf)
    return P, P @ v, lse[:, 0]


def attention(q, K, V, pos, window, n_sink, scale=None):
    """q [r, Hq, d] at positions pos over K, V [n, Hkv, d].

    Returns (O [r, Hq, d], lse [r, Hq], spread [r, Hq, d], reach [r, Hq]):
    spread = sum_c P_c |V_c| (the rounding of P moves O by at most that times
    its relative size) and reach = scale * max_c sum_d |q_d K_cd| over the
    visible keys (the fp32 sum of a score is off by at most that times its
    relative error)."""
    r, Hq, d = q.shape
    G = Hq // K.shape[1]
    sc = 1.0 / math.sqrt(d) if not scale else scale
    see = visible(pos, K.shape[0], window, n_sink)
    O, spread = np.zeros((r, Hq, d)), np.zeros((r, Hq, d))
    lse, reach = np.zeros((r, Hq)), np.zeros((r, Hq))
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        # keys that no row sees may hold anything
        dark = ~see.any(axis=0)
        k, v = np.where(dark[:, None], 0.0, k), np.where(dark[:, None], 0.0, v)
        P, O[:, h], lse[:, h] = _head(q[:, h], k, v, see, sc)
        spread[:, h] = P @ np.abs(v)
        reach[:, h] = sc * np.where(see, np.abs(q[:, h]) @ np.abs(k).T, 0.0).max(axis=1, initial=0.0)
    return O, lse, spread, reach


def backward(q, K, V, dO, window, n_sink, scale=None):
    """Gradients of attention(q, K, V, 0 .. T-1, ...) [T, H, d] given dO:
        dV = P^T dO,  dS = P (dO V^T - rowsum(dO O)),
        dQ = scale dS K,  dK = scale dS^T q.
    Returns ((dQ, dK, dV), (eQ, eK, eV)): the second triple holds the same
    sums over absolute values, with each dS widened by what the rounding of
    O (in rowsum(dO O)) can add per unit of relative error."""
    T, Hq, d = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    sc = 1.0 / math.sqrt(d) if not scale else scale
    see = visible(np.arange(T), T, window, n_sink)
    g = [np.zeros_like(q), np.zeros_like(K), np.zeros_like(V)]
    e = [np.zeros_like(q), np.zeros_like(K), np.zeros_like(V)]
    for h in range(Hq):
        j = h // G
        k, v, do = K[:, j], V[:, j], dO[:, h]
        P, o, _ = _head(q[:, h], k, v, see, sc)
        dS = P * (do @ v.T - (do * o).sum(axis=1, keepdims=True))
        # O is stored in bf16 and P was rounded on the way to it
        dD = (np.abs(do) * (np.abs(o) + P @ np.abs(v))).sum(axis=1, keepdims=True)
        wide = np.abs(dS) + P * dD
        g[0][:, h], e[0][:, h] = sc * dS @ k, sc * wide @ np.abs(k)
        g[1][:, j] += sc * dS.T @ q[:, h]
        e[1][:, j] += sc * wide.T @ np.abs(q[:, h])
        g[2][:, j] += P.T @ do
        e[2][:, j] += P.T @ np.abs(do)
    return tuple(g), tuple(e)


def paged_tables(kv_lens, q_lens, free_pages, table, page, n_tokens):
    """Block tables and slot maps, request by request: pages are popped off
    the end of free_pages, none for a column that the table lacks; -1 where
    there is none.  Returns (table, cu_q,
    seqlens, slots, positions, free_left, taken_all)."""
    table = [list(r) for r in table]
    stack = list(free_pages)
    cu, seqlens, fine = [0], [], True
    slots, positions = [-1] * n_tokens, [-1] * n_tokens
    for i, (kv, q) in enumerate(zip(kv_lens, q_lens)):
        kv, q = max(kv, 0), max(q, 0)
        for c in range(-(-kv // page), min(-(-(kv + q) // page), len(table[i]))):
            table[i][c] = stack.pop() if stack else -1
            fine = fine and table[i][c] != -1
        fine = fine and not (q > 0 and kv + q > len(table[i]) * page)
        for j in range(q):
            r, t = cu[-1] + j, kv + j
            if r >= n_tokens:
                fine = False
                continue
            positions[r] = t
            p = table[i][t // page] if t // page < len(table[i]) else -1
            if p >= 0:
                slots[r] = p * page + t % page
            else:
                fine = False
        cu.append(cu[-1] + q)
        seqlens.append(kv + q)
    return table, cu, seqlens, slots, positions, len(stack), fine
