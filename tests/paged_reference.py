"""The paged memory cache's operators in float64 numpy, token by token and memory by memory, for the tests.

Sequences are given as Python lists; memories as dense float64 arrays, so that nothing here knows about pages."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def place(n, N):
    """Where the code of row n of a column stands among the column's N codes."""
    return n % 16 // 4 * (N // 4) + 4 * (n // 16) + n % 4


def quantize(V):
    """(codes uint8 [..., P, N/2], scales uint8 [..., P, N/32]) of V [..., N, P] float64."""
    *lead, N, P = V.shape
    block = np.moveaxis(V.reshape(*lead, N // 32, 32, P), -1, -3)          # [..., P, N/32, 32]
    finite = np.isfinite(block).all(-1)
    a = np.where(finite[..., None], np.abs(block), 0.0)
    most = a.max(-1)
    k = np.full(most.shape, -126)
    for e in range(-126, 127):                                              # the least k with most <= 6 * 2^k
        k = np.where(most > 6.0 * 2.0 ** e, e + 1, k)
    k = np.minimum(k, 126)
    off = np.abs(a[..., None] - LEVELS * 2.0 ** k[..., None, None].astype(float))
    best = np.where(off == off.min(-1, keepdims=True), np.arange(8) % 2, 9).argmin(-1)   # of two as near, the even code
    code = np.where(finite[..., None], best + 8 * np.signbit(block), 0).reshape(*lead, P, N)
    out = np.zeros((*lead, P, N), np.uint8)
    for n in range(N):
        out[..., place(n, N)] = code[..., n]
    return out[..., 0::2] | out[..., 1::2] << 4, np.where(finite, k + 127, 255).astype(np.uint8)


def dequantize(codes, scales):
    """V [..., N, P] float64 of codes and scales."""
    *lead, P, half = codes.shape
    N = 2 * half
    both = np.stack((codes & 15, codes >> 4), -1).reshape(*lead, P, N)
    V = np.empty((*lead, N, P))
    scale = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    for n in range(N):
        c = both[..., place(n, N)]
        V[..., n, :] = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7] * scale[..., n // 32]
    return V


def extend(x, dt, A, Bm, Cm, lens, state, cur, n, pos, S):
    """The recurrence over packed tokens.  Returns y, state, cur, n, pos, counts and appended, a list for every
    sequence of the memories [H, N, P] that closed."""
    H = x.shape[1]
    group = np.arange(H) // (H // Bm.shape[1])
    y = np.zeros(x.shape)
    state, cur, n, pos = state.copy(), cur.copy(), list(n), list(pos)
    counts, appended, t = [], [[] for _ in lens], 0
    for b, length in enumerate(lens):
        for _ in range(length):
            counts.append(n[b])
            a = np.exp(dt[t] * A)[:, None, None]
            new = dt[t][:, None, None] * Bm[t][group][:, :, None] * x[t][:, None, :]
            state[b] = a * state[b] + new
            cur[b] = a * cur[b] + new
            y[t] = np.einsum("hn,hnp->hp", Cm[t][group], state[b])
            pos[b] += 1
            if pos[b] == S:
                appended[b].append(cur[b].copy())
                cur[b] = 0.0
                n[b], pos[b] = n[b] + 1, 0
            t += 1
    return y, state, cur, n, pos, counts, appended


def sma(Q, E, Cm, lens, memories, counts):
    """The attention's readout o [T, H, P]; memories: for every sequence [M, H, N, P]."""
    T, H, N = Q.shape
    group = np.arange(H) // (H // Cm.shape[1])
    o = np.zeros(E.shape)
    t = 0
    for b, length in enumerate(lens):
        for _ in range(length):
            c = counts[t]
            if c > 0:
                M = memories[b][:c]
                key = np.einsum("mhnp,hp->mhn", M, E[t])
                score = np.einsum("mhn,hn->mh", key, Q[t]) / np.sqrt(N)
                w = np.exp(score - score.max(0))
                w /= w.sum(0)
                value = np.einsum("hn,mhnp->mhp", Cm[t][group], M)
                o[t] = np.einsum("mh,mhp->hp", w, value)
            t += 1
    return o
