"""Plain 64-bit forms of expert routing and of the products in 8-bit integers
(TEST INFRASTRUCTURE ONLY), in numpy, sharing no code with the GPU path.

bf16 inputs come as float64 values.  Besides each result the functions give
what the tests' tolerances need (sums of magnitudes).
"""
import numpy as np


def plan(experts, E):
    """experts [T, k] -> (offsets [E + 1], row_index [T k], token_rows [T, k]):
    the slots by (expert, token, slot); ids outside [0, E) have no row."""
    T, k = experts.shape
    pairs = sorted((int(experts[t, j]), t, j) for t in range(T) for j in range(k) if 0 <= experts[t, j] < E)
    row_index, token_rows = np.full(T * k, -1, np.int64), np.full((T, k), -1, np.int64)
    offsets = np.zeros(E + 1, np.int64)
    for r, (e, t, j) in enumerate(pairs):
        row_index[r], token_rows[t, j] = t, r
        offsets[e + 1:] += 1
    return offsets, row_index, token_rows


def choose(logits, k):
    """The k experts of the largest logits of each token, ties to the lower id,
    NaN above all, -inf never: [T, k], -1 for none."""
    T, E = logits.shape
    out = np.full((T, k), -1, np.int64)
    for t in range(T):
        can = [e for e in range(E) if logits[t, e] != -np.inf]
        can.sort(key=lambda e: (not np.isnan(logits[t, e]), 0.0 if np.isnan(logits[t, e]) else -logits[t, e], e))
        out[t, :len(can[:k])] = can[:k]
    return out


def gates(logits, experts, renormalize):
    """(weights [T, k], distance of each chosen logit from the maximum)."""
    out, dist = np.zeros(experts.shape), np.zeros(experts.shape)
    for t in range(experts.shape[0]):
        kept = experts[t] >= 0
        v = logits[t, experts[t, kept]]
        over = v if renormalize else logits[t]
        if not v.size:
            continue
        if np.isnan(over).any() or np.isposinf(over).any():
            out[t, kept] = np.nan
            continue
        m = v.max()
        out[t, kept] = np.exp(v - m) / np.exp(over - m).sum()
        dist[t, kept] = m - v
    return out, dist


def route_backward(dgates, logits, gate, experts, renormalize):
    """(dlogits, the largest of the terms they are made of)."""
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        kept = (experts[t] >= 0) & (experts[t] < E)
        e, g, d = experts[t, kept], gate[t, kept], dgates[t, kept]
        D, S = (g * d).sum(), np.abs(g * d).sum()
        if renormalize:
            np.add.at(out[t], e, g * (d - D))
            np.add.at(mag[t], e, g * (np.abs(d) + S))
        elif (logits[t] != -np.inf).any():
            p = np.exp(logits[t] - logits[t].max())
            p /= p.sum()
            np.add.at(out[t], e, g * d)
            np.add.at(mag[t], e, np.abs(g * d))
            out[t] -= p * D
            mag[t] += p * S
    return out, mag


def gather(x, token_rows, rows):
    """x [T, N] into a copy of rows [R, N]."""
    rows = rows.copy()
    for t in range(token_rows.shape[0]):
        for r in token_rows[t]:
            if 0 <= r < rows.shape[0]:
                rows[r] = x[t]
    return rows


def combine(y, token_rows, gate):
    """(out [T, N], sums of magnitudes)."""
    T, N = token_rows.shape[0], y.shape[1]
    out, mag = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j, r in enumerate(token_rows[t]):
            if 0 <= r < y.shape[0]:
                out[t] += gate[t, j] * y[r]
                mag[t] += np.abs(gate[t, j] * y[r])
    return out, mag


def combine_backward(dout, y, token_rows, gate, dy):
    """(a copy of dy with the named rows written, dgates, sums of magnitudes of dgates)."""
    dy, dg, mag = dy.copy(), np.zeros(gate.shape), np.zeros(gate.shape)
    for t in range(token_rows.shape[0]):
        for j, r in enumerate(token_rows[t]):
            if 0 <= r < y.shape[0]:
                dy[r] = gate[t, j] * dout[t]
                dg[t, j], mag[t, j] = (dout[t] * y[r]).sum(), np.abs(dout[t] * y[r]).sum()
    return dy, dg, mag


def quantise(x):
    """Rows x [M, K] of fp32 values -> (codes int8, float32 scales)."""
    x = np.asarray(x, np.float32)
    codes, scales = np.zeros(x.shape, np.int8), np.ones(x.shape[0], np.float32)
    for m, row in enumerate(x):
        amax = np.abs(row).max()
        if np.isnan(amax) or np.isinf(amax):
            scales[m] = amax
            continue
        if amax > 0:
            scales[m] = max(np.float32(amax / np.float32(127)), np.float32(2.0 ** -126))
        codes[m] = np.rint((row / scales[m]).astype(np.float64)).astype(np.int8)     # numpy divides to nearest
    return codes, scales


def product(a, w):
    """The exact sums a . w^T of codes [M, K] and [N, K] (64-bit floats hold
    them: below 2^53)."""
    return a.astype(np.float64) @ w.astype(np.float64).T


def packed(w):
    """Codes [N, K] in the packed order, filled up: int8 [Np, Kp]."""
    N, K = w.shape
    n, k = -(-N // 16) * 16, -(-K // 128) * 128
    full = np.zeros((n, k), np.int8)
    full[:N, :K] = w
    out = full.reshape(n // 16, 16, k // 64, 4, 16)            # panel, r, chunk, g, b
    return np.ascontiguousarray(out.transpose(2, 0, 3, 1, 4)).reshape(n, k)
