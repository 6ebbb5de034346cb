"""Float64 reference of the operators of include/moe_experts.h: the stable sort of tokens' slots by expert and the
copies both ways with their gradients, grouped products with bias, activation and residual and their gradients, and
dropout's generator.  Plain loops over groups and slots."""

import math

import numpy as np


# ---- tokens ----

def sort(idx, E):
    """(offsets [E+1], pos [T, k], row_slot [T*k]) of the slots idx [T, k]; outside [0, E): dropped."""
    flat = idx.reshape(-1)
    lists = [np.nonzero(flat == e)[0] for e in range(E)]
    offsets = np.cumsum([0] + [len(v) for v in lists]).astype(np.int32)
    order = np.concatenate(lists)
    pos = np.full(flat.size, -1, np.int32)
    pos[order] = np.arange(order.size)
    row_slot = np.full(flat.size, -1, np.int32)
    row_slot[:order.size] = order
    return offsets, pos.reshape(idx.shape), row_slot


def slots(pos, rows):
    """(token, slot, row) of every slot with a row."""
    return [(t, j, int(pos[t, j])) for t in range(pos.shape[0]) for j in range(pos.shape[1]) if 0 <= pos[t, j] < rows]


def collect(y, pos, w, residual):
    """Sums of w * rows per token, and the sums of their magnitudes."""
    T, d = pos.shape[0], y.shape[1]
    out = np.zeros((T, d)) if residual is None else residual.astype(np.float64)
    mag = np.abs(out)
    for t, j, r in slots(pos, y.shape[0]):
        part = y[r].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
        out[t] += part
        mag[t] += np.abs(part)
    return out, mag


def dots(tok, y, pos):
    """<tok[t], y[pos]> per slot (0 where it has no row), and the sums of magnitudes."""
    v, mag = np.zeros(pos.shape), np.zeros(pos.shape)
    for t, j, r in slots(pos, y.shape[0]):
        prod = tok[t].astype(np.float64) * y[r].astype(np.float64)
        v[t, j], mag[t, j] = prod.sum(), np.abs(prod).sum()
    return v, mag


# ---- products ----

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(z, name):
    """(value, list of derivatives: one, or those of the gate and up half)."""
    if name == "none":
        return z, [np.ones_like(z)]
    if name == "relu":
        return np.maximum(z, 0), [(z > 0).astype(np.float64)]
    if name == "gelu":
        cdf = 0.5 * _erfc(-z / math.sqrt(2))
        return z * cdf, [cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)]
    h = z if name == "silu" else z[:, :z.shape[1] // 2]
    s = 1 / (1 + np.exp(-h))
    value, slope = h * s, s * (1 + h * (1 - s))
    if name == "silu":
        return value, [slope]
    u = z[:, z.shape[1] // 2:]
    return value * u, [slope * u, value]


def ranges(offsets, rows):
    return [(0, rows)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def gemm(a, b, offsets, bias):
    """z [rows, N] (NaN outside every group) and the sums of magnitudes."""
    z, mag = np.full((a.shape[0], b.shape[1]), np.nan), np.zeros((a.shape[0], b.shape[1]))
    for g, (lo, hi) in enumerate(ranges(offsets, a.shape[0])):
        z[lo:hi] = a[lo:hi] @ b[g].T
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(b[g]).T
        if bias is not None:
            z[lo:hi] += bias[g]
            mag[lo:hi] += np.abs(bias[g])
    return z, mag


def dgrad(dz, b, offsets):
    return gemm(dz, b.transpose(0, 2, 1), offsets, None)


def wgrad(dz, a, offsets, G):
    db, mag = np.zeros((G, dz.shape[1], a.shape[1])), np.zeros((G, dz.shape[1], a.shape[1]))
    for g, (lo, hi) in enumerate(ranges(offsets, a.shape[0])):
        db[g] = dz[lo:hi].T @ a[lo:hi]
        mag[g] = np.abs(dz[lo:hi]).T @ np.abs(a[lo:hi])
    return db, mag


# ---- dropout ----

def philox(counter, key):
    """Philox4x32-10 of one 128-bit counter and 64-bit key, as four 32-bit words each (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(n, p, seed, call, first=0):
    """(mask of elements first .. n - 1, probability of keeping)."""
    words = lambda v: (v & 0xFFFFFFFF, (v >> 32) & 0xFFFFFFFF)
    q = round((1.0 - p) * 65536)
    out, block, u = [], -1, None
    for i in range(first, n):
        if i // 8 != block:
            block = i // 8
            u = philox(words(block) + words(call), words(seed))
        out.append((u[i % 8 // 2] >> (16 * (i % 2))) & 0xFFFF)
    return np.array(out, np.int64) < q, q / 65536
