"""Plain 64-bit forms of the verify-step operators, for the tests: written from
the definitions in include/lora_mi355x.h, token by token."""
import numpy as np

E_MIN, E_MAX = 10, 247


def e4m3_table():
    """The number that each code stands for: 4 exponent bits (bias 7), 3 of mantissa, no infinities."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if (c & 127) == 127 else (-x if c >= 128 else x)
    return t


TABLE = e4m3_table()


def encode(x):
    """Nearest codes of values of at most 448, ties to the even code; NaN and infinities to NaN."""
    x = np.asarray(x, np.float64)
    pos = TABLE[:127]  # ascending
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = c + 128 * np.signbit(x)
    return np.where(np.isfinite(x), c, 127).astype(np.uint8)


def scale_byte(amax):
    """The smallest power of two s with amax <= 448 s, as an exponent byte."""
    if amax == 0:
        return E_MIN
    e = int(np.ceil(np.log2(amax / 448.0)))
    while 448.0 * 2.0 ** e < amax:
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= amax:
        e -= 1
    return int(np.clip(e + 127, E_MIN, E_MAX))


def k_order(P, D):
    t, d = np.arange(P)[:, None], np.arange(D)[None]
    return (((t // 16 * 4 + t % 16 // 4) * (D // 16) + d // 16) * 4 + t % 4) * 16 + d % 16


def v_order(P, D):
    t, d = np.arange(P)[:, None], np.arange(D)[None]
    return (t // 16 * D + d) * 16 + t % 16


class Cache:
    """Host copy of a cache: codes [pages][heads][P][D] in token order, and exponent bytes."""

    def __init__(self, k, v, ke, ve, P, D):
        self.P, self.D = P, D
        self.k, self.v = k[:, :, k_order(P, D)].copy(), v[:, :, v_order(P, D)].copy()
        self.ke, self.ve = ke.copy(), ve.copy()

    def raw(self):
        n, H = self.ke.shape
        k, v = (np.empty((n, H, self.P * self.D), np.uint8) for _ in range(2))
        k[:, :, k_order(self.P, self.D).reshape(-1)] = self.k.reshape(n, H, -1)
        v[:, :, v_order(self.P, self.D).reshape(-1)] = self.v.reshape(n, H, -1)
        return k, v

    def token(self, codes, exps, page, h, t):
        return TABLE[codes[page, h, t]] * 2.0 ** (int(exps[page, h]) - 127)


def page_at(seqs, i, pos, P, n_pages):
    if pos < 0 or pos >= seqs["table"].shape[1] * P:
        return -1
    p = int(seqs["table"][i, pos // P])
    return p if 0 <= p < n_pages else -1


def rows_of(seqs):
    """(sequence, row, position) of every row."""
    for i in range(len(seqs["kv_len"])):
        lo, hi = int(seqs["indptr"][i]), int(seqs["indptr"][i + 1])
        for r in range(lo, hi):
            yield i, r, max(int(seqs["kv_len"][i]), 0) - (hi - lo) + r - lo


def write(cache, seqs, k, v):
    """k, v: [n][H][D] f64; updates the cache in place."""
    P, n_pages = cache.P, len(cache.ke)
    pages = {}
    for i, r, pos in rows_of(seqs):
        page = page_at(seqs, i, pos, P, n_pages)
        if page >= 0:
            pages.setdefault(page, []).append((pos % P, r))
    for page, toks in pages.items():
        first = min(t for t, _ in toks)
        for codes, exps, x in ((cache.k, cache.ke, k), (cache.v, cache.ve, v)):
            for h in range(codes.shape[1]):
                new = np.stack([x[r, h] for _, r in toks])
                e = scale_byte(np.abs(np.where(np.isfinite(new), new, 0)).max())
                if first > 0:
                    was = int(exps[page, h])
                    e = max(e, was)
                    old = TABLE[codes[page, h, :first]]
                    moved = encode(old * 2.0 ** (was - e))
                    codes[page, h, :first] = np.where(np.isnan(old), codes[page, h, :first], moved)
                exps[page, h] = e
                for t, r in toks:
                    codes[page, h, t] = encode(x[r, h] * 2.0 ** (127 - e))


def read(cache, seqs, k, v):
    """Fills k, v [n][H][D] where the row's position names a page."""
    for i, r, pos in rows_of(seqs):
        page = page_at(seqs, i, pos, cache.P, len(cache.ke))
        if page < 0:
            continue
        for h in range(cache.ke.shape[1]):
            k[r, h] = cache.token(cache.k, cache.ke, page, h, pos % cache.P)
            v[r, h] = cache.token(cache.v, cache.ve, page, h, pos % cache.P)


def attend(cache, seqs, q, scale, window):
    """q [n][heads][D] f64.  Returns out, lse, and per row and head what the
    error bounds need: sum w |v|, the largest sum |q k| scale, the tokens."""
    n, heads, D = q.shape
    H, P = cache.ke.shape[1], cache.P
    G = heads // H
    out, lse = np.full(q.shape, np.nan), np.full((n, heads), np.nan)
    mag, big, toks = np.zeros(q.shape), np.zeros((n, heads)), np.zeros(n, int)
    for i in range(len(seqs["kv_len"])):
        lo, hi = int(seqs["indptr"][i]), int(seqs["indptr"][i + 1])
        length = max(int(seqs["kv_len"][i]), 0)
        if hi <= lo:
            continue
        at = [(t, page_at(seqs, i, t, P, len(cache.ke))) for t in range(min(length, seqs["table"].shape[1] * P))]
        at = [(t, p) for t, p in at if p >= 0]
        pos = np.array([t for t, _ in at], int)
        pg = np.array([p for _, p in at], int)
        for h in range(H):
            if len(at):
                k = TABLE[cache.k[pg, h, pos % P]] * np.exp2(cache.ke[pg, h].astype(int) - 127)[:, None]
                v = TABLE[cache.v[pg, h, pos % P]] * np.exp2(cache.ve[pg, h].astype(int) - 127)[:, None]
            for r in range(lo, hi):
                me = length - (hi - lo) + r - lo
                see = (pos <= me) & ((pos > me - window) if window else True)
                for g in range(h * G, (h + 1) * G):
                    if not see.any():
                        out[r, g], lse[r, g] = 0.0, -np.inf
                        continue
                    s = (k[see] @ q[r, g]) * scale
                    m = s.max()
                    w = np.exp(s - m)
                    out[r, g] = (w @ v[see]) / w.sum()
                    lse[r, g] = m + np.log(w.sum())
                    mag[r, g] = (w @ np.abs(v[see])) / w.sum()
                    big[r, g] = (np.abs(k[see]) @ np.abs(q[r, g])).max() * scale
                toks[r] = see.sum()
    return out, lse, mag, big, toks


def attend_bounds(dtype, out, lse, mag, big, toks, D):
    """How far out and lse may be off: one rounding of the output; for bf16
    calls the weights' f16 rounding (2^-11) and its subnormals (2^-25 a token,
    against weights of at most 1, times the largest code over the smallest
    page sum, covered by 2^-13 of the same magnitude); the scores' f32 sums
    (D terms) and the exponent's rounding (|exponent| up to `big` plus page
    scales of up to 2^40 here) in every weight, twice (numerator and
    denominator); f32 sums over the tokens."""
    u = 2.0 ** -24
    es = (D + 8) * u * big + 4 * u * (1.5 * big + 64)
    rel = 2 * es + (toks[:, None] + 64) * u
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    weights = 2.0 ** -11 + 2.0 ** -13 if dtype == "bf16" else 2.0 ** -22
    bound = half * np.abs(out) + (rel + weights)[..., None] * mag + 1e-37
    with np.errstate(invalid="ignore"):
        return bound, rel + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0)) + 2.0 ** -22


def score(x, ids, top):
    """x [n][V] f64."""
    n, V = x.shape
    logp, ent, rank = np.empty(n), np.empty(n), np.zeros(n, np.int32)
    tid, tlp = np.zeros((n, top), np.int32), np.empty((n, top))
    for i in range(n):
        m = x[i].max()
        there = 0 <= ids[i] < V
        order = np.lexsort((np.arange(V), -x[i]))[:top]
        tid[i] = order
        if m == -np.inf:
            logp[i], ent[i], tlp[i] = -np.inf, 0.0, -np.inf
            rank[i] = 1 if there else 0
            continue
        e = np.exp(x[i] - m)
        ls = np.log(e.sum())
        with np.errstate(invalid="ignore"):
            ent[i] = ls - np.where(e > 0, e * (x[i] - m), 0).sum() / e.sum()
        logp[i] = x[i, ids[i]] - m - ls if there else -np.inf
        rank[i] = 1 + (x[i] > x[i, ids[i]]).sum() if there else 0
        tlp[i] = x[i, order] - m - ls
    return logp, ent, rank, tid, tlp
