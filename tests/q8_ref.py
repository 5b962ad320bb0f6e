"""Plain 64-bit reference of the 8-bit cache (numpy) and of filtered sampling, shared by their tests."""
import numpy as np


def _table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = np.nan if (c & 127) == 127 else (-mag if c & 128 else mag)
    return t


TABLE = _table()


def encode(x):
    """Codes of values x (already divided by the scale): nearest, ties to the even code, saturating."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    mags = TABLE[:127]
    hi = np.clip(np.searchsorted(mags, np.where(np.isnan(mag), 0, mag)), 1, 126)
    lo = hi - 1
    dl, dh = mag - mags[lo], mags[hi] - mag
    idx = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    idx = np.where(np.isnan(x), 127, idx)
    return (idx + np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def scale_byte(rows):
    a = np.abs(rows[np.isfinite(rows)])
    m = a.max() if a.size else 0.0
    k = -40
    while m > 448.0 * 2.0 ** k:
        k += 1
    return k + 127


class Cache:
    """The cache as numpy arrays: codes [pages, Hkv, bs, d], scales [pages, Hkv]; the contiguous layout is
    the same with the pages of sequence b at b * nb .. (its last page may be partial)."""

    def __init__(self, k, v, k_scale, v_scale, table, prefix, bs):
        self.code, self.scale = {"k": k, "v": v}, {"k": k_scale, "v": v_scale}
        self.table, self.prefix, self.bs = table, prefix, bs

    def write(self, b, k_rows, v_rows):
        """Rows [n, Hkv, d] behind the committed ones (prefix is not advanced)."""
        L, bs = int(self.prefix[b]), self.bs
        for name, rows in (("k", k_rows), ("v", v_rows)):
            rows = np.asarray(rows, np.float64)
            n = rows.shape[0]
            for j in range(L // bs, (L + n - 1) // bs + 1 if n else 0):
                p, lo, hi = self.table[b, j], max(L, j * bs), min(L + n, (j + 1) * bs)
                for h in range(rows.shape[1]):
                    new = rows[lo - L:hi - L, h]
                    s = scale_byte(new)
                    old = int(self.scale[name][p, h])
                    c = self.code[name][p, h]
                    if L > j * bs:
                        s = max(s, old)
                        if s > old:
                            c[:L - j * bs] = encode(TABLE[c[:L - j * bs]] * 2.0 ** (old - s))
                    c[lo - j * bs:hi - j * bs] = encode(new / 2.0 ** (s - 127))
                    self.scale[name][p, h] = s

    def rows(self, b, lo, hi):
        """Values of positions lo..hi-1: K and V, [n, Hkv, d]."""
        out = []
        for name in ("k", "v"):
            pos = np.arange(lo, hi)
            p, r = self.table[b, pos // self.bs], pos % self.bs
            s = 2.0 ** (self.scale[name][p].astype(np.float64) - 127)
            out.append(TABLE[self.code[name][p, :, r]] * s[..., None])
        return out


def attention(q, K, V, k_tree, v_tree, parent, scale):
    """One sequence in 64 bits.  q [N, Hq, d]; K, V [L, Hkv, d]; returns out, lse, and for the tolerance the
    attention of |V| and the largest score error of fp32 sums (and of a query split in two 8-bit pieces)."""
    N, Hq, d = q.shape
    L, Hkv, _ = K.shape
    G = Hq // Hkv
    out, lse = np.zeros((N, Hq, d)), np.zeros((N, Hq))
    absv, err = np.zeros((N, Hq, d)), np.zeros((N, Hq))
    for i in range(N):
        anc, j = [], i
        while j >= 0:
            anc.append(j)
            j = int(parent[j])
        for h in range(Hq):
            k = np.concatenate([K[:, h // G], k_tree[anc, h // G]])
            v = np.concatenate([V[:, h // G], v_tree[anc, h // G]])
            s = scale * (k @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            out[i, h], lse[i, h] = p @ v / p.sum(), m + np.log(p.sum())
            absv[i, h] = p @ np.abs(v) / p.sum()
            mass = np.abs(k) @ np.abs(q[i, h])
            err[i, h] = scale * ((d + 8) * 2.0 ** -24 * mass.max() +
                                 2.0 ** -17 * np.abs(q[i, h]).max() * np.abs(k).sum(1).max())
    return out, lse, absv, err


def sample(z, T, k, P, m, u):
    """(token, probability, margin): margin = the distance of u Z to the nearest border, over Z."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    V = z.shape[0]
    M = z.max()
    if M == -np.inf:
        return 0, 0.0, 1.0
    if not T > 0:
        return int(np.argmax(z)), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(z == M, 0.0, z - M) / np.float64(T))
    order = np.lexsort((np.arange(V), -z))
    n = V if k <= 0 or k > V else int(k)
    ws = w[order][:n]
    cum = np.cumsum(ws)
    if P < 1:
        n = min(n, max(1, int((cum - ws < np.float64(P) * cum[-1]).sum())))
    if m > 0:
        n = min(n, max(1, int((w[order][:n] >= min(np.float64(m), 1.0)).sum())))
    kept = np.sort(order[:n])
    c = np.cumsum(w[kept])
    x = np.float64(u) * c[-1]
    t = min(int(np.searchsorted(c, x, side="right")), n - 1)
    return int(kept[t]), w[kept[t]] / c[-1], float(np.abs(c - x).min() / c[-1])
