"""A plain 64-bit model of the paged E4M3 cache and of attention over it (CPU,
shares no code with the package): what tests of csa_cache_* compare with."""
import math

import numpy as np
import torch


def e4m3_table():
    """Value of every code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = (-x if c & 0x80 else x) if (c & 0x7F) != 0x7F else np.nan
    return v


VALUES = e4m3_table()


def e4m3_codes(x):
    """Codes of float64 values within 448: nearest, ties to the even code; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    pos = VALUES[:0x7F]
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(pos[hi] == a, hi, c)
    c = np.where(np.isfinite(x), c, 0x7F)
    return (c | np.where(np.signbit(x) & np.isfinite(x), 0x80, 0)).astype(np.uint8)


def block_scale(rows):
    """Smallest 2^e, e >= -126, with max |finite| / 2^e <= 448."""
    fin = np.abs(rows[np.isfinite(rows)])
    amax = float(fin.max()) if fin.size else 0.0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Model:
    """The cache of one of K, V in numpy: codes and float64 scales."""

    def __init__(self, codes, scale, table):
        self.codes, self.scale, self.table = codes.copy(), scale.astype(np.float64).copy(), table
        self.block = codes.shape[2]

    def write(self, x, cu, pos0):
        for b in range(len(cu) - 1):
            n, p = cu[b + 1] - cu[b], pos0[b]
            i = 0
            while i < n:
                blk, lo = self.table[b][(p + i) // self.block], (p + i) % self.block
                m = min(n - i, self.block - lo)
                rows = x[cu[b] + i:cu[b] + i + m].astype(np.float64)     # [m, H_kv, d]
                for h in range(rows.shape[1]):
                    s = block_scale(rows[:, h])
                    if lo:
                        old = self.scale[blk, h]
                        s = max(s, old)
                        if s > old:
                            self.codes[blk, h, :lo] = self.rescaled(self.codes[blk, h, :lo], old / s)
                    self.scale[blk, h] = s
                    self.codes[blk, h, lo:lo + m] = e4m3_codes(rows[:, h] / s)
                i += m

    @staticmethod
    def rescaled(codes, f):
        v = VALUES[codes] * f
        out = e4m3_codes(v)
        nan = (codes & 0x7F) == 0x7F
        return np.where(nan, np.uint8(0x7F), out) if nan.any() else out

    def rows(self, b, pos):
        """Values [len(pos), H_kv, d] of positions of sequence b."""
        pos = np.asarray(pos, np.int64)
        blk = np.asarray(self.table[b])[pos // self.block]
        return VALUES[self.codes[blk, :, pos % self.block]] * self.scale[blk][:, :, None]

    def scales(self, b, pos):
        return self.scale[np.asarray(self.table[b])[np.asarray(pos, np.int64) // self.block]]


def attend(q, cu, pos0, scale, cmp=None, raw=None, idx=None, base=None, ratio=0, window=0, sink=None):
    """(out, lse, mass, ds, low) of attention over Models given as (K, V) pairs, in float64, for check():
    mass = sum of p |V|, ds the error of a score in float32, low that of weights below a half's range."""
    T, H, d = q.shape
    out, lse = np.zeros((T, H, d)), np.full((T, H), -math.inf)
    mass, ds, low = np.zeros((T, H, d)), np.zeros((T, H)), np.zeros((T, H, d))
    hk = (cmp or raw)[0].codes.shape[1]
    G = H // hk
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            p = pos0[b] + t - cu[b]
            ks, vs, ss = [], [], []
            if cmp is not None:
                vis = (p + 1) // ratio
                e = np.arange(vis)
                if idx is not None:
                    e = idx[t].astype(np.int64)
                    e = e[e >= 0] - (base[b] if base is not None else 0)
                    e = e[(e >= 0) & (e < vis)]
                ks.append(cmp[0].rows(b, e))
                vs.append(cmp[1].rows(b, e))
                ss.append(cmp[1].scales(b, e))
            if raw is not None:
                w = np.arange(max(0, p - window + 1), p + 1)
                ks.append(raw[0].rows(b, w))
                vs.append(raw[1].rows(b, w))
                ss.append(raw[1].scales(b, w))
            K, V, S = np.concatenate(ks), np.concatenate(vs), np.concatenate(ss)
            n = len(K)
            for h in range(H):
                x = (K[:, h // G] @ q[t, h]) * scale
                top = max([-math.inf] + ([float(np.max(x))] if n else []) + ([sink[h]] if sink is not None else []))
                if top == -math.inf:
                    continue
                e = np.exp(x - top)
                z = e.sum() + (math.exp(sink[h] - top) if sink is not None else 0.0)
                lse[t, h] = top + math.log(z)
                if not n:
                    continue
                out[t, h] = (e @ V[:, h // G]) / z
                mass[t, h] = (e @ np.abs(V[:, h // G])) / z
                # V = code s; the products take codes, with weights p s in halves, the largest of them as 2^7 or
                # more.  Halves below 2^-14 are multiples of 2^-24: an error of up to 2^-25 a key, 2^-32 of the largest.
                ps = e * S[:, h // G]
                low[t, h] = 2.0 ** -32 * np.max(ps) / z * (np.abs(V[:, h // G]) / S[:, h // G][:, None]).sum(0)
                # a score: d products summed in float32, then scaled, taken to log2 units and reduced
                dot = scale * float(np.max(np.abs(K[:, h // G]) @ np.abs(q[t, h])))
                ds[t, h] = 2.0 ** -24 * ((d + 4) * dot + 4 * float(np.max(np.abs(x)) + abs(top)) + n + 16)
    return out, lse, mass, ds, low


def check(got, got_lse, ref, q_dtype):
    """The kernel's outputs against attend()'s: each rounding counted once."""
    out, lse, mass, ds, low = ref
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(out))
    # weights 11 bits for bf16 queries (half a step: 2^-11), 22 bits for float32 (hi + lo halves: 2^-21 with the
    # queries' own); a relative error of 2 ds in the weights from the scores and the sum
    w = 2.0 ** -11 if q_dtype == torch.bfloat16 else 2.0 ** -21
    own = 2.0 ** -8 if q_dtype == torch.bfloat16 else 2.0 ** -23
    bound = own * np.abs(out) + (w + 4 * ds[..., None]) * mass * 1.01 + low + 1e-37
    bad = np.abs(g - out) > bound
    assert not bad[~np.isnan(out)].any(), float(np.nanmax((np.abs(g - out) / bound)))
    if got_lse is not None:
        z = got_lse.double().cpu().numpy()
        fin = np.isfinite(lse)
        assert np.array_equal(z[~fin], lse[~fin], equal_nan=True)
        lb = 4 * ds + 2.0 ** -21 * (1 + np.abs(np.where(fin, lse, 0)))
        if q_dtype == torch.float32:  # the queries' 22 bits move a score by 2^-21 of its products' sizes
            lb = lb * 8
        off = np.abs(z[fin] - lse[fin])
        assert (off <= lb[fin]).all(), float((off / lb[fin]).max())


class Setup:
    """Random caches with shuffled tables and their models."""

    def __init__(self, seed, B, rows, H_kv, d, block, shared, max_blocks=None, device="cuda"):
        self.rng = rng = np.random.default_rng(seed)
        need = [(r + block - 1) // block for r in rows]
        n = sum(need) + 2
        order = rng.permutation(n)
        width = max_blocks or max(need + [1])
        table = np.full((B, width), -7, np.int32)        # entries no call may reach
        k = 0
        for b in range(B):
            table[b, :need[b]] = order[k:k + need[b]]
            k += need[b]
        self.table, self.block, self.shared, self.B, self.n = table, block, shared, B, n
        self.kinds = []
        for _ in range(1 if shared else 2):
            x = rng.standard_normal((n, H_kv, block, d)) * np.exp(rng.standard_normal((n, H_kv, 1, 1)))
            s = np.array([[block_scale(x[i, h]) for h in range(H_kv)] for i in range(n)])
            self.kinds.append((e4m3_codes(x / s[:, :, None, None]), s))
        self.t_table = torch.from_numpy(table).to(device)

    def tensors(self, device="cuda"):
        t = [(torch.from_numpy(c).to(device), torch.from_numpy(s.astype(np.float32)).to(device)) for c, s in self.kinds]
        return dict(k=t[0][0], k_scale=t[0][1], table=self.t_table, v=None if self.shared else t[1][0],
                    v_scale=None if self.shared else t[1][1])

    def models(self):
        m = [Model(c, s, self.table) for c, s in self.kinds]
        return (m[0], m[0]) if self.shared else (m[0], m[1])
