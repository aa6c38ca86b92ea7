"""Plain 64-bit references (numpy) of draft verification, of pools of blocks and of
the e4m3 cache, written from the definitions in include/libattn.h."""
import math

import numpy as np

BS = 16


# --------------------------------------------------------------------------
# draft verification
# --------------------------------------------------------------------------
def verify_one(p, q, tokens, parents, u, replacement):
    """One sequence: p, q [T, V] (q None: certain drafts).  The residual row is kept whole."""
    T, V = p.shape
    p = np.nan_to_num(np.asarray(p, np.float64), nan=0.0)
    q = None if q is None else np.nan_to_num(np.asarray(q, np.float64), nan=0.0)
    u = np.asarray(u, np.float64)
    path = [0]
    if parents[0] != -1:
        return [-1] * T, 0, -1

    def absent(t):
        return parents[t] >= t or (parents[t] >= 0 and not 0 <= tokens[t] < V)

    node = 0
    while True:
        r, S, Q, gone, taken = p[node].copy(), 1.0, 1.0, set(), -1
        for t in range(node + 1, T):
            x = int(tokens[t])
            if parents[t] != node or absent(t):
                continue
            if q is None:
                if x in gone:
                    continue
                if u[t] * S < r[x]:
                    taken = t
                    break
                S -= r[x]
                r[x] = 0.0
            else:
                if not replacement and (x in gone or Q <= 0.0):
                    continue
                if u[t] * q[node, x] * S < r[x] * Q:
                    taken = t
                    break
                r = np.maximum(r - (S / Q) * q[node], 0.0)
                if not replacement:
                    Q -= q[node, x]
                S = r.sum()
            gone.add(x)
        if taken < 0:
            break
        node = taken
        path.append(node)
    if not r.sum() > 0.0:
        r = p[node]
    sums = np.cumsum(r)
    if not sums[-1] > 0.0:
        token = -1
    else:
        past = np.nonzero(sums > u[0] * sums[-1])[0]
        token = int(past[0]) if past.size else int(np.nonzero(r > 0)[0][-1])
    return path + [-1] * (T - len(path)), len(path), token


def verify(p, q, tokens, parents, u, replacement):
    got = [verify_one(p[b], None if q is None else q[b], tokens[b], parents[b], u[b], replacement)
           for b in range(len(p))]
    return [np.array(x, np.int32) for x in zip(*got)]


# --------------------------------------------------------------------------
# pools of blocks
# --------------------------------------------------------------------------
class Pool:
    """refs, tables and lengths as lists; caches as arrays [num_blocks, ...]."""

    def __init__(self, refs, caches=()):
        self.refs, self.caches, self.flag = list(map(int, refs)), [np.array(c) for c in caches], False

    def lowest(self, n):
        free = [i for i, r in enumerate(self.refs) if r == 0][:n]
        return free + [None] * (n - len(free))

    def free(self, table, lens, done=None):
        for b, row in enumerate(table):
            if done is not None and not done[b]:
                continue
            lens[b] = -1
            for i, x in enumerate(row):
                if x < 0:
                    continue
                row[i] = -1
                if x >= len(self.refs) or self.refs[x] <= 0:
                    self.flag = True
                else:
                    self.refs[x] -= 1

    def reserve(self, table, lens, n_new):
        want = []
        for b, row in enumerate(table):
            if lens[b] < 0 or n_new[b] <= 0:
                continue
            end = -(-(lens[b] + n_new[b]) // BS)
            if end > len(row):
                self.flag = True
                continue
            want += [(b, i) for i in range(lens[b] // BS, end) if row[i] < 0]
        for (b, i), new in zip(want, self.lowest(len(want))):
            table[b][i] = -1 if new is None else new
            if new is None:
                self.flag = True
            else:
                self.refs[new] = 1

    def fork(self, table, lens, src, width):
        rows, sizes, part = [], [], []
        N, B = len(self.refs), len(table)
        for j, s in enumerate(src):
            rows.append([-1] * width)
            sizes.append(-1)
            if s < 0 or (s < B and lens[s] < 0):
                continue
            L = lens[s] if s < B else 0
            last = -(-L // BS)
            if s >= B or last > len(table[s]) or last > width or (L % BS and not 0 <= table[s][L // BS] < N):
                self.flag = True
                continue
            sizes[j] = L
            if L % BS:
                part.append(j)
        for j, new in zip(part, self.lowest(len(part))):
            if new is None:
                self.flag = True
                sizes[j] = -1
                continue
            self.refs[new] = 1
            rows[j][sizes[j] // BS] = new
            for c in self.caches:
                c[new] = c[table[src[j]][sizes[j] // BS]]
        for j, s in enumerate(src):
            for i in range(max(sizes[j], 0) // BS):
                x = table[s][i]
                if 0 <= x < N:
                    rows[j][i] = x
                    self.refs[x] += 1
                else:
                    self.flag = True
        return rows, sizes

    def compact(self, table):
        used = [i for i, r in enumerate(self.refs) if r]
        n = len(used)
        moves = dict(zip([i for i in used if i >= n], [i for i in range(n) if not self.refs[i]]))
        for a, b in moves.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for c in self.caches:
                c[b] = c[a]
        for row in table:
            for i, x in enumerate(row):
                if x >= n:
                    if x in moves:
                        row[i] = moves[x]
                    else:
                        self.flag = True
        return n


# --------------------------------------------------------------------------
# e4m3
# --------------------------------------------------------------------------
E4M3 = np.empty(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    _v = math.ldexp(_m, -9) if _e == 0 else math.ldexp(8 + _m, _e - 10)
    E4M3[_c] = (math.nan if (_c & 127) == 127 else _v) * (-1 if _c & 128 else 1)


def to_e4m3(x):
    """Codes of x: nearest, ties to the even code, +-448 at most, NaN 0x7f (of either sign)."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:127]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def append_f8(codes, scale, table, start, rows, lens=None):
    """In place: codes uint8 [N, H, 16, D], scale [N, H], rows [B, H, T, D] (one of K and V).  Returns the flag."""
    B, H, T, D = rows.shape
    N, flag = len(codes), False
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        if start[b] < 0 or n == 0:
            continue
        if start[b] + n > len(table[b]) * BS:
            flag = True
            continue
        for lb in range(start[b] // BS, (start[b] + n - 1) // BS + 1):
            x = int(table[b][lb])
            if not 0 <= x < N:
                flag = True
                continue
            s0, s1 = max(start[b] - lb * BS, 0), min(start[b] + n - lb * BS, BS)
            for h in range(H):
                new = rows[b, h, lb * BS + s0 - start[b]:lb * BS + s1 - start[b]].astype(np.float64)
                fin = np.abs(new[np.isfinite(new)])
                a = fin.max() if fin.size else 0.0
                need = 0.0
                if a > 0:
                    need = math.ldexp(1.0, max(-126, math.ceil(math.log2(a / 448.0))))
                old = float(scale[x, h]) if s0 > 0 else 0.0
                sc = old if old >= need else need
                by = sc if sc > 0 else 1.0
                if sc != old and s0 > 0 and old != 0.0:
                    codes[x, h, :s0] = to_e4m3(E4M3[codes[x, h, :s0]] * old / by)
                codes[x, h, s0:s1] = to_e4m3(new / by)
                scale[x, h] = sc
    return flag


def attn_f8(q, kc, ks, vc, vs, table, start, scale, causal, lens=None):
    """(out, lse, weighted |v|, sum of |v|) in float64; q [B, Hq, T, D], codes uint8.  Keys of bad blocks are left
    out."""
    B, Hq, T, D = q.shape
    N, H = ks.shape
    G = Hq // H
    out, mag, all_v = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        if start[b] < 0 or start[b] + n > len(table[b]) * BS:
            continue
        end = start[b] + n
        at = np.arange(end)
        blk = np.array(table[b], dtype=np.int64)[at // BS]
        ok = (blk >= 0) & (blk < N)
        at, blk = at[ok], blk[ok]
        for h in range(Hq):
            g = h // G
            k = E4M3[kc[blk, g, at % BS]] * ks[blk, g].astype(np.float64)[:, None]
            v = E4M3[vc[blk, g, at % BS]] * vs[blk, g].astype(np.float64)[:, None]
            for i in range(n):
                see = at <= start[b] + i if causal else np.ones(len(at), bool)
                if not see.any():
                    continue
                s = scale * (k[see] @ q[b, h, i])
                m = s.max()
                w = np.exp(s - m)
                lse[b, h, i] = m + math.log(w.sum()) if not np.isnan(m) else np.nan
                out[b, h, i] = w @ v[see] / w.sum()
                mag[b, h, i] = w @ np.abs(v[see]) / w.sum()
                all_v[b, h, i] = np.abs(v[see]).sum(0)
    return out, lse, mag, all_v
