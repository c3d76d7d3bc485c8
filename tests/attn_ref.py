"""Plain 64-bit references of the attention and cache operators, and the
tolerances their arithmetic allows -- TEST INFRASTRUCTURE ONLY (numpy, no code
shared with the library)."""
import numpy as np

# unit roundoffs: a rounding is off by at most half a step
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}      # half of fp16's smallest step
U32 = 2.0 ** -24


# ------------------------------------------------------------ 16-bit formats

def to_bits(x, dtype):
    """float array -> uint16 bit patterns, round to nearest even."""
    x = np.asarray(x, np.float32)
    if dtype == "fp16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint16)
    b = x.view(np.uint32).astype(np.uint64)
    out = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), out)


def from_bits(b, dtype):
    """uint16 bit patterns -> float64."""
    b = np.ascontiguousarray(b)
    if dtype == "fp16":
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def normal(g, shape, dtype, scale=1.0):
    return to_bits(g.standard_normal(shape) * scale, dtype)


# ------------------------------------------------------------------ attention

def rows(q, k, v, see, scale, dtype):
    """One head.  q [n, D], k, v [m, D] in 64 bits, see [n, m]: (o, lse, tolerance of o, of lse).

    With u the unit roundoff of the 16-bit type: a weight p has a relative
    error e from the fp32 score (a dot of D terms accumulated in fp32, scaled
    and rounded, through exp: its absolute error), from the fp32 exp itself
    (2 units) and from the sum (m + 4 additions), and u from its rounding to the type;
    the output adds m fp32 additions and one last rounding:
      |do| <= (u + e) sum p |v| / l + u |o|."""
    n, D = q.shape
    u = U[dtype]
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(see, scale * (q @ k.T), -np.inf)
        m = s.max(1, initial=-np.inf)
        some = ~(m == -np.inf)                       # rows with a score above -inf (or NaN)
        p = np.where(see, np.exp(s - np.where(some, m, 0.0)[:, None]), 0.0)
        l = np.where(some, p.sum(1), 1.0)
        fine = np.where(np.isfinite(v), v, 0.0)
        o, mag_o = p @ fine / l[:, None], p @ np.abs(fine) / l[:, None]
        for j in np.nonzero(~np.isfinite(v).all(1))[0]:   # where seen, as the formula has it
            o[see[:, j] & some] += np.where(np.isfinite(v[j]), 0.0, v[j])
        lse = np.where(some, m + np.log(l), -np.inf)
        o = np.where(some[:, None], o, 0.0)
        mag = abs(scale) * np.where(see, np.abs(q) @ np.abs(k).T, 0.0).max(1, initial=0.0)
        e = U32 * ((D + 4) * mag + 8 * (np.abs(np.where(some, m, 0.0)) + 16) + 2 * see.sum(1) + 64)
        to = (u + e)[:, None] * (1 + u) * mag_o + u * np.abs(o) + TINY[dtype] * 2
        tl = e + U32 * 4 * np.abs(lse)
    return o, lse, to, tl


def prompt(q, k, v, q_starts, k_starts, diag, causal, scale, dtype):
    """q [T, H, D] bits, k, v [Tk, KV, D] bits -> (o, lse, tol o, tol lse, written rows)."""
    T, H, D = q.shape
    KV = k.shape[1]
    qf, kf, vf = (from_bits(x, dtype) for x in (q, k, v))
    o, to = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, tl = np.zeros((T, H)), np.zeros((T, H))
    written = np.zeros(T, bool)
    for b in range(len(q_starts) - 1):
        a, z, c, e = q_starts[b], q_starts[b + 1], k_starts[b], k_starts[b + 1]
        if a < 0 or z <= a or z > T:
            continue
        if c < 0 or e <= c or e > k.shape[0]:
            c = e = 0
        n, m = z - a, e - c
        d = m - n if diag is None else int(diag[b])
        see = np.ones((n, m), bool)
        if causal:
            see = np.arange(m)[None] <= np.arange(n)[:, None] + d
        for h in range(H):
            kh = h // (H // KV)
            o[a:z, h], lse[a:z, h], to[a:z, h], tl[a:z, h] = rows(qf[a:z, h], kf[c:e, kh], vf[c:e, kh], see,
                                                                  scale, dtype)
        written[a:z] = True
    return o, lse, to, tl, written


def decode(q, k_pool, v_pool, table, lens, seqs, scale, dtype):
    """q [B, H, D] bits; pools [N, P, KV, D] bits -> (o, lse, tol o, tol lse)."""
    B, H, D = q.shape
    N, P, KV, _ = k_pool.shape
    o, to = np.zeros((B, H, D)), np.zeros((B, H, D))
    lse, tl = np.full((B, H), -np.inf), np.zeros((B, H))
    for b in range(B):
        s = b if seqs is None else int(seqs[b])
        if s < 0 or s >= table.shape[0]:
            continue
        t = np.arange(min(max(int(lens[s]), 0), table.shape[1] * P))
        page = table[s, t // P]
        t = t[(page >= 0) & (page < N)]
        page = table[s, t // P]
        k, v = from_bits(k_pool[page, t % P], dtype), from_bits(v_pool[page, t % P], dtype)
        qf = from_bits(q[b], dtype)
        see = np.ones((1, len(t)), bool)
        for h in range(H):
            kh = h // (H // KV)
            a = rows(qf[h][None], k[:, kh], v[:, kh], see, scale, dtype)
            o[b, h], lse[b, h], to[b, h], tl[b, h] = a[0][0], a[1][0], a[2][0], a[3][0]
    return o, lse, to, tl


def check(name, got_o, got_lse, o, lse, to, tl, dtype):
    """got_o bits, got_lse fp32 against the reference within its tolerances
    (NaN and infinities in the same places)."""
    g = from_bits(got_o, dtype)
    for what, x, y, t in (("o", g, o, to), ("lse", got_lse.astype(np.float64), lse, tl)):
        if x.shape != y.shape:
            raise AssertionError(f"{name} {what}: shape {x.shape} for {y.shape}")
        fine = np.isfinite(y)
        if not (np.array_equal(np.isnan(x), np.isnan(y)) and
                np.array_equal(x[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])):
            raise AssertionError(f"{name} {what}: not finite at other places")
        d = np.where(fine, np.abs(np.where(fine, x, 0.0) - np.where(fine, y, 0.0)) - t, -np.inf)
        if d.size and d.max() > 0:
            i = np.argmax(d)
            at = np.unravel_index(i, x.shape)
            raise AssertionError(f"{name} {what}: {x[at]} for {y[at]} at {at}, allowed {t[at]}")


# ---------------------------------------------------------------------- pages

class Pages:
    """The page state as Python lists, one entry after the other."""

    def __init__(self, table, lens, ref, page_size):
        self.table, self.lens, self.ref = np.array(table), np.array(lens), np.array(ref)
        self.P = page_size

    def _free(self):
        return [p for p in range(len(self.ref)) if self.ref[p] == 0]

    def extend(self, seqs, add):
        status, wanted, free, seen = [], 0, self._free(), set()
        rows, width = self.table.shape
        for s, a in zip(map(int, seqs), map(int, add)):
            dup = s in seen
            seen.add(s)
            if s < 0 or s >= rows or dup or a < 0 or self.lens[s] + a > width * self.P:
                status.append(-1)
                continue
            have, then = -(-int(self.lens[s]) // self.P), -(-(int(self.lens[s]) + a) // self.P)
            first, wanted = wanted, wanted + then - have
            if wanted > len(free):
                status.append(-2)
                continue
            for j, p in enumerate(free[first:wanted]):
                self.table[s, have + j] = p
                self.ref[p] = 1
            self.lens[s] += a
            status.append(0)
        return np.array(status, np.int32)

    def fork(self, src, dst):
        status, moves, wanted, free, seen = [], [], 0, self._free(), set()
        table, lens = self.table.copy(), self.lens.copy()       # as the call begins
        rows, width = table.shape
        for s, d in zip(map(int, src), map(int, dst)):
            dup = d in seen
            seen.add(d)
            if not (0 <= s < rows and 0 <= d < rows) or s == d or dup or lens[d] != 0:
                status.append(-1)
                continue
            full, part = int(lens[s]) // self.P, int(lens[s]) % self.P > 0
            wanted += part
            if wanted > len(free):
                status.append(-2)
                continue
            self.table[d] = -1
            self.table[d, :full] = table[s, :full]
            for p in table[s, :full]:
                self.ref[p] += 1
            if part:
                self.table[d, full] = free[wanted - 1]
                self.ref[free[wanted - 1]] = 1
                moves.append((int(table[s, full]), free[wanted - 1]))
            self.lens[d] = lens[s]
            status.append(0)
        return np.array(status, np.int32), moves

    def free(self, seqs):
        seen = set()
        for s in map(int, seqs):
            if 0 <= s < self.table.shape[0] and s not in seen:
                for p in self.table[s]:
                    if 0 <= p < len(self.ref):
                        self.ref[p] -= 1
                self.table[s] = -1
                self.lens[s] = 0
            seen.add(s)

    def compact(self):
        used = [p for p in range(len(self.ref)) if self.ref[p] != 0]
        n = len(used)
        moves = list(zip([p for p in used if p >= n], [p for p in range(n) if self.ref[p] == 0]))
        to = dict(moves)
        self.table = np.array([[to.get(int(p), int(p)) for p in row] for row in self.table],
                              np.int32).reshape(self.table.shape)
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        return moves
