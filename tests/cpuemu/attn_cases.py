"""The attention and cache entry points under CPU emulation on guarded host
buffers, compared with the 64-bit references of tests/attn_ref.py -- TEST
INFRASTRUCTURE ONLY.  Run like cases.py:

    python tests/cpuemu/attn_cases.py <family> <start|end>
"""
from __future__ import annotations

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import numpy as np  # noqa: E402

import attn_ref as ref  # noqa: E402
import cases  # noqa: E402
from cases import DT, case, ok, same  # noqa: E402
from guarded import Heap, ptr, table  # noqa: E402

H = None
POISON = 0x7FAB                     # a NaN of both 16-bit types


def few(x):
    return x if len(x) <= 8 else f"{len(x)} lengths"


def starts(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def poisoned(shape):
    x = H.empty(shape, np.uint16)
    x[...] = POISON
    return x


def strided(rows, width, stride):
    """[rows, width] view of rows `stride` apart, in a buffer that ends with the last row."""
    n = (rows - 1) * stride + width if rows else 0
    buf = H.empty(max(n, 8), np.uint16)
    buf[...] = POISON
    return np.lib.stride_tricks.as_strided(buf, (rows, width), (2 * stride, 2))


def prompt_case(name, R, heads, kv, D, qlens, klens, *, dtype="bf16", causal=True, diag=None,
                scale=None, pad=0, tail=0, lse=True, plant=None, mag=1.0, seed=1,
                q_starts=None, k_starts=None):
    case("attn_prompt", name, R, heads, kv, D, few(qlens), few(klens), dtype)
    g = np.random.default_rng(seed)
    scale = D ** -0.5 if scale is None else scale
    qs = starts(qlens) if q_starts is None else np.array(q_starts, np.int32)
    ks = starts(klens) if k_starts is None else np.array(k_starts, np.int32)
    Tq, Tk = sum(qlens) + tail, sum(klens) + tail
    ins, outs, lses, want = [], [], [], []
    for r in range(R):
        q, k, v = (strided(n, h * D, h * D + pad) for n, h in ((Tq, heads), (Tk, kv), (Tk, kv)))
        q[...] = ref.normal(g, q.shape, dtype, mag)
        k[...] = ref.normal(g, k.shape, dtype, mag)
        v[...] = ref.normal(g, v.shape, dtype)
        if plant:
            plant(q.reshape(Tq, heads, D) if not pad else None, k, v)
        ins.append((q, k, v))
        outs.append(strided(Tq, heads * D, heads * D + pad))
        lses.append(H.empty((Tq, heads), np.float32))
        lses[-1][...] = 7.0
        want.append(ref.prompt(np.array(q).reshape(Tq, heads, D), np.array(k).reshape(Tk, kv, D),
                               np.array(v).reshape(Tk, kv, D), qs, ks, None if diag is None else diag[r],
                               causal, scale, dtype))
    qd, kd = [H.copy(qs) for _ in range(R)], [H.copy(ks) for _ in range(R)]
    dg = None if diag is None else [H.copy(np.array(d, np.int32)) for d in diag]
    ok(cases.L.coll_attn_prompt(
        R, table([x[0] for x in ins]), table([x[1] for x in ins]), table([x[2] for x in ins]),
        table(outs), table(lses) if lse else None, table(qd), table(kd), None if dg is None else table(dg),
        len(qs) - 1, Tq, Tk, heads, kv, D, heads * D + pad, kv * D + pad, kv * D + pad, heads * D + pad,
        int(causal), scale, DT[dtype], None), "attn_prompt")
    for r in range(R):
        o, l, to, tl, w = want[r]
        got = np.array(outs[r]).reshape(Tq, heads, D)
        ref.check(f"{name} rank {r}", got[w], lses[r][w] if lse else l[w].astype(np.float32), o[w], l[w],
                  to[w], tl[w], dtype)
        if not (got[~w] == POISON).all() or not (lses[r][~w] == 7.0).all():
            raise AssertionError(f"{name}: rows of no sequence were written")
        if not lse and not (lses[r] == 7.0).all():
            raise AssertionError(f"{name}: lse written")


def fam_prompt():
    prompt_case("one token", 1, 2, 1, 64, [1], [1])
    prompt_case("short ragged", 2, 4, 2, 64, [17, 1, 40], [17, 1, 40])
    prompt_case("zero lengths", 1, 2, 2, 64, [5, 0, 33, 0], [5, 0, 33, 0], tail=3)
    for D, dtype in ((64, "fp16"), (96, "bf16"), (128, "bf16"), (128, "fp16"), (192, "fp16"), (256, "bf16")):
        prompt_case("tiles", 1, 2, 1, D, [130], [130], dtype=dtype, seed=D)
    prompt_case("eight waves", 1, 8, 4, 128, [300], [300], seed=3)
    prompt_case("eight waves, two ranks", 2, 8, 2, 96, [258, 3], [258, 70], seed=4)
    prompt_case("more keys than queries", 1, 2, 1, 128, [70, 3], [200, 65])
    prompt_case("more queries than keys", 1, 2, 1, 64, [70, 9], [20, 0])
    prompt_case("all keys", 1, 3, 3, 96, [40, 65], [129, 7], causal=False)
    prompt_case("diagonals", 3, 2, 1, 64, [50, 40], [50, 40], diag=[[0, 39], [-20, -40], [100000, -5]])
    prompt_case("extreme diagonals", 2, 1, 1, 64, [5], [70], diag=[[2 ** 31 - 1], [-2 ** 31]])
    prompt_case("strides", 1, 2, 1, 64, [40, 30], [40, 30], pad=24)
    prompt_case("no lse", 1, 2, 1, 64, [40], [40], lse=False)
    prompt_case("negative scale", 1, 2, 1, 64, [40], [40], scale=-0.2)
    prompt_case("large scores", 1, 2, 1, 64, [100], [100], mag=8.0, scale=1.0)
    prompt_case("many sequences", 1, 1, 1, 64, [3] * 70, [3] * 70)
    prompt_case("bad starts", 1, 1, 1, 64, [20, 20], [20, 20], q_starts=[0, 20, 12, 50, 30, 40],
                k_starts=[0, 20, 10, 30, 35, 40])
    prompt_case("bad key rows", 1, 1, 1, 64, [20, 20], [20, 20], k_starts=[-1, 20, 60])

    # what a row does not see must not reach it
    def bad_v(q, k, v):
        v[9], v[70], v[99, :5], k[55] = 0x7F80, 0x7FC1, 0xFF80, 0x7FC1
    prompt_case("infinities and NaN behind the diagonal", 1, 2, 1, 64, [100], [100], plant=bad_v)
    prompt_case("... and 8 waves", 1, 8, 1, 128, [260], [260], plant=bad_v)

    # sequences of 4096 keys and more take 256 rows at a time, of 96 and 128 elements
    def far(q, k, v):
        v[4100], v[4120, :7], k[4130] = 0x7E00, 0xFF80, 0x7FC1
    prompt_case("eight waves, long", 1, 4, 2, 96, [262], [4131], plant=far, seed=5)
    prompt_case("eight waves, long, partly unseen", 2, 4, 4, 128, [3, 35], [4110, 4161], dtype="fp16", seed=6,
                diag=[[4000, 4140], [-1, 10000]])

    def bad_tail(q, k, v):
        v[-3:], k[-3:] = 0x7FC1, 0x7F80
    prompt_case("NaN behind the last sequence", 1, 2, 1, 128, [45, 37], [45, 37], plant=bad_tail, tail=3)

    def bad_q(q, k, v):
        q[3] = 0x7FC1
    prompt_case("a NaN query keeps to its row", 1, 2, 1, 64, [40], [40], plant=bad_q)

    def low(q, k, v):                        # scores of -inf: a row that sees only such keys is empty
        q[...], k[:30] = 0x3F80, 0xFF80
    prompt_case("scores of -inf", 1, 1, 1, 64, [60], [60], plant=low)


def decode_case(name, R, heads, kv, D, lens, P, *, dtype="bf16", width=None, seqs=None, scale=None,
                layout="token", spoil=None, rows=None, lse=True, pad=0, pool_pad=0, mag=1.0, seed=1,
                num_pages=None):
    case("attn_decode", name, R, heads, kv, D, few(lens), P, dtype)
    g = np.random.default_rng(seed)
    scale = D ** -0.5 if scale is None else scale
    S = len(lens)
    B = S if seqs is None else len(seqs)
    width = max(1, -(-max(lens) // P)) if width is None else width
    need = sum(min(width, -(-max(n, 0) // P)) for n in lens)
    N = need + 2 if num_pages is None else num_pages
    ts, ls, qs, ks, vs, os_, lo, want, sqs = [], [], [], [], [], [], [], [], []
    for r in range(R):
        t = np.full((S, width), -1, np.int32)
        perm, at = g.permutation(N), 0
        for s, n in enumerate(lens):
            m = min(width, -(-max(n, 0) // P))
            t[s, :m] = perm[at:at + m] if N else 0
            at += m
        row = kv * D + pool_pad
        shape, st = ((N, P, kv, D), (P * row, row, D)) if layout == "token" else \
            ((N, P, kv, D), (kv * P * D, D, P * D))
        pools = []
        for _ in range(2):
            n = (N - 1) * st[0] + (P - 1) * st[1] + (kv - 1) * st[2] + D if N else 8
            buf = H.empty(n, np.uint16)
            buf[...] = POISON
            p = np.lib.stride_tricks.as_strided(buf, shape, tuple(2 * x for x in st) + (2,))
            p[...] = ref.normal(g, shape, dtype, mag)
            pools.append(p)
        for s, n in enumerate(lens):                     # NaN where no token is
            if 0 <= n < width * P and n % P and 0 <= t[s, n // P] < N:
                pools[0][t[s, n // P], n % P:] = POISON
                pools[1][t[s, n // P], n % P:] = POISON
        q = strided(B, heads * D, heads * D + pad)
        q[...] = ref.normal(g, q.shape, dtype, mag)
        ln = np.array(lens, np.int32)
        if spoil:
            spoil(t, ln, pools)
        sq = None if seqs is None else np.array(seqs, np.int32)
        want.append(ref.decode(np.array(q).reshape(B, heads, D), pools[0], pools[1], t, ln, sq, scale, dtype))
        ts.append(H.copy(t)), ls.append(H.copy(ln)), qs.append(q), ks.append(pools[0]), vs.append(pools[1])
        os_.append(strided(B, heads * D, heads * D + pad))
        lo.append(H.empty((B, heads), np.float32))
        lo[-1][...] = 7.0
        sqs.append(None if sq is None else H.copy(sq))
    ws = H.empty(cases.L.coll_attn_decode_workspace_bytes(R, B, width * P, heads, kv, D), np.uint8)
    ws[...] = 0xFF                                       # NaN
    ok(cases.L.coll_attn_decode(
        R, table(qs), table(ks), table(vs), table(ts), table(ls), None if seqs is None else table(sqs),
        table(os_), table(lo) if lse else None, B, S, width, N, P, heads, kv, D, heads * D + pad,
        heads * D + pad, *st, scale, DT[dtype], ptr(ws), ws.nbytes, None), "attn_decode")
    for r in range(R):
        o, l, to, tl = want[r]
        ref.check(f"{name} rank {r}", np.array(os_[r]).reshape(B, heads, D),
                  lo[r] if lse else l.astype(np.float32), o, l, to, tl, dtype)
        if not lse and not (lo[r] == 7.0).all():
            raise AssertionError(f"{name}: lse written")


def fam_decode():
    decode_case("one token", 1, 2, 1, 64, [1], 16)
    decode_case("no token", 1, 2, 1, 64, [0, 0], 16)
    decode_case("one unit", 1, 4, 1, 128, [77], 16)
    decode_case("split in many", 1, 4, 1, 64, [5000], 16)
    decode_case("ragged ranks", 2, 4, 2, 64, [300, 0, 1, 129, 128, 40], 32, dtype="fp16")
    for D, dtype in ((64, "bf16"), (96, "fp16"), (128, "fp16"), (192, "bf16"), (256, "fp16")):
        decode_case("dims", 1, 3, 3, D, [200, 37], 8, dtype=dtype, seed=D)
        decode_case("dims, split", 2, 3, 3, D, [200, 37, 700], 8, dtype=dtype, seed=D, width=130)
    decode_case("ragged ranks, split", 2, 4, 2, 64, [300, 0, 1, 129, 128, 40], 32, dtype="fp16", width=40)
    decode_case("20 heads share, split", 1, 40, 2, 64, [640, 260], 16, width=70)
    decode_case("pages of 3, split", 1, 2, 1, 128, [650, 3], 3, width=400)
    decode_case("300 entries, split", 2, 1, 1, 64, [1 + (7 * i) % 300 for i in range(300)], 32, width=40)
    decode_case("pages of 20", 1, 4, 2, 128, [333, 19, 20, 21], 20)
    decode_case("pages of 1", 1, 2, 1, 64, [150], 1)
    decode_case("pages of 3, D 256", 1, 2, 1, 256, [150], 3)
    decode_case("pages of 128", 1, 2, 1, 96, [150, 300], 128)
    decode_case("16 heads share", 1, 16, 1, 64, [140], 16)
    decode_case("20 heads share", 1, 40, 2, 64, [140, 260], 16)
    decode_case("head-major pool", 1, 4, 2, 64, [140, 33], 16, layout="head")
    decode_case("padded pool and rows", 1, 4, 2, 64, [140, 33], 16, pad=8, pool_pad=40)
    decode_case("rows by name", 1, 2, 1, 64, [140, 33, 7], 16, seqs=[2, 0, 0, -1, 3, 1])
    decode_case("no lse", 1, 2, 1, 64, [140], 16, lse=False)
    decode_case("negative scale", 1, 2, 1, 64, [140], 16, scale=-0.3)
    decode_case("large scores", 1, 2, 1, 64, [600], 16, mag=8.0, scale=1.0)
    decode_case("300 entries", 1, 1, 1, 64, [1 + (7 * i) % 150 for i in range(300)], 32)
    decode_case("more entries than workgroups", 4, 2, 2, 64, [1 + i % 3 for i in range(150)], 8)
    decode_case("empty pool", 1, 2, 1, 64, [5], 16, num_pages=0, width=1,
                spoil=lambda t, n, p: t.fill(0))

    def bad_pages(t, ln, pools):
        t[0, 1], t[0, 4], t[1, 0] = -1, 10 ** 6, -(2 ** 31)
    decode_case("pages that do not exist", 1, 2, 1, 64, [140, 16, 100], 16, spoil=bad_pages)
    decode_case("pages of 5 that do not exist", 1, 2, 1, 64, [140, 4, 100], 5, spoil=bad_pages)

    def bad_lens(t, ln, pools):
        ln[0], ln[1] = 10 ** 9, -5
    decode_case("lengths outside the row", 1, 2, 1, 64, [160, 16, 100], 16, spoil=bad_lens)

    def bad_first(t, ln, pools):
        pools[0][0], pools[1][0] = POISON, POISON
        t[t == 0] = -1
    decode_case("NaN in the pool's first page", 1, 2, 1, 64, [140, 20], 16, spoil=bad_first)


# ---------------------------------------------------------------------- pages

def page_state(g, S, width, P, N, lens):
    t, refs, perm, at = np.full((S, width), -1, np.int32), np.zeros(N, np.int32), g.permutation(N), 0
    for s, n in enumerate(lens):
        m = -(-n // P)
        t[s, :m] = perm[at:at + m]
        refs[perm[at:at + m]] = 1
        at += m
    return t, np.array(list(lens) + [0] * (S - len(lens)), np.int32), refs


def state_case(name, S, width, P, N, lens, steps, seed=1):
    """Runs the steps (op, lists...) on one state and compares it after each."""
    g = np.random.default_rng(seed)
    t, ln, rf = (H.copy(x) for x in page_state(g, S, width, P, N, lens))
    want = ref.Pages(t, ln, rf, P)
    for step in steps:
        op, lists = step[0], [H.copy(np.array(x, np.int32)) for x in step[1:]]
        n = len(lists[0]) if lists else 0
        case("pages", name, op, n)
        args = (ptr(t), ptr(ln), ptr(rf), S, width, N, P)
        status = H.poison((n,), np.int32)
        if op == "extend":
            ok(cases.L.coll_kv_extend(*args, ptr(lists[0]), ptr(lists[1]), n, ptr(status), None), op)
            same(status, want.extend(*lists), f"{name}: extend status")
        elif op == "fork":
            moves, count = H.poison((n, 2), np.int32), H.poison((1,), np.int32)
            ok(cases.L.coll_kv_fork(*args, ptr(lists[0]), ptr(lists[1]), n, ptr(moves), ptr(count),
                                    ptr(status), None), op)
            st, mv = want.fork(*lists)
            same(status, st, f"{name}: fork status")
            full = np.full((n, 2), -1, np.int32)
            full[:len(mv)] = np.array(mv, np.int32).reshape(-1, 2)
            same(moves, full, f"{name}: fork moves")
            assert count[0] == len(mv), (name, count, mv)
        elif op == "free":
            ok(cases.L.coll_kv_free(*args[:6], ptr(lists[0]), n, None), op)
            want.free(*lists)
        else:
            moves, count = H.poison((N // 2 + 1, 2), np.int32), H.poison((1,), np.int32)
            ws = H.poison(cases.L.coll_kv_compact_workspace_bytes(N), np.uint8)
            ok(cases.L.coll_kv_compact(ptr(t), ptr(rf), S, width, N, ptr(moves), N // 2 + 1, ptr(count),
                                       ptr(ws), ws.nbytes, None), op)
            mv = want.compact()
            full = np.full((N // 2 + 1, 2), -1, np.int32)
            full[:len(mv)] = np.array(mv, np.int32).reshape(-1, 2)
            same(moves, full, f"{name}: compact moves")
            assert count[0] == len(mv), (name, count, mv)
        same(t, want.table.astype(np.int32), f"{name}: table after {op}")
        same(ln, want.lens.astype(np.int32), f"{name}: lens after {op}")
        same(rf, want.ref.astype(np.int32), f"{name}: ref after {op}")


def far_case():
    """Entries that together ask for more than 2^31 pages: the rows of a table of
    2^30 columns, of which only the first entry's pages are ever written."""
    case("pages", "more than 2^31 asked for")
    S, width, N = 4, 1 << 30, 8
    t, ln, rf = H.copy(np.full(3, -1, np.int32)), H.copy(np.zeros(S, np.int32)), H.copy(np.zeros(N, np.int32))
    seqs, add, status = H.copy(np.arange(4, dtype=np.int32)), H.copy(np.array([3] + [1 << 30] * 3, np.int32)), \
        H.poison((4,), np.int32)
    ok(cases.L.coll_kv_extend(ptr(t), ptr(ln), ptr(rf), S, width, N, 1, ptr(seqs), ptr(add), 4, ptr(status), None),
       "extend")
    same(status, np.array([0, -2, -2, -2], np.int32), "status")
    same(t, np.arange(3, dtype=np.int32), "pages")
    same(ln, np.array([3, 0, 0, 0], np.int32), "lens")
    same(rf, np.array([1] * 3 + [0] * 5, np.int32), "ref")


def copy_case(name, pools, layers, N, page_bytes, moves, count=None, seed=1):
    case("copy_pages", name, pools, layers, N, page_bytes)
    g = np.random.default_rng(seed)
    bufs = [H.copy(g.integers(0, 256, (layers, N, page_bytes), np.uint8)) for _ in range(pools)]
    want = [b.copy() for b in bufs]
    mv = np.array(moves, np.int32).reshape(-1, 2)
    used = mv if count is None else mv[:max(0, min(count, len(mv)))]
    for a, b in used:
        if 0 <= a < N and 0 <= b < N:
            for w in want:
                w[:, b] = w[:, a]
    mvd, ct = H.copy(mv), None if count is None else H.copy(np.array([count], np.int32))
    ok(cases.L.coll_kv_copy_pages(pools, table(bufs), layers, N, page_bytes, ptr(mvd), len(mv), ptr(ct), None),
       "copy_pages")
    for b, w in zip(bufs, want):
        same(b, w, name)


def write_case(name, R, kv, D, lens, new, P, *, first=0, tail=0, pad=0, seqs=None, spoil=None, layout="token"):
    case("kv_write", name, R, kv, D, lens, new, P)
    g = np.random.default_rng(5)
    S = len(lens)
    width = -(-max(lens) // P)
    N = sum(-(-n // P) for n in lens) + 1
    T = first + sum(new) + tail
    st = starts(new, first)
    ins, pools, tabs, lns, want, sqs, std = [], [], [], [], [], [], []
    for r in range(R):
        t, ln, _ = page_state(g, S, width, P, N, lens)
        if spoil:
            spoil(t, ln, st)
        k, v = (strided(T, kv * D, kv * D + pad) for _ in range(2))
        k[...], v[...] = ref.normal(g, k.shape, "bf16"), ref.normal(g, v.shape, "bf16")
        pair = []
        for x in (k, v):
            shape = (N, P, kv, D) if layout == "token" else (N, kv, P, D)
            p = poisoned(shape)
            w = np.array(p)
            view = w if layout == "token" else w.transpose(0, 2, 1, 3)
            for b in range(len(new)):
                s = b if seqs is None else seqs[b]
                for i in range(st[b], st[b + 1]):
                    pos = ln[s] - (st[b + 1] - i) if 0 <= s < S else -1
                    if 0 <= pos < width * P and 0 <= t[s, pos // P] < N:
                        view[t[s, pos // P], pos % P] = x[i].reshape(kv, D)
            pair.append((p, w))
        ins.append((k, v)), pools.append(pair)
        tabs.append(H.copy(t)), lns.append(H.copy(ln)), std.append(H.copy(st))
        sqs.append(None if seqs is None else H.copy(np.array(seqs, np.int32)))
    strides = (P * kv * D, kv * D, D) if layout == "token" else (P * kv * D, D, P * D)
    ok(cases.L.coll_kv_write(R, table([x[0] for x in ins]), table([x[1] for x in ins]),
                             table([p[0][0] for p in pools]), table([p[1][0] for p in pools]), table(tabs),
                             table(lns), table(std), None if seqs is None else table(sqs), T, len(new), S,
                             width, N, P, kv, D, kv * D + pad, kv * D + pad, *strides, DT["bf16"], None),
       "kv_write")
    for r in range(R):
        for (p, w) in pools[r]:
            same(p, w, name)


def fam_pages():
    steps = [("extend", [0, 3, 1], [5, 20, 0]), ("fork", [0, 1, 0], [4, 5, 6]), ("free", [1, 1, 9, -1]),
             ("extend", [0, 4, 4], [40, 3, 3]), ("compact",), ("fork", [6, 4], [1, 7]), ("free", [0, 4, 5, 6]),
             ("compact",), ("compact",)]
    state_case("small", 8, 8, 8, 40, [30, 17, 16], steps)
    state_case("pages of 1", 8, 30, 1, 60, [10, 3, 0], steps[:1] + steps[4:5] + steps[2:3])
    state_case("pages of 5", 8, 20, 5, 90, [31, 44, 5], steps)
    state_case("not enough pages", 6, 10, 4, 12, [17, 6],
               [("extend", [2, 1, 3], [16, 1, 9]), ("fork", [0, 1, 0], [4, 5, 3]), ("extend", [3, 2], [1, 0])])
    state_case("not valid", 4, 3, 4, 16, [5, 6],
               [("extend", [-1, 4, 2, 2, 0, 1], [1, 1, 4, 4, -1, 100]),
                ("fork", [0, 0, 0, 5, -1, 0, 3], [0, 3, 3, 2, 2, 1, 2])])
    state_case("chains and empty sources", 6, 4, 4, 20, [6, 9, 0],
               [("fork", [0, 3, 2, 1], [3, 4, 5, 2]), ("fork", [3, 4], [4, 5])])
    state_case("one sequence many times", 300, 2, 4, 400, [7], [("fork", [0] * 290, list(range(5, 295))),
                                                             ("free", list(range(0, 290)) + [294] * 3),
                                                             ("compact",)])
    state_case("1024 entries", 1100, 1, 2, 5000, [1] * 40,
               [("extend", list(range(1024)), [i % 3 for i in range(1024)]), ("free", list(range(0, 1024))),
                ("compact",)])
    state_case("rows of a wide table", 60, 700, 4, 700, [30, 2500],
               [("fork", [0, 1, 0] * 10, list(range(5, 35))), ("compact",), ("free", [1, 6])])
    far_case()
    state_case("nothing free", 3, 4, 2, 4, [8], [("extend", [1], [1]), ("compact",), ("fork", [0], [2])])
    state_case("nothing used", 3, 4, 2, 9, [], [("compact",), ("free", [0, 1])])
    copy_case("one", 1, 1, 4, 64, [(0, 2)])
    copy_case("layers and pools", 3, 2, 6, 4100 * 4, [(0, 2), (1, 5), (-1, -1), (0, 7), (9, 1), (3, 4)])
    copy_case("odd bytes", 2, 3, 5, 37, [(4, 0), (1, 2)])
    copy_case("counted", 2, 1, 5, 96, [(4, 0), (1, 2), (4, 3)], count=2)
    copy_case("count past the list", 1, 1, 5, 96, [(4, 0), (1, 2)], count=99)
    copy_case("none", 1, 1, 5, 96, [(4, 0)], count=0)
    copy_case("negative count", 1, 1, 5, 96, [(4, 0)], count=-3)
    write_case("one", 1, 1, 64, [1], [1], 16)
    write_case("ragged", 2, 2, 64, [40, 5, 33, 7], [30, 5, 0, 1], 16, first=2, tail=3, pad=8)
    write_case("pages of 5, wide", 1, 8, 128, [23, 4], [7, 4], 5)
    write_case("head-major", 1, 2, 24, [23, 4], [7, 4], 8, layout="head")
    write_case("rows by name", 1, 1, 64, [23, 4, 9], [7, 4, 2, 3], 8, seqs=[2, 0, 5, -1])

    def bad(t, ln, st):
        t[0, 1], t[1, 0], ln[2] = -1, 10 ** 6, 1
    write_case("pages that do not exist", 1, 1, 64, [23, 4, 9], [20, 4, 5], 8, spoil=bad)


FAMILIES = {"prompt": fam_prompt, "decode": fam_decode, "pages": fam_pages}


def main():
    global H
    H = Heap(sys.argv[2])
    cases.H = H
    cases.load()
    FAMILIES[sys.argv[1]]()
    print("all cases passed", flush=True)


if __name__ == "__main__":
    main()
