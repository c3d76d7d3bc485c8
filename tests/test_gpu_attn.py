"""attn_prompt, attn_decode and the cache's pages through the binding, against
the 64-bit references of attn_ref.py within tolerances counted in roundings."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from collective_communication_amd import coll
from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
POISON = 0x7FAB


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    coll.lib()
    yield
    torch.cuda.synchronize()


def up(bits, dtype):
    return dev(bits, dtype == "bf16")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def starts(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def poisoned(shape, dtype):
    return up(np.full(shape, POISON, np.uint16), dtype)


# -------------------------------------------------------------------- prompts

def make_prompt(R, heads, kv, D, qlens, klens, dtype, seed, tail=0, mag=1.0):
    g = np.random.default_rng(seed)
    Tq, Tk = sum(qlens) + tail, sum(klens) + tail
    return [[ref.normal(g, (T, h, D), dtype, mag if i < 2 else 1.0)
             for i, (T, h) in enumerate(((Tq, heads), (Tk, kv), (Tk, kv)))] for _ in range(R)]


def check_prompt(name, bits, qs, ks, dtype, causal=True, diag=None, scale=None, outs=None, lses=None):
    for r, (q, k, v) in enumerate(bits):
        s = q.shape[2] ** -0.5 if scale is None else scale
        o, l, to, tl, w = ref.prompt(q, k, v, qs, ks, None if diag is None else diag[r], causal, s, dtype)
        got, gl = host(outs[r]), host(lses[r])
        ref.check(f"{name} rank {r}", got[w], gl[w], o[w], l[w], to[w], tl[w], dtype)
        assert (got[~w] == POISON).all() and (gl[~w] == 7.0).all(), "rows of no sequence were written"


def run_prompt(name, R, heads, kv, D, qlens, klens, dtype="bf16", causal=True, diag=None, scale=None,
               tail=0, seed=1, mag=1.0, plant=None):
    say("attn_prompt", name, R, heads, kv, D, len(qlens), sum(qlens), dtype)
    bits = make_prompt(R, heads, kv, D, qlens, klens, dtype, seed, tail, mag)
    if plant:
        for b in bits:
            plant(*b)
    qs, ks = starts(qlens), starts(klens)
    q, k, v = ([up(b[i], dtype) for b in bits] for i in range(3))
    outs = [poisoned(b[0].shape, dtype) for b in bits]
    lses = [torch.full(b[0].shape[:2], 7.0, device="cuda") for b in bits]
    coll.attn_prompt(q, k, v, outs, [i32(qs)] * R, [i32(ks)] * R, lses=lses,
                     diags=None if diag is None else [i32(d) for d in diag], causal=causal, scale=scale)
    torch.cuda.synchronize()
    check_prompt(name, bits, qs, ks, dtype, causal, diag, scale, outs, lses)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_dims(D, dtype):
    run_prompt("dims", 1, 4, 2, D, [1, 333, 64, 0, 65], [1, 333, 64, 0, 65], dtype, tail=5, seed=D)
    run_prompt("dims, all keys", 2, 2, 2, D, [100, 31], [70, 257], dtype, causal=False, seed=D + 1)


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 1), (8, 8), (32, 8), (24, 3)])
def test_prompt_head_layouts(heads, kv):
    run_prompt("heads", 1, heads, kv, 64, [129, 40], [129, 40], seed=heads)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_prompt_lengths(n):
    run_prompt("lengths", 1, 2, 1, 128, [n], [n], seed=n)
    run_prompt("lengths, other keys", 1, 2, 1, 128, [n, 3], [65, n], seed=n + 1)


def test_prompt_large_grid_and_many_sequences():
    run_prompt("large grid", 2, 16, 4, 64, [900, 131], [900, 131], "fp16", seed=8)
    run_prompt("150 sequences", 1, 2, 1, 64, [(7 * i) % 40 for i in range(150)],
               [(7 * i) % 40 for i in range(150)], seed=9)


def test_prompt_long():
    run_prompt("long", 1, 1, 1, 128, [4100], [4100], seed=10)


@pytest.mark.parametrize("D,dtype", [(96, "fp16"), (96, "bf16"), (128, "fp16"), (128, "bf16")])
def test_prompt_of_256_rows_at_a_time(D, dtype):
    """Long sequences that fill the card, of 96 and 128 elements; unseen keys that are not finite."""
    def far(q, k, v):
        v[4095], v[4200, :, :7], k[4150] = 0x7FC1, 0xFF80, 0x7FC1
    run_prompt("256 rows", 2, 64, 4, D, [260, 3], [4205, 4001], dtype, seed=D + 30, plant=far)
    run_prompt("256 rows, all keys", 1, 128, 16, D, [257, 2], [4099, 4100], dtype, causal=False, seed=D + 31)
    run_prompt("256 rows, diagonals", 2, 64, 8, D, [250, 7], [4105, 4100], dtype, seed=D + 32,
               diag=[[3900, -3], [-100, 4096]])


def test_prompt_diagonals():
    lens = [150, 97]
    diag = [[(5 - r) * n for n in lens] for r in range(8)]
    run_prompt("context parallel", 8, 4, 2, 64, lens, lens, diag=diag, seed=11)
    run_prompt("partly empty rows", 2, 2, 1, 128, [150, 97], [70, 200], diag=[[-70, 3], [-149, 96]], seed=12)
    run_prompt("extreme diagonals", 2, 1, 1, 64, [5, 4], [70, 9],
               diag=[[2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1]])


def test_prompt_scales():
    run_prompt("negative", 1, 2, 1, 64, [140], [140], scale=-0.2)
    run_prompt("large scores", 1, 2, 1, 128, [300], [300], scale=1.0, mag=6.0)
    run_prompt("tiny scores", 1, 2, 1, 128, [300], [300], "fp16", scale=1e-6)


def test_prompt_unseen_keys_have_no_influence():
    def plant(q, k, v):
        v[9], v[70], v[199, :, :5], k[155] = 0x7F80, 0x7FC1, 0xFF80, 0x7FC1
        q[3] = 0x7FC1
    run_prompt("infinities and NaN", 1, 2, 1, 64, [200], [200], plant=plant)
    run_prompt("infinities and NaN, wide", 1, 64, 4, 64, [513], [513], plant=plant)
    run_prompt("NaN, 256", 1, 2, 1, 256, [220], [220], plant=plant)

    def behind(q, k, v):
        v[-6:], k[-6:] = 0x7FC1, 0x7F80
    run_prompt("behind the last sequence", 1, 2, 1, 128, [45, 37], [45, 37], plant=behind, tail=6)


def test_prompt_reads_a_fused_projection_and_writes_a_strided_output():
    """q, k and v are slices of one buffer; the output's tokens are apart."""
    H, KV, D, lens = 4, 2, 96, [61, 130]
    say("attn_prompt strides")
    g = np.random.default_rng(3)
    T = sum(lens)
    qkv = ref.normal(g, (T, H + 2 * KV, D), "bf16")
    t, out = up(qkv, "bf16"), poisoned((T, H + 2, D), "bf16")
    lse, st = torch.empty((T, H), device="cuda"), i32(starts(lens))
    coll.attn_prompt([t[:, :H]], [t[:, H:H + KV]], [t[:, H + KV:]], [out[:, :H]], [st], [st], lses=[lse])
    torch.cuda.synchronize()
    o, l, to, tl, _ = ref.prompt(qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:], starts(lens), starts(lens),
                                 None, True, D ** -0.5, "bf16")
    got = host(out)
    ref.check("strides", got[:, :H], host(lse), o, l, to, tl, "bf16")
    assert (got[:, H:] == POISON).all()


def test_prompt_without_keys():
    """No key rows at all: every output row is empty."""
    say("attn_prompt, no keys")
    q, kv = up(np.zeros((9, 4, 64), np.uint16), "bf16"), torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = poisoned((9, 4, 64), "bf16"), torch.zeros((9, 4), device="cuda")
    coll.attn_prompt([q], [kv], [kv], [out], [i32([0, 4, 9])], [i32([0, 0, 0])], lses=[lse])
    coll.attn_prompt([q[:0]], [kv], [kv], [out[:0]], [i32([0])], [i32([0])])
    torch.cuda.synchronize()
    assert (host(out) == 0).all() and np.isneginf(host(lse)).all()


def test_prompt_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 of their buffer, 4.9 GB away."""
    say("attn_prompt, far rows")
    T, stride, H, KV, D, n = 61000, 40000, 4, 2, 64, 150
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    rows = buf.view(T, stride)[:, :(2 * H + 2 * KV) * D].view(T, 2 * H + 2 * KV, D)
    b = ref.normal(np.random.default_rng(5), (n, H + 2 * KV, D), "bf16")
    rows[T - n:, :H + 2 * KV] = up(b, "bf16")
    out, lse = rows[:, H + 2 * KV:], torch.empty((T, H), device="cuda")
    st = i32([T - n, T - 40, T])
    coll.attn_prompt([rows[:, :H]], [rows[:, H:H + KV]], [rows[:, H + KV:H + 2 * KV]], [out], [st], [st],
                     lses=[lse])
    torch.cuda.synchronize()
    want = ref.prompt(b[:, :H], b[:, H:H + KV], b[:, H + KV:], [0, n - 40, n], [0, n - 40, n], None, True,
                      D ** -0.5, "bf16")
    ref.check("far rows", host(out[T - n:]), host(lse[T - n:]), *want[:4], "bf16")


def test_prompt_many_heads_and_ranks():
    run_prompt("16 ranks", 16, 2, 1, 64, [70, 3], [70, 3], seed=21)
    run_prompt("one kv head each", 1, 100, 100, 64, [33], [33], seed=22)
    run_prompt("65 sequences, one long", 1, 2, 1, 96, [1000] + [2] * 64, [1000] + [2] * 64, seed=23)
    run_prompt("64 sequences, tiles of all levels", 1, 8, 8, 128, [i * 11 for i in range(64)],
               [i * 11 for i in range(64)], seed=24)


# --------------------------------------------------------------------- decode

def make_cache(g, R, kv, D, lens, P, dtype, width=None, spare=2):
    """Per rank (k pool, v pool, table) bits: scattered pages, NaN where no token is."""
    width = max(1, -(-max(lens) // P)) if width is None else width
    need = [-(-n // P) for n in lens]
    N = sum(need) + spare
    ranks = []
    for _ in range(R):
        table, perm, at = np.full((len(lens), width), -1, np.int32), g.permutation(N), 0
        k, v = (ref.normal(g, (N, P, kv, D), dtype) for _ in range(2))
        for s, n in enumerate(lens):
            table[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
            if n % P:
                k[table[s, n // P], n % P:] = POISON
                v[table[s, n // P], n % P:] = POISON
        ranks.append((k, v, table))
    return ranks


def run_decode(name, R, heads, kv, D, lens, P, dtype="bf16", seqs=None, scale=None, seed=1, width=None,
               head_major=False, spoil=None, lens_given=None):
    say("attn_decode", name, R, heads, kv, D, len(lens), sum(lens), P, dtype)
    g = np.random.default_rng(seed)
    ranks = make_cache(g, R, kv, D, lens, P, dtype, width)
    if spoil:
        for x in ranks:
            spoil(x[2])
    given = np.array(lens if lens_given is None else lens_given, np.int32)
    B, W = len(lens) if seqs is None else len(seqs), ranks[0][2].shape[1]
    q = [ref.normal(g, (B, heads, D), dtype) for _ in range(R)]
    pools = [[up(x[i], dtype) for x in ranks] for i in range(2)]
    if head_major:
        pools = [[p.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for p in ps] for ps in pools]
    outs = [poisoned((B, heads, D), dtype) for _ in range(R)]
    lses = [torch.full((B, heads), 7.0, device="cuda") for _ in range(R)]
    ws = torch.full((coll.attn_decode_workspace_bytes(R, B, W * P, heads, kv, D),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    coll.attn_decode([up(x, dtype) for x in q], *pools, [i32(x[2]) for x in ranks], [i32(given)] * R, outs, ws,
                     lses=lses, seqs=None if seqs is None else [i32(seqs)] * R, scale=scale)
    torch.cuda.synchronize()
    for r, (k, v, table) in enumerate(ranks):
        o, l, to, tl = ref.decode(q[r], k, v, table, given, seqs, D ** -0.5 if scale is None else scale, dtype)
        ref.check(f"{name} rank {r}", host(outs[r]), host(lses[r]), o, l, to, tl, dtype)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("P", [1, 5, 16, 24])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_dims_and_pages(D, P, dtype):
    run_decode("dims", 1, 6, 2, D, [1, 333, 64, 0, 1100], P, dtype, seed=D + P)


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 1), (16, 1), (17, 1), (40, 1), (64, 2), (8, 8), (32, 8)])
def test_decode_head_layouts(heads, kv):
    run_decode("heads", 1, heads, kv, 128, [300, 17, 129], 16, seed=heads)


@pytest.mark.parametrize("n", [1, 7, 8, 31, 32, 33, 127, 128, 129, 512, 5000, 70001])
def test_decode_lengths(n):
    run_decode("lengths", 1, 4, 1, 64, [n], 16, seed=n)
    run_decode("lengths, in a wide table", 1, 4, 2, 128, [n, 1], 64, seed=n, width=2000)


def test_decode_ranks_and_batches():
    run_decode("8 ranks", 8, 4, 1, 64, [300, 0, 1, 129, 128, 40, 2000], 32, "fp16", seed=2)
    run_decode("300 entries", 2, 2, 2, 64, [1 + (37 * i) % 400 for i in range(300)], 16, seed=3)
    run_decode("more entries than workgroups", 4, 2, 2, 64, [i % 3 for i in range(260)], 8, seed=4)
    run_decode("nothing at all", 2, 2, 1, 64, [0, 0, 0], 8, seed=5)


def test_decode_16_ranks_and_wide_batches():
    run_decode("16 ranks", 16, 2, 1, 64, [40, 300], 16, seed=31)
    run_decode("600 heads", 1, 600, 600, 64, [40, 300], 16, seed=32)
    run_decode("600 heads, split", 1, 600, 600, 64, [400], 16, seed=33, width=200)
    run_decode("1000 entries", 1, 2, 1, 64, [(13 * i) % 300 for i in range(1000)], 16, "fp16", seed=34)


def test_decode_rows_by_name_and_layouts():
    run_decode("by name", 1, 4, 2, 64, [140, 33, 700], 16, seqs=[2, 0, 0, -1, 3, 1, 2], seed=6)
    run_decode("head-major pool", 2, 4, 2, 96, [140, 333], 16, head_major=True, seed=7)
    run_decode("negative scale", 1, 2, 1, 64, [1400], 16, scale=-0.3, seed=8)
    run_decode("large scores", 1, 2, 1, 128, [1400], 16, scale=2.0, seed=9)


def test_decode_pages_and_lengths_that_do_not_exist():
    def bad(t):
        t[0, 1], t[0, 4], t[1, 0] = -1, 10 ** 6, -(2 ** 31)
    run_decode("bad pages", 1, 2, 1, 64, [140, 16, 100], 16, spoil=bad, seed=10)
    run_decode("bad pages of 5", 1, 2, 1, 64, [140, 4, 100], 5, spoil=bad, seed=11)
    run_decode("bad lengths", 1, 2, 1, 64, [160, 16, 96], 16, lens_given=[10 ** 9, -5, 96], seed=12)


def test_decode_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^31 and 2^32 elements of the pool."""
    say("attn_decode, a pool of 2.2 G elements")
    P, D, N = 64, 128, 270000                           # 2.2e9 elements, 4.4 GB a pool
    g = np.random.default_rng(1)
    k, v = (torch.empty((N, P, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = np.array([[N - 1, 3, 262144, N - 2, 131072]], np.int32)
    kb, vb = (ref.normal(g, (5, P, 1, D), "bf16") for _ in range(2))
    k[i32(pages[0]).long()] = up(kb, "bf16")
    v[i32(pages[0]).long()] = up(vb, "bf16")
    q, lens = ref.normal(g, (1, 4, D), "bf16"), np.array([5 * P - 9], np.int32)
    out, lse = poisoned((1, 4, D), "bf16"), torch.empty((1, 4), device="cuda")
    ws = torch.empty(coll.attn_decode_workspace_bytes(1, 1, 5 * P, 4, 1, D), dtype=torch.uint8, device="cuda")
    coll.attn_decode([up(q, "bf16")], [k], [v], [i32(pages)], [i32(lens)], [out], ws, lses=[lse])
    new = ref.normal(g, (2, 1, D), "bf16")
    coll.kv_write([up(new, "bf16")], [up(new, "bf16")], [k], [v], [i32(pages[:, ::-1].copy())], [i32([130])],
                  [i32([0, 2])])
    torch.cuda.synchronize()
    o, l, to, tl = ref.decode(q, kb, vb, np.arange(5, dtype=np.int32)[None], lens, None, D ** -0.5, "bf16")
    ref.check("far pages", host(out), host(lse), o, l, to, tl, "bf16")
    assert np.array_equal(host(k[262144, :2]), new) and np.array_equal(host(v[262144, :2]), new)


def _one_decode(seed, lens=(700, 33, 0, 129)):
    g = np.random.default_rng(seed)
    H, KV, D, P = 8, 2, 128, 16
    (k, v, table), = make_cache(g, 1, KV, D, list(lens), P, "bf16")
    args = dict(q=up(ref.normal(g, (len(lens), H, D), "bf16"), "bf16"), k=up(k, "bf16"), v=up(v, "bf16"),
                table=i32(table), lens=i32(lens))
    need = coll.attn_decode_workspace_bytes(1, len(lens), table.shape[1] * P, H, KV, D)
    return args, torch.empty(need, dtype=torch.uint8, device="cuda")


def _decode(a, out, lse, ws, **kw):
    return coll.attn_decode([a["q"]], [a["k"]], [a["v"]], [a["table"]], [a["lens"]], [out], ws, lses=[lse], **kw)


def test_captured_calls_share_a_workspace_and_see_new_lengths():
    """Two graphs over one workspace, replayed in turn with eager work between;
    the lengths change between the replays, as they do in serving."""
    say("graphs")
    a, ws = _one_decode(1)
    b, _ = _one_decode(2)
    outs = [torch.empty_like(a["q"]) for _ in range(2)]
    lses = [torch.empty(a["q"].shape[:2], device="cuda") for _ in range(2)]
    st = i32(starts([1] * 4))
    pouts = torch.empty_like(a["q"])
    for x, o, l in zip((a, b), outs, lses):
        _decode(x, o, l, ws)
    coll.attn_prompt([a["q"]], [a["q"][:, :2]], [b["q"][:, :2]], [pouts], [st], [st])
    torch.cuda.synchronize()
    graphs = []
    for x, o, l in zip((a, b), outs, lses):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _decode(x, o, l, ws)
            coll.attn_prompt([x["q"]], [a["q"][:, :2]], [b["q"][:, :2]], [pouts], [st], [st])
        graphs.append(g)
    for n in range(4):
        for i, x in enumerate((a, b)):
            x["lens"].copy_(i32([700 - 13 * n, 33 - n, n % 2 * 0, 100 + n]))
            o, l, p = torch.empty_like(outs[i]), torch.empty_like(lses[i]), torch.empty_like(pouts)
            ws2 = torch.empty_like(ws)
            _decode(x, o, l, ws2)
            coll.attn_prompt([x["q"]], [a["q"][:, :2]], [b["q"][:, :2]], [p], [st], [st])
            outs[i].fill_(float("nan")), lses[i].fill_(7.0), pouts.fill_(float("nan"))
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(o.view(torch.int16), outs[i].view(torch.int16)), n
            assert torch.equal(l, lses[i]) and torch.equal(p.view(torch.int16), pouts.view(torch.int16)), n


def test_calls_on_another_stream_and_repeated_calls_give_the_same_bits():
    say("streams")
    a, ws = _one_decode(3)
    o1, l1 = torch.empty_like(a["q"]), torch.empty(a["q"].shape[:2], device="cuda")
    _decode(a, o1, l1, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    plan = None
    for n in range(3):
        o2, l2 = torch.full_like(o1, float("nan")), torch.full_like(l1, 7.0)
        torch.cuda.synchronize()
        if n == 0:
            _decode(a, o2, l2, torch.empty_like(ws), stream=side)
        elif n == 1:
            with torch.cuda.stream(side):
                _decode(a, o2, l2, torch.empty_like(ws))
        else:
            plan = coll.prepare(_decode, a, o2, l2, torch.empty_like(ws))
            plan(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)


# ---------------------------------------------------------------------- pages

def _state(g, S, width, P, N, lens):
    t, refs, perm, at = np.full((S, width), -1, np.int32), np.zeros(N, np.int32), g.permutation(N), 0
    for s, n in enumerate(lens):
        m = -(-n // P)
        t[s, :m] = perm[at:at + m]
        refs[perm[at:at + m]] = 1
        at += m
    return t, np.array(list(lens) + [0] * (S - len(lens)), np.int32), refs


@pytest.mark.parametrize("P,N,S", [(1, 9000, 40), (16, 3000, 200), (20, 100, 12), (64, 40000, 600)])
def test_random_page_histories(P, N, S):
    """Random calls on one state, compared after each with the Python lists."""
    g = np.random.default_rng(P)
    width = max(4, 2 * N // S)
    first = [int(x) for x in g.integers(0, width * P // 4 + 1, S // 3)]
    t, ln, rf = (i32(x) for x in _state(g, S, width, P, N, first))
    want = ref.Pages(host(t), host(ln), host(rf), P)
    for step in range(14):
        op, n = ["extend", "fork", "free", "extend", "compact"][step % 5], int(g.integers(1, 1 + S))
        say("pages", P, N, S, op, n)
        st = i32(np.full(n, 99))
        if op == "extend":
            sq, ad = g.integers(-1, S + 1, n), g.integers(-1, width * P // 3 + 2, n)
            coll.kv_extend(t, ln, rf, i32(sq), i32(ad), P, st)
            assert np.array_equal(host(st), want.extend(sq, ad))
        elif op == "fork":
            src, dst = g.integers(-1, S + 1, n), g.integers(-1, S + 1, n)
            mv, ct = i32(np.full((n, 2), 99)), i32([99])
            coll.kv_fork(t, ln, rf, i32(src), i32(dst), P, mv, ct, st)
            status, moves = want.fork(src, dst)
            assert np.array_equal(host(st), status) and int(ct) == len(moves)
            full = np.full((n, 2), -1)
            full[:len(moves)] = np.array(moves, np.int64).reshape(-1, 2)
            assert np.array_equal(host(mv), full)
        elif op == "free":
            sq = g.integers(-1, S + 1, max(1, n // 3))
            coll.kv_free(t, ln, rf, i32(sq))
            want.free(sq)
        else:
            mv, ct = i32(np.full((N // 2 + 1, 2), 99)), i32([99])
            ws = torch.empty(coll.kv_compact_workspace_bytes(N), dtype=torch.uint8, device="cuda")
            coll.kv_compact(t, rf, mv, ct, ws)
            moves = want.compact()
            assert int(ct) == len(moves)
            full = np.full((N // 2 + 1, 2), -1)
            full[:len(moves)] = np.array(moves, np.int64).reshape(-1, 2)
            assert np.array_equal(host(mv), full)
        assert np.array_equal(host(t), want.table) and np.array_equal(host(ln), want.lens), (step, op)
        assert np.array_equal(host(rf), want.ref), (step, op)


@pytest.mark.parametrize("shape,layered", [((7, 3, 100), False), ((3, 40, 16, 2, 64), True), ((50, 1, 5), False),
                                           ((2, 30, 64, 8, 128), True)])
def test_copy_pages(shape, layered):
    say("copy_pages", shape)
    g = np.random.default_rng(1)
    N = shape[1] if layered else shape[0]
    pools = [dev(g.integers(0, 255, shape, np.int32)).to(torch.int16) for _ in range(3)]
    perm = g.permutation(N)
    moves = np.stack([perm[:N // 2], perm[N // 2:N // 2 * 2]], 1).astype(np.int32)
    moves[1] = -1, 2
    moves[2 % len(moves)] = 0, N
    for count in (None, 3, 1000):
        want = [p.clone() for p in pools]
        for a, b in moves if count is None else moves[:count]:
            if 0 <= a < N and 0 <= b < N:
                for w in want:
                    w.select(1 if layered else 0, int(b)).copy_(w.select(1 if layered else 0, int(a)))
        coll.kv_copy_pages(pools, i32(moves), None if count is None else i32([count]), layered=layered)
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(pools, want)), count


@pytest.mark.parametrize("head_major", [False, True])
def test_kv_write(head_major):
    say("kv_write", head_major)
    g = np.random.default_rng(2)
    KV, D, P, lens, new = 3, 72, 20, [400, 5, 33, 7, 90], [300, 5, 0, 1, 90]
    t, ln, _ = _state(g, 6, 20, P, 40, lens)
    T = sum(new) + 4
    kv = up(ref.normal(g, (T, 2 * KV, D), "fp16"), "fp16")
    pools = [poisoned((40, P, KV, D), "fp16") for _ in range(2)]
    want = [p.clone() for p in pools]
    if head_major:
        pools = [p.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for p in pools]
    st = starts(new, 2)
    for b in range(5):
        for i in range(st[b], st[b + 1]):
            pos = lens[b] - (st[b + 1] - i)
            for w, x in zip(want, (kv[:, :KV], kv[:, KV:])):
                w[t[b, pos // P], pos % P] = x[i]
    coll.kv_write([kv[:, :KV]], [kv[:, KV:]], [pools[0]], [pools[1]], [i32(t)], [i32(ln)], [i32(st)])
    torch.cuda.synchronize()
    assert all(torch.equal(p.contiguous().view(torch.int16), w.view(torch.int16)) for p, w in zip(pools, want))


# ------------------------------------------------------------------- together

def test_a_cache_from_prompt_to_merge():
    """Prompts fill pages, sequences are forked, grown by a token, decoded,
    compacted and decoded again; split among context-parallel ranks and merged,
    the same tokens give the same attention."""
    say("together")
    H, KV, D, P, N, S, width = 8, 2, 64, 16, 64, 6, 12
    g = np.random.default_rng(4)
    lens = [45, 100]
    T, st = sum(lens), i32(starts(lens))
    qkv_b = ref.normal(g, (T, H + 2 * KV, D), "bf16")
    qkv = up(qkv_b, "bf16")
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    table, cl, rf = i32(np.full((S, width), -1)), i32(np.zeros(S)), i32(np.zeros(N))
    pools = [poisoned((N, P, KV, D), "bf16") for _ in range(2)]

    status = i32([9, 9])
    coll.kv_extend(table, cl, rf, i32([0, 1]), i32(lens), P, status)
    coll.kv_write([k], [v], [pools[0]], [pools[1]], [table], [cl], [st])
    out = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    coll.attn_prompt([q], [k], [v], [out], [st], [st])

    # fork sequence 0 twice, then every sequence gets a token of its own
    moves, count, fst = i32(np.zeros((2, 2))), i32([0]), i32([9, 9])
    coll.kv_fork(table, cl, rf, i32([0, 0]), i32([4, 2]), P, moves, count, fst)
    coll.kv_copy_pages(pools, moves, count)
    seqs, one = i32([0, 1, 2, 4]), i32([1, 1, 1, 1])
    est = i32([9] * 4)
    coll.kv_extend(table, cl, rf, seqs, one, P, est)
    new_b = ref.normal(g, (4, H + 2 * KV, D), "bf16")
    new = up(new_b, "bf16")
    coll.kv_write([new[:, H:H + KV]], [new[:, H + KV:]], [pools[0]], [pools[1]], [table], [cl],
                  [i32([0, 1, 2, 3, 4])], seqs=[seqs])
    o1, l1 = torch.empty((4, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((4, H), device="cuda")
    ws = torch.empty(coll.attn_decode_workspace_bytes(1, 4, width * P, H, KV, D), dtype=torch.uint8, device="cuda")

    def decode(o, l):
        coll.attn_decode([new[:, :H]], [pools[0]], [pools[1]], [table], [cl], [o], ws, lses=[l], seqs=[seqs])
    decode(o1, l1)
    torch.cuda.synchronize()
    assert (host(status) == 0).all() and (host(fst) == 0).all() and (host(est) == 0).all()

    # the plain attention of each sequence's tokens
    base = starts(lens)
    want = []
    for i, s in enumerate((0, 1, 0, 0)):
        rows = np.concatenate([qkv_b[base[s]:base[s + 1]], new_b[i:i + 1]])
        want.append(ref.prompt(rows[-1:, :H], rows[:, H:H + KV], rows[:, H + KV:], [0, 1], [0, len(rows)], None,
                               True, D ** -0.5, "bf16"))
    cat = [np.concatenate([w[j] for w in want]) for j in range(4)]
    ref.check("decode after fork", host(o1), host(l1), *cat, "bf16")

    # free a fork, compact: the same bits from other pages
    coll.kv_free(table, cl, rf, i32([1]))
    seqs_left = [0, 2, 3]
    cmoves = i32(np.zeros((N // 2, 2)))
    cws = torch.empty(coll.kv_compact_workspace_bytes(N), dtype=torch.uint8, device="cuda")
    coll.kv_compact(table, rf, cmoves, count, cws)
    coll.kv_copy_pages(pools, cmoves, count)
    o2, l2 = torch.empty_like(o1), torch.empty_like(l1)
    decode(o2, l2)
    torch.cuda.synchronize()
    assert int(count) > 0
    used = int((host(rf) != 0).sum())
    assert (host(rf)[:used] > 0).all() and (host(rf)[used:] == 0).all()
    assert (host(o2)[1] == 0).all() and np.isneginf(host(l2)[1]).all()      # the freed sequence
    for i in seqs_left:
        assert np.array_equal(host(o1)[i], host(o2)[i]) and np.array_equal(host(l1)[i], host(l2)[i])

    # context parallel: rank r holds every R-th page's tokens of the cache as its own
    R, merged = 2, []
    ranks = []
    for r in range(R):
        tr = np.full((S, width), -1, np.int32)
        lr = np.zeros(S, np.int32)
        full, cur = host(table), host(cl)
        for s in range(S):
            mine = [p for j, p in enumerate(full[s]) if p >= 0 and j % R == r]
            last = -(-int(cur[s]) // P) - 1
            tr[s, :len(mine)] = mine
            lr[s] = len(mine) * P - ((P - int(cur[s]) % P) % P if last >= 0 and last % R == r else 0)
        ranks.append((tr, lr))
    os_ = [torch.empty_like(o1) for _ in range(R)]
    ls_ = [torch.empty_like(l1) for _ in range(R)]
    ws2 = torch.empty(coll.attn_decode_workspace_bytes(R, 4, width * P, H, KV, D), dtype=torch.uint8, device="cuda")
    coll.attn_decode([new[:, :H]] * R, [pools[0]] * R, [pools[1]] * R, [i32(x[0]) for x in ranks],
                     [i32(x[1]) for x in ranks], os_, ws2, lses=ls_, seqs=[seqs] * R)
    mo, ml = [torch.empty_like(o1) for _ in range(R)], [torch.empty_like(l1) for _ in range(R)]
    coll.lse_merge(os_, ls_, mo, ml)
    torch.cuda.synchronize()
    # each partial output is rounded before the merge, and the merge rounds again:
    # sum_r w_r |o_r| <= sum p |v| / l, so twice the tolerance plus a rounding of o
    for i in seqs_left:
        extra = 2 * cat[2][i] + ref.U["bf16"] * np.abs(cat[0][i])
        ref.check("merged", host(mo[1])[i], host(ml[1])[i], cat[0][i], cat[1][i], extra,
                  cat[3][i] * 2 + 1e-5, "bf16")
