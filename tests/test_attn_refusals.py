"""What the attention and cache calls refuse, on the host and before any launch
(CPU only: no call here reaches a kernel)."""
import ctypes
import os

import pytest
import torch

from collective_communication_amd import coll

INVALID, UNSUPPORTED = -1, -2
NULL = None


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(coll.LIB_PATH):
        from collective_communication_amd import build
        build.build()
    return coll.lib()


def t(*p):
    return (ctypes.c_void_p * len(p))(*p)


P2 = t(0x10000, 0x20000)


def prompt(L, **kw):
    a = dict(R=2, q=P2, k=P2, v=P2, o=P2, lse=NULL, qs=P2, ks=P2, diag=NULL, nseq=2, q_rows=8, k_rows=8,
             heads=4, kv=2, D=64, q_stride=256, k_stride=128, v_stride=128, o_stride=256, causal=1, scale=0.1,
             dtype=0)
    a.update(kw)
    return L.coll_attn_prompt(*a.values(), NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(R=0), INVALID), (dict(R=17), INVALID), (dict(dtype=9), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(heads=0), INVALID), (dict(kv=0), INVALID), (dict(heads=5), INVALID),
    (dict(heads=1 << 17, kv=1), INVALID), (dict(D=0), INVALID), (dict(D=80, q_stride=512, k_stride=512,
                                                                      v_stride=512, o_stride=512), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(nseq=-1), INVALID), (dict(q_rows=-1), INVALID),
    (dict(k_rows=-1), INVALID), (dict(q_rows=1 << 31), INVALID), (dict(k_rows=1 << 31), INVALID),
    (dict(q_stride=255), INVALID), (dict(q_stride=260), INVALID), (dict(k_stride=120), INVALID),
    (dict(v_stride=129), INVALID), (dict(o_stride=0), INVALID), (dict(q_stride=1 << 60), INVALID),
    (dict(q=NULL), INVALID), (dict(q=t(0x10000, 0)), INVALID), (dict(k=NULL), INVALID), (dict(v=t(0, 0x10000)), INVALID),
    (dict(o=NULL), INVALID), (dict(qs=NULL), INVALID), (dict(ks=t(0x10000, 0)), INVALID),
    (dict(diag=t(0x10000, 0)), INVALID), (dict(q=t(0x10008, 0x20000)), INVALID), (dict(k=t(0x10000, 0x20002)), INVALID),
    (dict(o=t(0x10000, 0x20004)), INVALID), (dict(nseq=0), 0), (dict(q_rows=0), 0),
    (dict(k_stride=(1 << 25) + 8), UNSUPPORTED), (dict(v_stride=1 << 26), UNSUPPORTED),
    (dict(nseq=1 << 22), UNSUPPORTED), (dict(nseq=1 << 22, D=256, q_stride=1024, o_stride=1024, k_stride=512,
                                             v_stride=512), UNSUPPORTED),
])
def test_prompt(L, kw, want):
    assert prompt(L, **kw) == want


def decode(L, **kw):
    need = L.coll_attn_decode_workspace_bytes(2, 3, 160, 4, 2, 64)
    a = dict(R=2, q=P2, k=P2, v=P2, tab=P2, lens=P2, seqs=NULL, o=P2, lse=NULL, batch=3, rows=3, width=10, N=50,
             P=16, heads=4, kv=2, D=64, q_stride=256, o_stride=256, ps=2048, ts=128, hs=64, scale=0.1, dtype=0,
             ws=0x100000, ws_bytes=need)
    a.update(kw)
    return L.coll_attn_decode(*a.values(), NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(R=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(heads=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(batch=-1), INVALID), (dict(batch=1 << 25), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=2), INVALID), (dict(width=-1), INVALID), (dict(N=-1), INVALID), (dict(N=1 << 31), INVALID),
    (dict(P=0), INVALID), (dict(ps=-8), INVALID), (dict(ps=2050), INVALID), (dict(ts=4), INVALID),
    (dict(hs=63), INVALID), (dict(ps=1 << 60), INVALID), (dict(q_stride=248), INVALID), (dict(o_stride=257), INVALID),
    (dict(q=NULL), INVALID), (dict(o=t(0x10000, 0)), INVALID), (dict(lens=NULL), INVALID), (dict(k=NULL), INVALID),
    (dict(v=t(0x10000, 0)), INVALID), (dict(tab=NULL), INVALID), (dict(seqs=t(0x10000, 0)), INVALID),
    (dict(k=t(0x10000, 0x20008)), INVALID), (dict(q=t(0x10002, 0x20000)), INVALID), (dict(ws=NULL), INVALID),
    (dict(ws=0x100080), INVALID), (dict(ws_bytes=0), INVALID), (dict(width=1 << 28, P=16), UNSUPPORTED),
    (dict(width=(1 << 31) - 1, P=1, ws_bytes=1 << 40), UNSUPPORTED),
    (dict(batch=1 << 24, rows=1 << 24, width=1 << 20, ws_bytes=1 << 40), UNSUPPORTED), (dict(batch=0), 0),
])
def test_decode(L, kw, want):
    assert decode(L, **kw) == want


def test_decode_workspace(L):
    f = L.coll_attn_decode_workspace_bytes
    need = f(2, 3, 160, 4, 2, 64)
    assert need > 0 and need % 256 == 0
    assert decode(L, ws_bytes=need - 1) == INVALID
    # the size stops growing with the batch and the length
    assert f(8, 512, 131072, 32, 8, 128) == f(8, 4096, 1 << 20, 32, 8, 128) < 32 << 20
    assert f(0, 3, 160, 4, 2, 64) == f(2, 0, 160, 4, 2, 64) == f(2, 3, -1, 4, 2, 64) == 0
    assert f(2, 3, 160, 5, 2, 64) == f(2, 3, 160, 4, 2, 80) == f(2, 3, 1 << 31, 4, 2, 64) == 0


def write(L, **kw):
    a = dict(R=2, k=P2, v=P2, kp=P2, vp=P2, tab=P2, lens=P2, starts=P2, seqs=NULL, tokens=9, batch=3, rows=3, width=10,
             N=50, P=16, kv=2, D=64, ks=128, vs=128, ps=2048, ts=128, hs=64, dtype=0)
    a.update(kw)
    return L.coll_kv_write(*a.values(), NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(R=17), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), INVALID), (dict(D=60), UNSUPPORTED),
    (dict(D=2048, ks=4096, vs=4096), UNSUPPORTED), (dict(kv=0), INVALID), (dict(tokens=-1), INVALID),
    (dict(batch=4), INVALID), (dict(batch=-1), INVALID), (dict(ks=127), INVALID), (dict(vs=120), INVALID),
    (dict(ps=2049), INVALID), (dict(P=0), INVALID), (dict(k=NULL), INVALID), (dict(vp=t(0x10000, 0)), INVALID),
    (dict(tab=NULL), INVALID), (dict(lens=NULL), INVALID), (dict(starts=NULL), INVALID),
    (dict(seqs=t(0, 0x10000)), INVALID), (dict(kp=t(0x10008, 0x20000)), INVALID), (dict(width=1 << 28), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(tokens=1 << 26), UNSUPPORTED), (dict(tokens=0), 0), (dict(batch=0), 0), (dict(rows=0), 0), (dict(N=0), 0),
])
def test_write(L, kw, want):
    assert write(L, **kw) == want


def test_page_calls(L):
    st = (0x1000, 0x2000, 0x3000)
    ok = (*st, 4, 8, 100, 16)
    for n, want in ((0, 0), (-1, INVALID), (1025, INVALID)):
        assert L.coll_kv_extend(*ok, 0x4000, 0x5000, n, 0x6000, NULL) == want
        assert L.coll_kv_fork(*ok, 0x4000, 0x5000, n, 0x6000, 0x7000, 0x8000, NULL) == want
        assert L.coll_kv_free(*ok[:6], 0x4000, n, NULL) == want
    for bad in ((-1, 8, 100, 16), (4, -1, 100, 16), (4, 8, -1, 16), (4, 8, (1 << 31) - 1, 16), (4, 8, 100, 0),
                (4, 1 << 27, 100, 16)):
        assert L.coll_kv_extend(*st, *bad, 0x4000, 0x5000, 2, 0x6000, NULL) == INVALID
        assert L.coll_kv_fork(*st, *bad, 0x4000, 0x5000, 2, 0x6000, 0x7000, 0x8000, NULL) == INVALID
    for i in range(3):
        null = tuple(NULL if j == i else p for j, p in enumerate(st)) + (4, 8, 100, 16)
        assert L.coll_kv_extend(*null, 0x4000, 0x5000, 2, 0x6000, NULL) == INVALID
        assert L.coll_kv_fork(*null, 0x4000, 0x5000, 2, 0x6000, 0x7000, 0x8000, NULL) == INVALID
        assert L.coll_kv_free(*null[:6], 0x4000, 2, NULL) == INVALID
    assert L.coll_kv_extend(*ok, NULL, 0x5000, 2, 0x6000, NULL) == INVALID
    assert L.coll_kv_extend(*ok, 0x4000, NULL, 2, 0x6000, NULL) == INVALID
    assert L.coll_kv_extend(*ok, 0x4000, 0x5000, 2, NULL, NULL) == INVALID
    for i in range(3):
        outs = [NULL if j == i else p for j, p in enumerate((0x6000, 0x7000, 0x8000))]
        assert L.coll_kv_fork(*ok, 0x4000, 0x5000, 2, *outs, NULL) == INVALID
    assert L.coll_kv_free(*ok[:6], NULL, 2, NULL) == INVALID


def test_compact_and_copy(L):
    assert L.coll_kv_compact_workspace_bytes(100) == 512 and L.coll_kv_compact_workspace_bytes(-1) == 0
    good = dict(table=0x1000, ref=0x2000, rows=4, width=8, N=100, moves=0x3000, most=50, count=0x4000, ws=0x10000,
                ws_bytes=512)
    for kw in (dict(table=NULL), dict(ref=NULL), dict(rows=-1), dict(width=-1), dict(N=-1), dict(moves=NULL),
               dict(most=49), dict(count=NULL), dict(ws=NULL), dict(ws=0x10010), dict(ws_bytes=511)):
        assert L.coll_kv_compact(*dict(good, **kw).values(), NULL) == INVALID, kw
    assert L.coll_kv_compact(*dict(good, rows=1 << 16, width=1 << 16).values(), NULL) == UNSUPPORTED
    good = dict(n=2, pools=P2, layers=3, N=100, page=4096, moves=0x3000, most=50, count=NULL)
    for kw in (dict(n=0), dict(n=17), dict(pools=NULL), dict(pools=t(0x1000, 0)), dict(moves=NULL), dict(most=-1),
               dict(layers=1 << 60), dict(page=1 << 60)):
        assert L.coll_kv_copy_pages(*dict(good, **kw).values(), NULL) == INVALID, kw
    for kw in (dict(layers=0), dict(N=0), dict(page=0), dict(most=0)):
        assert L.coll_kv_copy_pages(*dict(good, **kw).values(), NULL) == 0, kw


def test_binding_refuses_before_it_asks_the_library():
    bf = torch.bfloat16
    q, k = [torch.zeros(4, 4, 64, dtype=bf)], [torch.zeros(4, 2, 64, dtype=bf)]
    st = [torch.zeros(2, dtype=torch.int32)]
    with pytest.raises(ValueError, match="bf16 or fp16"):
        coll.attn_prompt([q[0].float()], k, k, q, st, st)
    with pytest.raises(ValueError, match="3 kv heads|kv heads"):
        coll.attn_prompt(q, [torch.zeros(4, 3, 64, dtype=bf)], k, q, st, st)
    with pytest.raises(ValueError, match="current GPU"):
        coll.attn_prompt(q, k, k, q, st, st)
    with pytest.raises(ValueError, match="contiguous"):
        coll.attn_prompt([q[0].transpose(0, 1)], k, k, q, st, st)
    with pytest.raises(ValueError, match="every rank"):
        coll.attn_prompt([q[0], q[0][:2]], k * 2, k * 2, q * 2, st * 2, st * 2)
    with pytest.raises(ValueError, match="pools are"):
        coll._pool_tables(k, k, bf, "attn_decode", 1)
    pool = [torch.zeros(3, 16, 2, 64, dtype=bf)]
    with pytest.raises(ValueError, match="current GPU"):
        coll.attn_decode(q, pool, pool, [torch.zeros(4, 3, dtype=torch.int32)], [torch.zeros(4, dtype=torch.int32)],
                         q, st[0])
    with pytest.raises(ValueError):
        coll.kv_fork(torch.zeros(4, 3, dtype=torch.int64), st[0], st[0], st[0], st[0], 16, st[0], st[0], st[0])
    with pytest.raises(ValueError, match="at least 2"):
        coll._kv_moves(torch.zeros(1, 2, dtype=torch.int32), st[0], 2, "kv_fork")
    with pytest.raises(ValueError, match="one shape|same shape|pools are"):
        coll.kv_copy_pages([torch.zeros(4, 3), torch.zeros(4, 2)], torch.zeros(1, 2, dtype=torch.int32))


def test_binding_wants_one_buffer_per_rank():
    bf = torch.bfloat16
    q, k = [torch.zeros(4, 4, 64, dtype=bf)], [torch.zeros(4, 2, 64, dtype=bf)]
    for call in (lambda: coll.attn_prompt(q, [], k, q, [], []), lambda: coll.attn_prompt([], k, k, q, [], []),
                 lambda: coll._rows_of_cache([], [], None, 1, "attn_decode", 1),
                 lambda: coll._ints([], (1,), "lens", 1), lambda: coll._each([], "starts", 1)):
        with pytest.raises(ValueError, match="rank"):
            call()


def test_a_plan_keeps_the_pointer_tables_it_converted():
    """The converted arguments hold the tables: their contents survive the lists
    they came from."""
    import gc
    a = (ctypes.c_void_p * 3)(11, 22, 33)
    kept = coll._as_c(a, ctypes.c_void_p)
    del a
    gc.collect()
    junk = [(ctypes.c_void_p * 3)(7, 7, 7) for _ in range(1000)]
    assert list((ctypes.c_void_p * 3).from_address(kept.value)) == [11, 22, 33] and junk
    assert coll._as_c(5, ctypes.c_int).value == 5 and coll._as_c(None, ctypes.c_void_p) is None
    assert coll._as_c(0x1234, ctypes.c_void_p).value == 0x1234
