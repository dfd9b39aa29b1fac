"""Attention of rows that share the fronts of their contexts: refusals on the CPU, GPU parity against the fp64 oracle
(the paged attention's, on tables whose rows begin with the same pages).

By the room of the tables and the pool, and by a row's query rows, a call goes by fronts or by rows; the tests of fronts
give the batches room (roomy).

Tolerances as for the paged attention (test_paged_cache): its parts are joined in fp32 the same way, one more time.
"""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged_cache_oracle as oracle
from test_paged_cache import FAKE, Batch, cache_struct, check_attention, dev, host, random_tree

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------------------------------------
# Refusals (CPU: no call gets as far as the device)
# ------------------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def L():
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m.lib()


def status(L, cache, **kw):
    a = dict(q=FAKE + (4 << 20), rs=9 * 32 * 128, ts=32 * 128, pre=FAKE + (5 << 20), com=FAKE + (6 << 20),
             st=FAKE + (7 << 20), g=2, num=None, par=None, scale=0.1, out=FAKE + (8 << 20), lse=FAKE + (9 << 20), B=2, N=9,
             Hq=32, ws=FAKE + (10 << 20), wsb=1 << 30)
    a.update(kw)
    c = None if cache is None else ctypes.byref(cache)
    return L.spec_verify_shared_attention(a["q"], a["rs"], a["ts"], c, a["pre"], a["com"], a["st"], a["g"], a["num"],
                                          a["par"], a["scale"], a["out"], a["lse"], a["B"], a["N"], a["Hq"], a["ws"],
                                          a["wsb"], None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), 1), (dict(pre=None), 1), (dict(com=None), 1), (dict(st=None), 1), (dict(out=None), 1),
    (dict(B=0), 2), (dict(N=0), 2), (dict(N=66), 2), (dict(Hq=30), 2), (dict(g=0), 2), (dict(g=-1), 2),
    (dict(g=(1 << 20) + 1), 2), (dict(scale=0.0), 2), (dict(scale=math.nan), 2), (dict(rs=10 * 32 * 128), 2),
    (dict(B=1 << 20, Hq=32), 2),
    (dict(q=FAKE + (4 << 20) + 8), 5), (dict(com=FAKE + (6 << 20) + 2), 5), (dict(st=FAKE + (7 << 20) + 1), 5),
    (dict(num=FAKE + 2), 5), (dict(par=FAKE + 2), 5), (dict(out=FAKE + (8 << 20) + 8), 5), (dict(ws=FAKE + (10 << 20) + 128), 5),
    (dict(ws=None), 4), (dict(wsb=1 << 20), 4),
    (dict(out=FAKE + (6 << 20)), 9), (dict(out=FAKE + (7 << 20)), 9), (dict(lse=FAKE + (6 << 20)), 9),
    (dict(ws=FAKE + (7 << 20)), 9), (dict(lse=FAKE + (8 << 20)), 9),
])
def test_refusals(L, change, want):
    assert status(L, cache_struct(), **change) == want


def test_cache_refusals(L):
    assert status(L, None) == 1
    assert status(L, cache_struct(dtype=0)) == 3
    assert status(L, cache_struct(head_dim=96)) == 2
    assert status(L, cache_struct(k=FAKE + 8)) == 5


def test_workspace_size(L):
    f = L.spec_verify_shared_attention_workspace_size
    c = ctypes.byref(cache_struct())
    assert f(64, 9, 32, 3, c) >= 2 * 64 * 9 * 32 * (128 * 4 + 8) and f(64, 9, 32, 3, c) % 256 == 0
    for bad in ((0, 9, 32, 3), (64, 0, 32, 3), (64, 66, 32, 3), (64, 9, 30, 3), (1 << 20, 65, 32, 3), (64, 9, 32, 0)):
        assert f(*bad, c) == 0
    assert f(64, 9, 32, 3, None) == 0


def test_binding_refusals():
    import speculative_decoding_verification_55_gb300 as sv
    k = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    c = sv.PagedCache(k, k, torch.zeros((3, 2), dtype=torch.int32))
    n, two = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((3, 4, 8, 64), dtype=torch.bfloat16)
    out, ws = torch.zeros_like(q), torch.zeros(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        sv.attend_shared(q, c, n, n, two)
    with pytest.raises(ValueError, match="group_start"):
        sv.spec_verify_shared_attention(q, c, n, n, two[:1], None, None, out, None, ws)
    with pytest.raises(TypeError, match="group_start"):
        sv.spec_verify_shared_attention(q, c, n, n, two.long(), None, None, out, None, ws)
    with pytest.raises(ValueError, match="shared_len"):
        sv.spec_verify_shared_attention(q, c, n, two, two, None, None, out, None, ws)
    with pytest.raises(ValueError, match="follow one another"):
        sv.spec_verify_shared_attention(torch.zeros((3, 6, 8, 64), dtype=torch.bfloat16)[:, :4], c, n, n, two, None, None,
                                        out, None, ws)


# ------------------------------------------------------------------------------------------------
# GPU parity
# ------------------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


def with_fronts(a, start, fronts):
    """The rows of each group begin with the pages of its first row: (shared_len [B], a copy of the table)."""
    common = np.zeros(len(a.prefix), np.int32)
    for g, s in enumerate(fronts):
        rows = slice(start[g], start[g + 1])
        common[rows] = s
        if start[g] < start[g + 1]:
            a.table[rows, :s // a.S] = a.table[start[g], :s // a.S]
    return common, a.table.copy()


def roomy(a, table, packed=False):
    """(k, v, table) with pages behind the pool's and columns behind the table's, which nobody reads: room for more than the
    bytes of keys and values, and the 512 entries a row, up to which rows go by themselves; packed: and for more than the
    2^25 entries times query heads up to which the tokens that are used are not packed."""
    P, H, S, D = a.k.shape
    rows = a.q.shape[1] * a.q.shape[2] // H
    room = (49 if rows <= 64 else 257 if rows <= 96 else 641) << 20
    pages = max(-(-room // (len(a.prefix) * H * S * D * 4)), 513 // S + 1, P) + 1
    if packed:
        pages = max(pages, min(-(-(1 << 25) // (a.q[..., 0].numel() * S)) + 1, (1 << 20) // S))
    slots_first = a.k.stride(1) < a.k.stride(2)
    pools = []
    for x in (a.k, a.v):
        big = torch.full((pages, S, H, D) if slots_first else (pages, H, S, D), math.nan, dtype=a.t, device="cuda")
        big = big.transpose(1, 2) if slots_first else big
        big[:P] = x
        pools.append(big)
    wide = np.full((table.shape[0], max(pages, table.shape[1])), 1 << 30, np.int32)
    wide[:, :table.shape[1]] = table
    return pools[0], pools[1], wide


def attend_shared(sv, a, common, call, start, num=None, parents=None, scale=None, rows=False, packed=False):
    k, v, table = (a.k, a.v, call) if rows else roomy(a, call, packed)
    cache = sv.PagedCache(k, v, dev(table))
    return sv.attend_shared(a.q, cache, dev(a.prefix), dev(common), dev(start), dev(num), dev(parents), scale)


CASES = [
    # prefix lengths, starts, fronts, N, Hkv, group, D, page, dtype, nhd (more than a tile's query rows go by rows)
    ((16,), (0, 1), (16,), 1, 1, 1, 64, 16, "bf16", False),                      # a row of its own, nothing behind
    ((20, 16, 33, 48), (0, 4), (16,), 1, 2, 4, 128, 16, "bf16", False),
    ((200, 129, 128, 500), (0, 4), (128,), 1, 2, 4, 128, 64, "f16", True),
    ((0, 40, 50, 60, 7, 300, 310, 0), (1, 4, 4, 5, 7), (32, 16, 0, 288), 2, 2, 4, 128, 16, "bf16", True),
    ((40, 41, 42, 43, 44, 45), (0, 3, 6), (32, 16), 9, 2, 4, 128, 16, "f16", False),
    ((600, 555, 700), (0, 3), (512,), 5, 3, 7, 64, 64, "bf16", False),
    ((257, 300, 270), (0, 3), (256,), 4, 1, 16, 256, 32, "bf16", True),
    ((64, 150), (0, 2), (64,), 17, 2, 3, 256, 16, "f16", False),
    ((140, 300, 170), (0, 3), (128,), 31, 1, 8, 128, 16, "bf16", False),
    ((140, 300, 170, 128, 200), (0, 5), (128,), 31, 2, 2, 128, 16, "bf16", False),
    ((100, 80, 90, 95), (0, 3, 4), (64, 80), 64, 1, 1, 64, 16, "f16", True),
    ((300, 257, 600), (0, 3), (256,), 3, 2, 4, 128, 256, "bf16", False),
    ((600, 512, 530, 100), (0, 3), (512,), 8, 2, 4, 64, 128, "f16", True),
    ((390, 384, 500), (0, 3), (384,), 2, 1, 3, 256, 128, "bf16", True),
    ((210, 192, 250, 200), (0, 4), (192,), 9, 1, 8, 128, 16, "bf16", False),     # 72 query rows a row
    ((210, 192, 250), (0, 3), (192,), 8, 1, 16, 64, 32, "f16", True),            # 128
    ((130, 192, 128), (0, 3), (128,), 17, 1, 7, 256, 16, "bf16", False),         # 119
    ((530, 512), (0, 2), (512,), 65, 2, 2, 64, 128, "bf16", True),
    ((300, 257), (0, 2), (256,), 3, 1, 128, 128, 256, "f16", False),
    ((2100, 2049, 2500, 2048), (0, 4), (2048,), 2, 1, 5, 128, 16, "bf16", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("by", ["fronts", "packed", "rows"])
@pytest.mark.parametrize("prefix,start,fronts,N,H,G,D,S,dtype,nhd", CASES)
def test_gpu_shared(sv, prefix, start, fronts, N, H, G, D, S, dtype, nhd, by):
    rows, packed = by == "rows", by == "packed"
    rng = np.random.default_rng(N * 31 + D)
    a = Batch(prefix, N, H, G, D, S, dtype, nhd, seed=N + D, poison=False)
    B = len(prefix)
    common, call = with_fronts(a, start, fronts)
    num = rng.integers(0, N + 1, B).astype(np.int32)
    num[-1] = N
    out, lse = attend_shared(sv, a, common, call, start, num, rows=rows, packed=packed)
    check_attention(a, out, lse, a.prefix, num, None)
    again, lse2 = attend_shared(sv, a, common, call, start, num, rows=rows, packed=packed)
    assert torch.equal(again, out) and torch.equal(lse2, lse)          # the same call, the same bits
    tree = random_tree(rng, B, N)
    out, lse = attend_shared(sv, a, common, call, start, num if packed else None, tree, 0.25, rows=rows, packed=packed)
    check_attention(a, out, lse, a.prefix, num if packed else np.full(B, N), tree, 0.25)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype,N,G", [(64, "bf16", 1, 4), (128, "f16", 3, 5), (256, "bf16", 2, 2)])
def test_gpu_many_groups(sv, D, dtype, N, G):
    """More rows and groups than the GPU holds blocks, groups of many sizes, some empty, some rows in none."""
    rng = np.random.default_rng(D)
    start = np.sort(rng.integers(3, 395, 90)).astype(np.int32)
    fronts = rng.integers(0, 6, 89) * 16
    prefix = rng.integers(0, 30, 400)
    for g in range(89):
        prefix[start[g]:start[g + 1]] += fronts[g]
    a = Batch(prefix, N, 1, G, D, 16, dtype, seed=D, poison=False)
    common, call = with_fronts(a, start, fronts)
    num = rng.integers(0, N + 1, 400).astype(np.int32)
    for packed in (False, True):
        out, lse = attend_shared(sv, a, common, call, start, num, packed=packed)
        check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,D,B,front", [(1, 4, 128, 70, 3008), (9, 4, 64, 33, 1600), (5, 8, 256, 20, 1024), (1, 1, 128, 3, 9008)])
def test_gpu_large_groups(sv, N, G, D, B, front):
    """More query rows a group than one query tile or two have, over fronts that many blocks share."""
    rng = np.random.default_rng(B)
    prefix = front + rng.integers(0, 60, B)
    a = Batch(prefix, N, 1, G, D, 16, seed=B, poison=False)
    common, call = with_fronts(a, (0, B), (front,))
    num = rng.integers(0, N + 1, B).astype(np.int32)
    tree = random_tree(rng, B, N)
    for parents, packed in ((None, False), (tree, False), (None, True), (tree, True)):
        out, lse = attend_shared(sv, a, common, call, (0, B), num, parents, packed=packed)
        check_attention(a, out, lse, a.prefix, num, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 8), (2, 3)])
def test_gpu_a_very_large_group(sv, N, G):
    """Thousands of rows of one group, some without tokens, against the paged attention on the same tables."""
    rng = np.random.default_rng(N)
    B = 4000
    prefix = 48 + rng.integers(0, 20, B)
    a = Batch(prefix, N, 2, G, 64, 16, seed=B, poison=False, extra=40)
    common, call = with_fronts(a, (0, B), (48,))
    num = rng.integers(0, N + 1, B).astype(np.int32)
    out, lse = attend_shared(sv, a, common, call, (0, B), num)
    ref, rlse = sv.attend(a.q, a.cache(sv, weight=False), dev(a.prefix), dev(num))
    # Each is within half a step of the probabilities and of the output of the exact one, whose values are below 8.
    assert float((out.float() - ref.float()).abs().max()) <= 4 * 2.0 ** -8 * 8
    assert float((lse - rlse).abs().max()) <= 2 * (66 * 2.0 ** -24 * 600 + 1e-6)
    pick = [0, 1, 1999, 3998, 3999]
    b = Batch.__new__(Batch)
    b.__dict__ = dict(a.__dict__, q=a.q[pick], table=a.table[pick])
    check_attention(b, out[pick], lse[pick], a.prefix[pick], num[pick], None)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,packed", [(5, 1, False), (1, 4, False), (1, 4, True)])
def test_gpu_query_strides(sv, B, N, packed):
    """One token a row, or one row: any distance of the rows, and of the tokens, will do."""
    a = Batch((70,) * B, N, 2, 4, 128, 16, seed=2, poison=False)
    common, call = with_fronts(a, (0, B), (64,))
    wide = torch.zeros((B, 3 * N, a.q.shape[2], 128), dtype=a.q.dtype, device="cuda")
    if B > 1:
        wide[:, :1] = a.q
        a.q = wide[:, :1]
    else:
        wide[:, ::3] = a.q
        a.q = wide[:, ::3]
    num = np.full(B, N)
    out, lse = attend_shared(sv, a, common, call, (0, B), num, packed=packed)
    check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
def test_gpu_far_pages(sv):
    """Offsets past 32 bits: pages that lie over 2^32 bytes into the cache, the front's among them."""
    S, H, D, P = 16, 8, 128, (1 << 17) + 30                 # 4.3 GB of keys, as much of values
    a = Batch((50, 40, 33), 3, H, 2, D, S, seed=2, poison=False)
    common, call = with_fronts(a, (0, 3), (32,))
    big = [torch.zeros((P, H, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    n = len(a.k)
    for x, y in zip(big, (a.k, a.v)):
        x[P - n:] = y
    table = np.full((3, 4000), 1 << 30, np.int64)           # (room for fronts)
    table[:, :call.shape[1]] = call.astype(np.int64) + P - n
    c = sv.PagedCache(*big, dev(np.minimum(table, 1 << 30)))
    out, lse = sv.attend_shared(a.q, c, dev(a.prefix), dev(common), dev((0, 3)))
    check_attention(a, out, lse, a.prefix, np.array([3, 3, 3]), None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gpu_scores_of_tens_of_millions(sv, dtype):
    """Equal keys whose scores are in the tens of millions, in the front and behind it: the mean of the values."""
    a = Batch((640, 700, 655), 3, 2, 4, 128, 16, dtype, seed=6, poison=False)
    common, call = with_fronts(a, (0, 3), (640,))
    a.q.fill_(600.0)
    a.k.fill_(500.0)
    out, lse = attend_shared(sv, a, common, call, (0, 3), None, None, 1.0)
    v = host(a.v)
    for b in range(3):
        for i in range(3):
            e = oracle.entries(v, a.table, b, int(a.prefix[b]) + i + 1).mean(1)        # [heads, D]
            want = np.repeat(e, 4, 0)
            # A mean of values below 6 by equal weights: half a step of the output, and fp32 sums.
            assert np.abs(host(out)[b, i] - want).max() <= torch.finfo(a.t).eps / 2 * 6 + 1e-4
    assert np.abs(host(lse) / (600.0 * 500 * 128) - 1).max() <= 1e-6


@pytest.mark.gpu
def test_gpu_no_fronts(sv):
    """Groups without a front, and rows in no group: the paged attention."""
    a = Batch((40, 0, 130, 65), 3, 2, 4, 128, 16, seed=3)
    num = np.array([3, 1, 0, 2], np.int32)
    for start in ((0, 4), (2, 2), (1, 3, 3)):
        out, lse = attend_shared(sv, a, np.zeros(4, np.int32), a.table, start, num)
        check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_gpu_row_errors(sv, packed):
    """A row in error gets NaN, the others what they should; a front's bad page concerns all its rows."""
    prefix = np.array([40, 40, 40, 40, 40, 40, 40], np.int32)
    a = Batch(prefix, 3, 2, 4, 128, 16, seed=4, poison=False)
    start = (0, 6, 7)
    common, call = with_fronts(a, start, (32, 32))
    num = np.array([3, 4, -1, 3, 2, 3, 3], np.int32)
    bad = prefix.copy()
    bad[3] = 16                                # shorter than what it shares
    common[4] = 16                             # another front than its group's
    common[5] = 0                              # on its own
    call[5] = a.table[5]
    k, v, table = roomy(a, call, packed)
    cache = sv.PagedCache(k, v, dev(table))
    out, lse = sv.attend_shared(a.q, cache, dev(bad), dev(common), dev(start), dev(num))
    assert np.isnan(host(out)[[1, 2, 3, 4]]).all() and np.isnan(host(lse)[[1, 2, 3, 4]]).all()
    good = [0, 5, 6]
    for b in (1, 2, 3, 4):                     # (for the oracle rows without tokens)
        num[b] = 0
    out[[1, 2, 3, 4]], lse[[1, 2, 3, 4]] = 0, 0
    check_attention(a, out, lse, a.prefix, num, None)
    num = np.array([3, 1, 2, 3, 0, 3, 2], np.int32)
    common, call = with_fronts(a, start, (32, 32))
    call[:6, 1] = 1 << 29                      # in the first group's front
    out, lse = attend_shared(sv, a, common, call, start, num, packed=packed)
    o, z = host(out), host(lse)
    for b in range(6):
        assert np.isnan(o[b, :num[b]]).all() and np.isnan(z[b, :num[b]]).all()
        assert (o[b, num[b]:] == 0).all() and (z[b, num[b]:] == 0).all()
    assert np.isfinite(o[6]).all()
    common, call = with_fronts(a, start, (32, 32))
    call[2, 2] = -1                            # in the row's own entries
    out, lse = attend_shared(sv, a, common, call, start, num, packed=packed)
    o = host(out)
    assert np.isnan(o[2, :num[2]]).all() and np.isfinite(o[[0, 1, 3, 4, 5, 6]]).all()
    tree = np.tile(np.array([[-1, 0, 1]], np.int32), (7, 1))
    tree[1, 0] = 0
    call[2] = a.table[2]
    out, _ = attend_shared(sv, a, common, call, start, num, tree, packed=packed)
    assert np.isnan(host(out)[1, :1]).all() and np.isfinite(host(out)[[0, 2, 3, 4, 5, 6]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("start", [(0, 5, 3, 7), (-1, 7), (0, 8), (2, 1)])
def test_gpu_groups_in_error(sv, start):
    a = Batch((40,) * 7, 2, 1, 4, 64, 16, seed=4, poison=False)
    out, lse = attend_shared(sv, a, np.full(7, 32, np.int32), a.table, start)
    assert np.isnan(host(out)).all() and np.isnan(host(lse)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("common", [8, 24, -16, 48, 1 << 30, -(1 << 31)])
def test_gpu_fronts_in_error(sv, common):
    """Not whole pages, below zero, longer than the rows."""
    a = Batch((40,) * 4, 2, 1, 4, 64, 16, seed=4, poison=False)
    out, lse = attend_shared(sv, a, np.array([common] * 3 + [0], np.int32), a.table, (0, 3))
    assert np.isnan(host(out)[:3]).all() and np.isnan(host(lse)[:3]).all() and np.isfinite(host(out)[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,rows", [(2, 4, True), (31, 8, False)])
def test_gpu_by_rows(sv, N, G, rows):
    """Little room, or many query rows: shared_len and group_start are not read, the outputs are the paged attention's."""
    a = Batch((40, 0, 300, 77), N, 1, G, 64, 16, seed=4, poison=False)
    num = np.array([N, 1, N - 1, 0], np.int32)
    out, lse = attend_shared(sv, a, np.full(4, -7, np.int32), a.table, (3, 9), num, rows=rows)
    k, v, table = (a.k, a.v, a.table) if rows else roomy(a, a.table)
    want, want_lse = sv.attend(a.q, sv.PagedCache(k, v, dev(table)), dev(a.prefix), dev(num))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,packed", [(3, 2, False), (9, 4, False), (9, 8, False), (3, 2, True), (9, 4, True)])
def test_gpu_unattended_values_have_no_part(sv, N, G, packed):
    """Infinities and NaN behind the last entry, in tokens that a token does not attend and in queries without a token;
    an infinity in the front reaches every row."""
    a = Batch((70, 64, 66, 129), N, 2, G, 128, 16, seed=3)                # unused slots hold NaN
    common = np.full(4, 64, np.int32)
    for b in range(1, 4):
        a.table[b, :4] = a.table[0, :4]
    num = np.array([N - 1, N, N, N], np.int32)
    q = a.q.clone()
    q[0, N - 1] = math.nan
    p, s = oracle.place(a.table, 0, 70 + N - 1, 16)
    a.v[p, :, s] = math.inf
    p, s = oracle.place(a.table, 1, 64 + N - 1, 16)
    a.v[p, :, s, 1::2] = math.inf
    k, v, table = roomy(a, a.table, packed)
    cache = sv.PagedCache(k, v, dev(table))
    out, lse = sv.attend_shared(q, cache, dev(a.prefix), dev(common), dev((0, 4)), dev(num))
    o = host(out)
    assert np.isfinite(o[0]).all() and np.isfinite(o[2:]).all() and np.isfinite(o[1, :N - 1]).all()
    assert np.isinf(o[1, N - 1][:, 1::2]).all() and np.isfinite(host(lse)).all()
    ref, _ = sv.attend(q, cache, dev(a.prefix), dev(num))
    r = host(ref)
    fine = np.isfinite(r)
    assert np.abs(o[fine] - r[fine]).max() <= 2.0 ** -7 * 4
    v[a.table[0, 3], 0, 15, 5] = math.inf                               # the front's last entry
    out, _ = sv.attend_shared(q, cache, dev(a.prefix), dev(common), dev((0, 4)), dev(num))
    o = host(out)
    for b in range(4):
        assert np.isinf(o[b, :num[b], :G, 5]).all() and np.isfinite(o[b, :num[b] - 1, G:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_gpu_captured_and_streams(sv, packed):
    """A graph replayed on new contents; calls on two streams at once; a stream given; a workspace of any contents."""
    a = Batch((300, 290, 310, 77), 5, 2, 4, 128, 16, seed=8, poison=False)
    start = (0, 3)
    common, call = with_fronts(a, start, (256,))
    k, v, call = roomy(a, call, packed)
    cache = sv.PagedCache(k, v, dev(call))
    num = np.array([5, 3, 0, 4], np.int32) if packed else np.full(4, 5, np.int32)
    args = [dev(a.prefix), dev(common), dev(start), dev(num) if packed else None]
    want, want_lse = sv.attend_shared(a.q, cache, *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = sv.attend_shared(a.q, cache, *args)
    other = torch.cuda.Stream()
    for front in (256, 0, 128):
        args[1].copy_(dev(np.where(common > 0, front, 0)))
        if packed:                             # other lengths than the captured ones
            num = np.roll(num, 1)
            args[3].copy_(dev(num))
        graph.replay()
        check_attention(a, out, lse, a.prefix, num, None)
    args[1].copy_(dev(common))
    want, want_lse = sv.attend_shared(a.q, cache, *args)
    torch.cuda.synchronize()
    results = []
    for _ in range(20):
        results.append(sv.attend_shared(a.q, cache, *args))
        results.append(sv.attend_shared(a.q, cache, *args, stream=other))
    torch.cuda.synchronize()
    for o, z in results:
        assert torch.equal(o, want) and torch.equal(z, want_lse)
    need = sv.spec_verify_shared_attention_workspace_size(4, 5, 8, 1, cache)
    for fill in (0, 255):
        room = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)
        sv.spec_verify_shared_attention(a.q, cache, *args, None, out, None, room[:need])
        assert torch.equal(out, want) and bool((room[need:] == fill).all())


@pytest.mark.gpu
def test_gpu_a_round_of_one_prompt(sv):
    """Append, shared attention, verification of shaped logits, counts: rounds of a batch on one prompt, against the same
    rounds on pages of each row's own with the paged attention."""
    B, N, H, G, D, S, V = 12, 5, 2, 4, 64, 16, 512
    g = torch.Generator(device="cuda").manual_seed(4)
    front, rows = 96, 700                      # (room for fronts to be worth it)
    table = torch.zeros((B, rows), dtype=torch.int32, device="cuda")
    table[:, :6] = torch.arange(6, device="cuda")
    table[:, 6:] = 6 + torch.arange(B * (rows - 6), device="cuda").view(B, -1)
    own = torch.arange(B * rows, device="cuda", dtype=torch.int32).view(B, rows)
    k, v = (torch.randn((6 + B * (rows - 6), H, S, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    shared = sv.PagedCache(k, v, table)
    apart = sv.PagedCache(k[table.long()].flatten(0, 1).contiguous(), v[table.long()].flatten(0, 1).contiguous(), own)
    n = torch.full((B,), front + 3, dtype=torch.int32, device="cuda")
    common = torch.full((B,), front, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    head = torch.randn((H * G * D, V), generator=g, device="cuda").to(torch.bfloat16) * 0.3
    counts = torch.zeros((B, V), dtype=torch.int16, device="cuda")
    counts_apart = counts.clone()
    penalty = torch.full((B,), 1.3, device="cuda")
    for _ in range(4):
        qkv = torch.randn((B, N, H * G + 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        drafts = torch.randint(0, V, (B, N - 1), generator=g, device="cuda", dtype=torch.int32)
        draft = torch.randn((B, N - 1, V), generator=g, device="cuda").to(torch.bfloat16)
        u = torch.rand((B, N + 1), generator=g, device="cuda")
        ends = []
        for cache, c, f in ((shared, counts, lambda *x: sv.attend_shared(x[0], x[1], x[2], common, start)),
                            (apart, counts_apart, sv.attend)):
            sv.spec_verify_kv_append(qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:], cache, n)
            out, lse = f(qkv[:, :, :H * G], cache, n)
            logits = torch.matmul(out.flatten(2), head)
            logits = torch.round(logits.float()).to(torch.bfloat16)        # (what two roundings of out differ in)
            d = draft.clone()
            sv.spec_verify_shape_logits(logits, None, drafts, None, c, penalty)
            sv.spec_verify_shape_logits(d, None, drafts, None, c, penalty)
            tokens, num, _ = sv.verify(logits, d, drafts, None, torch.ones(B, device="cuda"), u)
            sv.spec_verify_count_tokens(tokens, num, c)
            ends.append((out.float(), lse, num))
        (o1, z1, m1), (o2, z2, m2) = ends
        assert int(m1.min()) >= 1
        assert float((o1 - o2).abs().max()) <= 2.0 ** -7 * float(o2.abs().max()) and float((z1 - z2).abs().max()) <= 1e-5
        length = torch.empty_like(n)
        sv.spec_verify_kv_rollback(n, None, m1, None, length, None, gamma_max=N - 1)
        counts_apart.copy_(counts)
        n = length
