"""Shared attention: values of a front's last entries that are not finite; starts that do not ascend; groups
that hold nothing; the workspace of calls whose rows go by themselves."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged_cache_oracle as oracle
from test_paged_cache import Batch, cache_struct, check_attention, dev, host
from test_shared_attention import attend_shared, roomy, with_fronts

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("front", [640, 656])              # a whole tile at its end, and a part of one
@pytest.mark.parametrize("N,G,D,dtype", [(1, 4, 128, "bf16"), (3, 4, 64, "f16"), (9, 8, 128, "bf16"), (2, 4, 256, "bf16")])
def test_gpu_infinity_in_a_fronts_last_entry(sv, N, G, D, dtype, front, packed):
    """A front's last entry whose probability is 0 in fp32 and whose value is infinite: NaN, as by the paged attention. So
    are the entries before it; where the probability is not too small it is infinite."""
    a = Batch((700, 690, 720), N, 1, G, D, 16, dtype, seed=N, poison=False)
    common, call = with_fronts(a, (0, 3), (front,))
    a.q[:] = 1.0
    a.k.clamp_(-0.1, 0.1)
    for j, d in ((front - 1, 5), (front - 2, 7), (130, 9)):
        p, s = oracle.place(a.table, 0, j, 16)
        a.k[p, :, s] = -100.0                              # scores of -800 and less, the others above -2
        a.v[p, :, s, d] = math.inf
    for j, d in ((front - 1, 11), (front - 3, 13)):
        p, s = oracle.place(a.table, 0, j, 16)
        a.v[p, :, s, d] = math.inf
    p, s = oracle.place(a.table, 0, front - 3, 16)
    a.k[p, :, s] = 0.0
    num = np.array([N, max(N - 1, 1), N], np.int32)
    k, v, table = roomy(a, call, packed)
    cache = sv.PagedCache(k, v, dev(table))
    out, lse = sv.attend_shared(a.q, cache, dev(a.prefix), dev(common), dev((0, 3)), dev(num))
    ref, _ = sv.attend(a.q, cache, dev(a.prefix), dev(num))
    o, r = host(out), host(ref)
    assert np.array_equal(np.isnan(o), np.isnan(r)) and np.array_equal(np.isinf(o), np.isinf(r))
    for b in range(3):
        assert np.isnan(o[b, :num[b]][..., [5, 7, 9, 11]]).all() and (o[b, :num[b], :, 13] == math.inf).all()
        rest = np.delete(o[b, :num[b]], [5, 7, 9, 11, 13], axis=-1)
        assert np.isfinite(rest).all()
    assert np.isfinite(host(lse)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 3])
def test_gpu_starts_that_do_not_ascend_cost_nothing(sv, N):
    """Starts that name the whole batch again and again: all rows are in error, and the call is not worked on. (Worked on, it
    would take what 4000 groups of all rows take, over ten times the call's time.)"""
    B = 64
    a = Batch((2100,) * B, N, 2, 4, 128, 16, seed=1, poison=False)
    common, call = with_fronts(a, (0, B), (2048,))
    k, v, table = roomy(a, call)
    cache = sv.PagedCache(k, v, dev(table))
    args = dev(a.prefix), dev(common)
    good, bad = dev((0, B)), dev((0, B) * 4000 + (B,))

    def timed(start):
        best = math.inf
        for _ in range(5):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            t0.record()
            out, lse = sv.attend_shared(a.q, cache, *args, start)
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1))
        return best, out, lse
    t_good, out, lse = timed(good)
    want = sv.attend(a.q, cache, args[0])
    assert float((out.float() - want[0].float()).abs().max()) <= 4 * 2.0 ** -8 * 6
    t_bad, out, lse = timed(bad)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    assert t_bad <= 5 * t_good, (t_bad, t_good)
    again, lse = sv.attend_shared(a.q, cache, *args, good)             # the next call is as it should be
    assert float((again.float() - want[0].float()).abs().max()) <= 4 * 2.0 ** -8 * 6
    assert float((lse - want[1]).abs().max()) <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("N,G,D,B", [(9, 4, 128, 20), (1, 4, 64, 150), (2, 8, 256, 20)])
def test_gpu_a_large_group_among_empty_ones(sv, N, G, D, B, packed):
    """A caller with room for many groups: one that has all the rows, the others empty, before it and behind it."""
    rng = np.random.default_rng(B)
    prefix = 1024 + rng.integers(0, 60, B)
    a = Batch(prefix, N, 1, G, D, 16, seed=B, poison=False)
    start = (0,) * 30 + (B,) * 40
    common, call = with_fronts(a, (0, B), (1024,))
    num = rng.integers(0, N + 1, B).astype(np.int32)
    out, lse = attend_shared(sv, a, common, call, start, num, packed=packed)
    check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
@pytest.mark.parametrize("lone", [0, 5])
def test_gpu_empty_groups_cost_little(sv, lone):
    """A group of 64 rows, with 1000 empty ones behind it and without them: the same outputs, in no more than twice the time.
    (With a wait for each empty group it would be over three times.)"""
    B = 64
    a = Batch((2100,) * B, 3, 2, 4, 128, 16, seed=1, poison=False)
    common, call = with_fronts(a, (0, B - lone), (2048,))
    k, v, table = roomy(a, call)
    cache = sv.PagedCache(k, v, dev(table))
    args = dev(a.prefix), dev(common)
    starts = dev((0, B - lone)), dev((0,) + (B - lone,) * 1001)

    def timed(start):
        best = math.inf
        for _ in range(10):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            t0.record()
            out, lse = sv.attend_shared(a.q, cache, *args, start)
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1))
        return best, out, lse
    (alone, out, lse), (among, out2, lse2) = timed(starts[0]), timed(starts[1])
    check_attention(a, out, lse, a.prefix, np.full(B, 3), None)
    check_attention(a, out2, lse2, a.prefix, np.full(B, 3), None)
    assert among <= 2 * alone, (among, alone)


def test_workspace_of_rows_by_themselves():
    """More than a query tile's rows of a row's key head: the paged attention's workspace, and no more, is asked for."""
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    L = m.lib()
    shared, paged = L.spec_verify_shared_attention_workspace_size, L.spec_verify_paged_attention_workspace_size
    c = ctypes.byref(cache_struct(max_pages=4096, num_pages=1 << 20))
    for N, Hq in ((33, 32), (65, 32), (65, 16), (17, 64), (2, 1024)):          # 8 key heads
        assert shared(64, N, Hq, 3, c) == paged(N, Hq, c) > 0
    for N, Hq in ((32, 32), (64, 16), (16, 64), (1, 1024)):
        assert shared(64, N, Hq, 3, c) >= 2 * 64 * N * Hq * (128 * 4 + 8)
    c = ctypes.byref(cache_struct(max_pages=4096, num_pages=1 << 20, heads=10))          # 3 heads a key head: a tile of 126
    assert shared(64, 43, 30, 3, c) == paged(43, 30, c) and shared(64, 42, 30, 3, c) > paged(42, 30, c)
    for bad in ((0, 65, 32, 3), (64, 66, 32, 3), (64, 65, 30, 3), (1 << 20, 65, 32, 3), (64, 65, 32, 0)):
        assert shared(*bad, ctypes.byref(cache_struct())) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,D", [(33, 4, 128), (65, 2, 64), (17, 16, 256)])
def test_gpu_workspace_of_rows_by_themselves(sv, N, G, D):
    """It is enough: nothing behind it is written, whatever it held."""
    a = Batch((40, 0, 300), N, 1, G, D, 16, seed=4, poison=False)
    k, v, table = roomy(a, a.table)
    cache = sv.PagedCache(k, v, dev(table))
    need = sv.spec_verify_shared_attention_workspace_size(3, N, G, 1, cache)
    assert need == sv.spec_verify_paged_attention_workspace_size(N, G, cache)
    for fill in (0, 255):
        room = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(a.q.contiguous()), torch.empty((3, N, G), device="cuda")
        sv.spec_verify_shared_attention(a.q, cache, dev(a.prefix), dev(np.zeros(3)), dev((0, 3)), None, None, out, lse, room[:need])
        check_attention(a, out, lse, a.prefix, np.full(3, N), None)
        assert bool((room[need:] == fill).all())
