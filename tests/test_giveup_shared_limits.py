"""The attention of rows that share fronts when a wait of its kernel runs out, at several limits of the waits: over all of
them some rows are lost and some are not; those that are not are right.

A wait of limit 0 still asks its barrier once (which may take a while, and may succeed), so which blocks are lost is a matter
of time: the sizes here have rows of many blocks, and what happened is counted over all calls. Test builds of the library,
compiled into a temporary directory, as in test_giveup_shared.
"""
import ctypes
import math

import pytest

from test_giveup_cache import bounded
from test_giveup_shared import batch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LIMITS = [0, 2, 20]
SIZES = [                                      # fronts, rows a group, own entries, N, key heads, group, D
    ((64,) * 60, 5, 500, 5, 2, 8, 64), ((0,) * 3 + (128,) * 3, 60, 400, 2, 2, 4, 128), ((16,) * 300, 2, 60, 1, 4, 4, 128),
    ((512,) * 8, 4, 900, 2, 1, 8, 256),
]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    from speculative_decoding_verification_55_gb300.build import build_library
    libs = {}
    for limit in LIMITS:
        out = tmp_path_factory.mktemp("hasty") / f"libspecverify_{limit}.so"
        build_library(force=True, out=out, extra_flags=[f"-DSV_SPIN_LIMIT={limit}"])
        L = ctypes.CDLL(str(out))
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.spec_verify_shared_attention.argtypes = [vp, i64, i64, vp, vp, vp, vp, i32, vp, vp, ctypes.c_float, vp, vp, i32, i32,
                                                   i32, vp, ctypes.c_size_t, vp]
        libs[limit] = L
    return libs


def test_lost_rows_and_others(sv, hasty):
    lost_rows = right_rows = both = 0
    for fronts, rows, own, N, H, G, D in SIZES:
        q, cache, n, common, start = batch(sv, fronts, rows, own, N, H, G, D, N)
        num = 1 + torch.arange(q.shape[0], dtype=torch.int32, device="cuda") % N
        B, Hq, groups = q.shape[0], H * G, len(fronts)
        need = sv.spec_verify_shared_attention_workspace_size(B, N, Hq, groups, cache)
        ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
        for lengths in (None, num):
            want, want_lse = sv.attend_shared(q, cache, n, common, start, lengths)
            assert bool(want.isfinite().all())
            for limit in LIMITS:
                for _ in range(4):
                    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
                    bounded(lambda: hasty[limit].spec_verify_shared_attention(
                        q.data_ptr(), q.stride(0), q.stride(1), cache.ref, n.data_ptr(), common.data_ptr(), start.data_ptr(),
                        groups, None if lengths is None else lengths.data_ptr(), None, 1 / math.sqrt(D), out.data_ptr(),
                        lse.data_ptr(), B, N, Hq, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
                    lost = lse.isnan()
                    assert torch.equal(out.isnan(), lost[..., None].expand_as(out))
                    assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
                    used = lost if lengths is None else lost[torch.arange(N, device="cuda")[None] < num[:, None]]
                    lost_rows, right_rows = lost_rows + int(used.sum()), right_rows + int((~used).sum())
                    both += bool(used.any()) and not bool(used.all())
            got, got_lse = sv.attend_shared(q, cache, n, common, start, lengths)   # the context is usable
            assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    print(f"lost {lost_rows}, right {right_rows}, calls with both {both}")
    assert lost_rows > 0 and right_rows > 0 and both > 0
