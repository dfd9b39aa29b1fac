"""The attention of rows that share fronts when a wait of its kernel runs out: it ends, what its block had a part of is
NaN, and the rest is right.

The waits run out without a fault: a test build of the library (compiled here, into a temporary directory, never the
library the package loads) whose waits give up at once, while copies and products are in flight.
"""
import ctypes
import math

import numpy as np
import pytest

from test_giveup_cache import bounded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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
    out = tmp_path_factory.mktemp("hasty") / "libspecverify_hasty.so"
    build_library(force=True, out=out, extra_flags=["-DSV_SPIN_LIMIT=0"])
    L = ctypes.CDLL(str(out))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.spec_verify_shared_attention.argtypes = [vp, i64, i64, vp, vp, vp, vp, i32, vp, vp, ctypes.c_float, vp, vp, i32, i32,
                                               i32, vp, ctypes.c_size_t, vp]
    return L


def batch(sv, fronts, rows, own, N, H, G, D, seed):
    """(q, cache, prefix_len, shared_len, group_start): len(fronts) groups of `rows` rows with `own` entries each (more than
    48 MB, or 12 of heads of 256, and 512 entries a row: by fronts)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, pages = len(fronts) * rows, -(-(own + N) // 16)
    table = np.zeros((B, max(fronts) // 16 + pages), np.int32)
    at = 0
    for k, f in enumerate(fronts):
        table[k * rows:(k + 1) * rows, :f // 16] = at + np.arange(f // 16)
        at += f // 16
        for b in range(k * rows, (k + 1) * rows):
            table[b, f // 16:f // 16 + pages] = at + np.arange(pages)
            at += pages
    def make(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    cache = sv.PagedCache(make(at, H, 16, D), make(at, H, 16, D), torch.from_numpy(table).cuda())
    common = torch.tensor(fronts, dtype=torch.int32, device="cuda").repeat_interleave(rows)
    start = torch.arange(0, B + 1, rows, dtype=torch.int32, device="cuda")
    return make(B, N, H * G, D), cache, common + own, common, start


@pytest.mark.parametrize("fronts,rows,own,N,H,G,D", [
    ((8000,), 64, 300, 1, 2, 4, 128), ((4000, 320, 0), 20, 150, 9, 2, 4, 128), ((1600, 1600), 130, 40, 31, 1, 2, 64),
    ((30000,), 3, 10, 1, 1, 8, 256), ((64,) * 40, 5, 500, 5, 2, 8, 64),
])
def test_shared_attention_gives_up(sv, hasty, fronts, rows, own, N, H, G, D):
    q, cache, n, common, start = batch(sv, fronts, rows, own, N, H, G, D, N)
    B, Hq, groups = q.shape[0], H * G, len(fronts)
    want, want_lse = sv.attend_shared(q, cache, n, common, start)
    assert bool(want.isfinite().all())
    need = sv.spec_verify_shared_attention_workspace_size(B, N, Hq, groups, cache)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        bounded(lambda: hasty.spec_verify_shared_attention(
            q.data_ptr(), q.stride(0), q.stride(1), cache.ref, n.data_ptr(), common.data_ptr(), start.data_ptr(), groups, None,
            None, 1 / math.sqrt(D), out.data_ptr(), lse.data_ptr(), B, N, Hq, ws.data_ptr(), need,
            torch.cuda.current_stream().cuda_stream))
        lost = lse.isnan()
        assert torch.equal(out.isnan(), lost[..., None].expand_as(out))
        assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
        assert lost.any()                      # with no polls at all, some wait did run out
    got, got_lse = sv.attend_shared(q, cache, n, common, start)   # the context is usable
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
