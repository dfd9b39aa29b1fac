"""The paged cache's kernels when a wait of theirs runs out: they end, what their block had a part of is NaN, and the
rest is right.

The waits run out without a fault: test builds of the library (compiled here, into a temporary directory, never the
library the package loads) whose waits give up at once or after a few polls, while copies and products are in flight.
"""
import ctypes
import math
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


@pytest.fixture(scope="module", params=[0, 2])
def hasty(request, tmp_path_factory):
    """The library with waits of so many polls, and that number."""
    from speculative_decoding_verification_55_gb300.build import build_library
    out = tmp_path_factory.mktemp("hasty") / "libspecverify_hasty.so"
    build_library(force=True, out=out, extra_flags=[f"-DSV_SPIN_LIMIT={request.param}"])
    L = ctypes.CDLL(str(out))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.spec_verify_paged_attention.argtypes = [vp, i64, i64, vp, vp, vp, vp, ctypes.c_float, vp, vp, i32, i32, i32, vp,
                                              ctypes.c_size_t, vp]
    L.spec_verify_kv_weights.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32, vp]
    return L, request.param


def batch(sv, prefix, N, H, G, D, seed):
    """(q, cache, prefix_len) with the pages in order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = [-(-(n + N) // 16) for n in prefix]
    first = np.cumsum([0] + pages)
    table = np.zeros((len(prefix), max(pages)), np.int32)
    for b, p in enumerate(pages):
        table[b, :p] = first[b] + np.arange(p)
    def make(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    cache = sv.PagedCache(make(first[-1], H, 16, D), make(first[-1], H, 16, D), torch.from_numpy(table).cuda(),
                          torch.rand((int(first[-1]), H, 16), generator=g, device="cuda"))
    return make(len(prefix), N, H * G, D), cache, torch.tensor(prefix, dtype=torch.int32, device="cuda")


def bounded(f):
    t0 = time.monotonic()
    st = f()
    torch.cuda.synchronize()                   # returns: every wait is bounded
    assert st == 0 and time.monotonic() - t0 < 20


LONG = (9000, 30, 4000, 0, 777)
ATTEND = [                                     # prefix lengths, N, key heads, group, D
    (LONG, 1, 2, 4, 128), ((3000,) * 200, 1, 2, 4, 64), ((20,) * 900, 1, 2, 1, 64), (LONG, 4, 2, 4, 256),
    (LONG, 9, 2, 4, 128), ((3000,) * 100, 9, 2, 4, 64), ((20,) * 900, 17, 1, 1, 128), (LONG, 9, 1, 8, 256),
    (LONG, 31, 2, 8, 128), ((1600,) * 152, 31, 1, 8, 64), ((1600,) * 152, 31, 1, 8, 128),   # the latter: two query tiles
]


@pytest.mark.parametrize("prefix,N,H,G,D", ATTEND)
def test_attention_gives_up(sv, hasty, prefix, N, H, G, D):
    L, limit = hasty
    q, cache, n = batch(sv, prefix, N, H, G, D, N)
    B, Hq = len(prefix), H * G
    want, want_lse = sv.attend(q, cache, n)
    need = sv.spec_verify_paged_attention_workspace_size(N, Hq, cache)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        bounded(lambda: L.spec_verify_paged_attention(
            q.data_ptr(), q.stride(0), q.stride(1), cache.ref, n.data_ptr(), None, None, 1 / math.sqrt(D), out.data_ptr(),
            lse.data_ptr(), B, N, Hq, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
        lost = lse.isnan()
        assert torch.equal(out.isnan(), lost[..., None].expand_as(out))
        assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
        assert limit > 0 or lost.any()         # with no polls at all, some wait did run out
    got, got_lse = sv.attend(q, cache, n)      # the context and the workspace of the next call are usable
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


WEIGH = [                                      # prefix lengths, N, key heads, group, D, along a path
    (LONG, 1, 2, 4, 128, False), ((3000,) * 100, 9, 2, 4, 64, False), ((20,) * 900, 17, 1, 1, 128, True),
    (LONG, 9, 1, 8, 256, True), (LONG, 31, 2, 8, 128, False), ((900,) * 40, 40, 1, 16, 128, False),
    ((900,) * 40, 33, 1, 8, 256, True),
]


@pytest.mark.parametrize("prefix,N,H,G,D,along", WEIGH)
def test_weights_give_up(sv, hasty, prefix, N, H, G, D, along):
    L, limit = hasty
    q, cache, n = batch(sv, prefix, N, H, G, D, N)
    B, Hq = len(prefix), H * G
    path = torch.stack([torch.randperm(N) for _ in prefix]).sort(1)[0].to(torch.int32).cuda() if along else None
    num = torch.arange(B, dtype=torch.int32, device="cuda") % (N + 1)
    lse = torch.full((B, N, Hq), 5.0, device="cuda")
    before = cache.weight.clone()
    sv.spec_verify_kv_weights(q, lse, cache, n, num, path)
    want = cache.weight.clone()
    added = torch.zeros_like(want, dtype=torch.bool)       # entries that the call adds to
    for b, (k, m) in enumerate(zip(prefix, num.tolist())):
        for j in range(0, k + m if m else 0, 16):
            added[int(cache.page_table[b, j // 16]), :, :min(16, k + m - j)] = True
    for _ in range(5):
        cache.weight.copy_(before)
        bounded(lambda: L.spec_verify_kv_weights(
            q.data_ptr(), q.stride(0), q.stride(1), lse.data_ptr(), cache.ref, n.data_ptr(), num.data_ptr(),
            None if path is None else path.data_ptr(), 1 / math.sqrt(D), B, N, Hq,
            torch.cuda.current_stream().cuda_stream))
        lost = cache.weight.isnan()
        assert torch.equal(cache.weight[~lost], want[~lost]) and not (lost & ~added).any()
        assert limit > 0 or lost.any()
    cache.weight.copy_(before)
    sv.spec_verify_kv_weights(q, lse, cache, n, num, path)
    assert torch.equal(cache.weight, want)
