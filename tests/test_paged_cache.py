"""The paged cache of a round: oracle pins and refusals on the CPU, GPU parity of the append, the
attention, the attention weights and the eviction against the fp64 oracle.

Tolerances. A probability is rounded to the cache's type once (half a step, e = finfo.eps / 2) and the
output once, so |out - exact| <= e (sum p|v| + |out|) plus fp32 arithmetic. A score is a sum of D
products in fp32, off by at most (D + 2) 2^-24 sum |q k| scale, then an exponential of relative error
2^-22 and, for lse, a logarithm of as much.
"""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged_cache_oracle as oracle

torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------
# Oracle pins (CPU)
# ------------------------------------------------------------------------------------------------

def small(rng, B=2, N=4, H=2, G=2, D=8, S=4, n=(5, 0), pages=9):
    """A batch in NumPy: q, k, v, table, prefix (every row has room for N more entries)."""
    q = rng.standard_normal((B, N, H * G, D))
    k, v = rng.standard_normal((2, pages, H, S, D))
    table = rng.permutation(pages)[:B * (pages // B)].reshape(B, -1).astype(np.int32)
    return q, k, v, table, np.array(n, np.int32)


def test_oracle_attention_pins():
    rng = np.random.default_rng(1)
    q, k, v, table, n = small(rng)
    num = np.array([4, 4])
    out, lse, _ = oracle.attention(q, k, v, table, n, num, None, 0.3)
    # A row's first token on an empty cache attends itself alone: its own value, its own score.
    page, slot = oracle.place(table, 1, 0, 4)
    assert np.allclose(out[1, 0, 3], v[page, 1, slot])
    assert np.isclose(lse[1, 0, 3], 0.3 * q[1, 0, 3] @ k[page, 1, slot])
    # Equal keys give the mean of the values.
    same, _, _ = oracle.attention(q, np.ones_like(k), v, table, n, num, None, 0.3)
    assert np.allclose(same[0, 2, 0], oracle.entries(v, table, 0, 8)[0].mean(0))
    # A chain is the tree whose parents are the tokens before.
    chain = np.array([[-1, 0, 1, 2]] * 2)
    again, _, _ = oracle.attention(q, k, v, table, n, num, chain, 0.3)
    assert np.allclose(again, out)
    # In a star every leaf attends the root and itself.
    star = np.array([[-1, 0, 0, 0]] * 2)
    assert oracle.attended(5, 4, 3, star[0]) == [0, 1, 2, 3, 4, 5, 8]


def test_oracle_weight_pins():
    """The softmax probabilities of a token sum to 1: the added weight is tokens times heads."""
    rng = np.random.default_rng(2)
    q, k, v, table, n = small(rng)
    num = np.array([3, 2])
    _, lse, _ = oracle.attention(q, k, v, table, n, np.array([4, 4]), None, 0.3)
    w = oracle.weights(q, lse, k, np.zeros(k.shape[:3]), table, n, num, None, 0.3)
    assert np.isclose(w.sum(), (3 + 2) * 4)
    # Kept path [0, 2] of a star, appended again as a chain, is what token 2 saw in the tree.
    star, path = np.array([[-1, 0, 0, 0]] * 2), np.array([[0, 2, -1, -1]] * 2)
    _, lse, _ = oracle.attention(q, k, v, table, n, np.array([4, 4]), star, 0.3)
    kn = np.stack([oracle.entries(k, table, b, n[b] + 4)[:, n[b]:].swapaxes(0, 1) for b in range(2)])
    k2, _, _, _ = oracle.append(k, v, None, kn, kn, table, n, np.array([2, 2]), path)
    w = oracle.weights(q, lse, k2, np.zeros(k.shape[:3]), table, n, np.array([2, 2]), path, 0.3)
    assert np.isclose(w.sum(), (2 + 2) * 4)


def test_oracle_evict_by_hand():
    w = np.array([3.0, 1.0, 2.0, 1.0, 2.0, 0.0, 9.0])
    assert oracle.kept_entries(w, 4, 1) == [0, 2, 4, 6]
    assert oracle.kept_entries(w, 5, 1) == [0, 1, 2, 4, 6]     # of the equal ones the first
    assert oracle.kept_entries(w, 3, 3) == [4, 5, 6]
    assert oracle.kept_entries(w, 1, 0) == [6]
    assert oracle.kept_entries(np.array([1.0, np.nan, np.inf]), 2, 0) == [1, 2]
    assert oracle.kept_entries(np.array([-0.0, 0.0, -1.0]), 1, 0) == [0]


# ------------------------------------------------------------------------------------------------
# Refusals (CPU: no call gets as far as the device)
# ------------------------------------------------------------------------------------------------

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m.lib()


def cache_struct(**kw):
    from speculative_decoding_verification_55_gb300._cache import _CacheStruct
    a = dict(k=FAKE, v=FAKE + (1 << 20), weight=FAKE + (2 << 20), page_table=FAKE + (3 << 20),
             page_stride=8 * 16 * 128, head_stride=16 * 128, slot_stride=128, num_pages=7,
             page_size=16, max_pages=5, heads=8, head_dim=128, dtype=1)
    a.update(kw)
    return _CacheStruct(*(a[f[0]] for f in _CacheStruct._fields_))


def calls(L, cache, **kw):
    """Status of each of the four calls for this cache and these arguments, by name."""
    a = dict(q=FAKE + (4 << 20), rs=9 * 32 * 128, ts=32 * 128, pre=FAKE + (5 << 20), num=None,
             par=None, scale=0.1, out=FAKE + (6 << 20), lse=FAKE + (7 << 20), B=2, N=9, Hq=32,
             ws=FAKE + (8 << 20), wsb=1 << 30, budget=8, recent=2, olen=FAKE + (9 << 20))
    a.update(kw)
    c = None if cache is None else ctypes.byref(cache)
    return {
        "attend": L.spec_verify_paged_attention(a["q"], a["rs"], a["ts"], c, a["pre"], a["num"],
                                                a["par"], a["scale"], a["out"], a["lse"], a["B"],
                                                a["N"], a["Hq"], a["ws"], a["wsb"], None),
        "weigh": L.spec_verify_kv_weights(a["q"], a["rs"], a["ts"], a["lse"], c, a["pre"], a["num"],
                                          a["par"], a["scale"], a["B"], a["N"], a["Hq"], None),
        "append": L.spec_verify_kv_append(a["q"], a["q"], a["rs"], a["ts"], c, a["pre"], a["num"],
                                          a["par"], a["olen"], a["B"], a["N"], None),
        "evict": L.spec_verify_kv_evict(c, a["pre"], a["budget"], a["recent"], a["olen"], a["B"], None),
    }


@pytest.mark.parametrize("change,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(page_table=None), 1),
    (dict(dtype=0), 3), (dict(dtype=7), 3),
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(page_size=8), 2), (dict(page_size=24), 2),
    (dict(page_size=512), 2), (dict(num_pages=0), 2), (dict(max_pages=0), 2), (dict(heads=0), 2),
    (dict(max_pages=(1 << 16) + 1), 2),               # more than 1048576 entries a row
    (dict(slot_stride=64), 2), (dict(head_stride=8), 2), (dict(page_stride=-128), 2),
    (dict(page_stride=1 << 40), 2),
    (dict(slot_stride=132), 5), (dict(page_stride=8 * 16 * 128 + 4), 5), (dict(k=FAKE + 8), 5),
    (dict(v=FAKE + 2), 5), (dict(page_table=FAKE + 2), 5), (dict(weight=FAKE + 4), 5),
])
def test_cache_refusals(L, change, status):
    got = calls(L, cache_struct(**change))
    assert set(got.values()) == {status}, got


def test_argument_refusals(L):
    c = cache_struct()
    assert set(calls(L, None).values()) == {1}
    assert set(calls(L, c, B=0).values()) == {2}
    assert set(calls(L, c, pre=None).values()) == {1}
    assert set(calls(L, c, pre=FAKE + 2).values()) == {5}
    for n in (0, 66):
        got = calls(L, c, N=n)
        assert (got["attend"], got["weigh"], got["append"]) == (2, 2, 2)
    for change, status in ((dict(q=None), 1), (dict(q=FAKE + 8), 5), (dict(ts=32 * 128 + 4), 5),
                           (dict(rs=-8), 2), (dict(ts=8), 2), (dict(num=FAKE + 1), 5),
                           (dict(par=FAKE + 2), 5)):
        got = calls(L, c, **change)
        assert (got["attend"], got["weigh"], got["append"]) == (status,) * 3, (change, got)
    for change, status in ((dict(Hq=0), 2), (dict(Hq=30), 2), (dict(Hq=1024 + 8), 2), (dict(scale=0.0), 2),
                           (dict(scale=-1.0), 2), (dict(scale=math.inf), 2), (dict(scale=math.nan), 2)):
        got = calls(L, c, **change)
        assert (got["attend"], got["weigh"]) == (status,) * 2, (change, got)
    got = calls(L, cache_struct(heads=4), Hq=1024, ts=1024 * 128, rs=9 * 1024 * 128)     # 256 heads a key head
    assert (got["attend"], got["weigh"]) == (2, 2)
    assert calls(L, c, out=None)["attend"] == 1
    assert calls(L, c, out=FAKE + 8)["attend"] == 5
    assert calls(L, c, lse=None)["weigh"] == 1
    assert calls(L, c, lse=FAKE + 2)["weigh"] == 5
    assert calls(L, c, ws=None)["attend"] == 4
    assert calls(L, c, wsb=64)["attend"] == 4
    assert calls(L, c, ws=FAKE + 128)["attend"] == 5
    assert calls(L, c, budget=0)["evict"] == 2
    assert calls(L, c, recent=-1)["evict"] == 2
    assert calls(L, c, recent=9)["evict"] == 2
    assert calls(L, c, olen=None)["evict"] == 1
    assert calls(L, c, olen=FAKE + (5 << 20))["evict"] == 9      # SV_ERR_OVERLAP: the lengths
    assert calls(L, c, olen=FAKE + (5 << 20))["append"] == 9
    got = calls(L, cache_struct(weight=None))
    assert got["weigh"] == 1 and got["evict"] == 1


def test_workspace_size(L):
    f = L.spec_verify_paged_attention_workspace_size
    assert f(9, 32, ctypes.byref(cache_struct())) >= 2 * 9 * 4 * 128 * 4
    assert f(0, 32, ctypes.byref(cache_struct())) == 0
    assert f(9, 30, ctypes.byref(cache_struct())) == 0
    assert f(9, 32, None) == 0


def test_binding_refusals():
    """The binding's own checks, on CPU tensors (no call is made)."""
    import speculative_decoding_verification_55_gb300 as sv
    k = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        sv.PagedCache(k.float(), k.float(), t)
    with pytest.raises(ValueError, match="shape"):
        sv.PagedCache(k, k[:4], t)
    with pytest.raises(ValueError, match="strides"):
        sv.PagedCache(k, torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16).transpose(1, 2), t)
    with pytest.raises(ValueError, match="contiguous"):
        sv.PagedCache(k.transpose(2, 3).contiguous().transpose(2, 3), k.transpose(2, 3).contiguous().transpose(2, 3), t)
    with pytest.raises(ValueError, match="page_table"):
        sv.PagedCache(k, k, t.long())
    with pytest.raises(ValueError, match="weight"):
        sv.PagedCache(k, k, t, torch.zeros((5, 16, 2)))
    c = sv.PagedCache(k, k, t)
    q = torch.zeros((3, 4, 8, 64), dtype=torch.bfloat16)
    pre = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        sv.spec_verify_kv_weights(q[:2], None, c, pre)
    with pytest.raises(TypeError, match="q must be"):
        sv.spec_verify_kv_weights(q.half(), None, c, pre)
    with pytest.raises(ValueError, match="heads of a token"):
        sv.spec_verify_kv_weights(q.transpose(1, 2).contiguous().transpose(1, 2), None, c, pre)
    with pytest.raises(TypeError, match="prefix_len"):
        sv.spec_verify_kv_weights(q, torch.zeros((3, 4, 8)), c, pre.long())
    with pytest.raises(ValueError, match="heads"):
        sv.spec_verify_kv_append(q, q, c, pre)
    with pytest.raises(ValueError, match="out_len"):
        sv.spec_verify_kv_evict(c, pre, 4, 1, torch.zeros(2, dtype=torch.int32))


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


class Batch:
    """A batch on the GPU whose unused slots hold NaN: pages in a random order, q, k_new and v_new as
    slices of one projection's output."""

    def __init__(self, prefix, N, H, G, D, S, dtype="bf16", nhd=False, seed=0, extra=0, poison=True):
        g = torch.Generator().manual_seed(seed)
        self.t, self.S, self.N, self.D = TYPES[dtype], S, N, D
        self.prefix = np.array(prefix, np.int32)
        B = len(prefix)
        used = [-(-(int(n) + N) // S) for n in prefix]
        self.table = np.full((B, max(used) + extra), 1 << 30, np.int32)
        ids = torch.randperm(sum(used) + 2, generator=g).numpy()
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u
        shape = (len(ids), H, S, D)
        k, v = torch.randn(shape, generator=g).to(self.t), torch.randn(shape, generator=g).to(self.t)
        if poison:
            held = torch.zeros(shape[0], S, dtype=torch.bool)
            for b, n in enumerate(prefix):
                for j in range(int(n) + N):
                    p, s = oracle.place(self.table, b, j, S)
                    held[p, s] = True
            k[~held[:, None].expand(-1, H, -1)] = math.nan
            v[~held[:, None].expand(-1, H, -1)] = math.nan
        put = (lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if nhd else (lambda x: x.cuda())
        self.k, self.v = put(k), put(v)
        self.weight = torch.rand(shape[:3], generator=g).cuda()
        qkv = torch.randn((B, N, H * G + 2 * H, D), generator=g)
        qkv[:, :, :H * G] *= 2
        qkv = qkv.to(self.t).cuda()
        self.q, self.k_new, self.v_new = qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:]
        self.scale = 1 / math.sqrt(D)

    def cache(self, sv, weight=True):
        return sv.PagedCache(self.k, self.v, dev(self.table), self.weight if weight else None)


def dev(a):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a, np.int32)).cuda()


def host(x):
    return x.detach().double().cpu().numpy()


def random_tree(rng, B, N):
    return np.array([[-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, N)] for _ in range(B)], np.int32)


def score_error(batch):
    """Bound on |score - exact| for normal inputs: (D + 2) 2^-24 times the largest sum |q k| scale."""
    D = batch.D
    q, k = host(batch.q).reshape(-1, D), np.nan_to_num(host(batch.k)).reshape(-1, D)
    most = batch.scale * np.sqrt((q ** 2).sum(1).max() * (k ** 2).sum(1).max())
    return (D + 2) * 2.0 ** -24 * most


def check_attention(batch, out, lse, prefix, num, parents, scale=None):
    scale = batch.scale if scale is None else scale
    want, wlse, mag = oracle.attention(host(batch.q), host(batch.k), host(batch.v), batch.table, prefix,
                                       num, parents, scale)
    out, lse = host(out), host(lse)
    assert np.array_equal(np.isnan(out), np.isnan(want)) and np.array_equal(np.isnan(lse), np.isnan(wlse))
    e, s = torch.finfo(batch.t).eps / 2, score_error(batch) * scale / batch.scale
    # 2 s: the errors of the entry's own score and of the normaliser; 1e-6: exponentials and sums.
    # A half's smallest step is 2^-24: a probability below it rounds by half of that.
    tiny = 2.0 ** -25 if batch.t == torch.float16 else 0.0
    tol = e * (mag + np.abs(want)) * (1 + e) + (2 * s + 1e-6) * mag + tiny * (prefix.max() + 65) * 6 + 1e-30
    fine = ~np.isnan(want)
    worst = (np.abs(out - want) / tol)[fine]
    assert worst.size == 0 or worst.max() <= 1, worst.max()
    fine = ~np.isnan(wlse)
    assert (np.abs(lse - wlse)[fine] <= s + 1e-6 + 2.0 ** -22 * np.abs(wlse)[fine]).all()


ATTEND = [
    # prefix lengths, N, Hkv, group, D, page, dtype, nhd
    ((0,), 1, 1, 1, 64, 16, "bf16", False),
    ((0, 1, 15, 16, 17, 63, 64, 65), 1, 2, 4, 128, 16, "bf16", False),
    ((127, 128, 129, 300, 1000), 1, 2, 8, 128, 32, "f16", True),
    ((5, 0, 250, 511, 77), 9, 2, 4, 128, 16, "bf16", True),
    ((5, 0, 250, 511, 77), 9, 2, 4, 128, 16, "f16", False),
    ((33, 700), 5, 3, 7, 64, 64, "bf16", False),
    ((1, 200, 90), 4, 1, 16, 256, 32, "bf16", True),
    ((40, 257), 17, 2, 3, 256, 16, "f16", False),
    ((3, 130, 400), 31, 1, 8, 128, 16, "bf16", False),
    ((3, 530), 65, 2, 2, 64, 128, "bf16", True),
    ((2, 130), 65, 1, 16, 128, 256, "f16", False),
    ((2500,), 2, 1, 5, 128, 16, "bf16", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,N,H,G,D,S,dtype,nhd", ATTEND)
def test_gpu_attention(sv, prefix, N, H, G, D, S, dtype, nhd):
    rng = np.random.default_rng(N * 31 + D)
    a = Batch(prefix, N, H, G, D, S, dtype, nhd, seed=N + D)
    B = len(prefix)
    num = rng.integers(0, N + 1, B).astype(np.int32)
    num[-1] = N
    c = a.cache(sv, weight=False)
    out, lse = sv.attend(a.q, c, dev(a.prefix), dev(num))
    check_attention(a, out, lse, a.prefix, num, None)
    again, lse2 = sv.attend(a.q, c, dev(a.prefix), dev(num))
    assert torch.equal(again, out) and torch.equal(lse2, lse)          # the same call, the same bits
    tree = random_tree(rng, B, N)
    out, lse = sv.attend(a.q, c, dev(a.prefix), None, dev(tree), scale=0.25)
    check_attention(a, out, lse, a.prefix, np.full(B, N), tree, 0.25)


@pytest.mark.gpu
def test_gpu_attention_many_rows(sv):
    """More rows than the GPU holds blocks, most of them short, some without tokens or entries."""
    rng = np.random.default_rng(5)
    prefix = rng.integers(0, 40, 700)
    prefix[::50] = 300
    a = Batch(prefix, 2, 1, 4, 64, 16, seed=9)
    num = rng.integers(0, 3, 700).astype(np.int32)
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num))
    check_attention(a, out, lse, a.prefix, num, None)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
def test_gpu_attention_large_trees_many_rows(sv, D, dtype):
    """More than 128 query rows a key head and an item for every SM: two query tiles at once."""
    rng = np.random.default_rng(7)
    prefix = rng.integers(0, 200, 170)
    a = Batch(prefix, 17, 1, 11, D, 16, dtype, seed=D)
    num = rng.integers(0, 18, 170).astype(np.int32)
    tree = random_tree(rng, 170, 17)
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num), dev(tree))
    check_attention(a, out, lse, a.prefix, num, tree)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,D", [(31, 8, 128), (65, 7, 64), (9, 16, 128)])
def test_gpu_attention_large_trees_in_parts(sv, N, G, D):
    """The same for a few long rows in tables with room for many more: two query tiles in parts."""
    a = Batch((3000, 129, 0), N, 1, G, D, 16, seed=N)
    table = np.full((3, 65536), 1 << 30, np.int32)
    table[:, :a.table.shape[1]] = a.table
    a.table = table
    tree = random_tree(np.random.default_rng(N), 3, N)
    num = np.array([N, N - 3, N], np.int32)
    for parents in (None, tree):
        out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num), dev(parents))
        check_attention(a, out, lse, a.prefix, num, parents)
    a.v[oracle.place(a.table, 0, 3000 + N - 1, 16)[0]] = math.inf      # entries of the round's last page
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num))
    seen = 3000 // 16 * 16 + 16 if (3000 + N - 1) // 16 == 3000 // 16 else (3000 + N - 1) // 16 * 16
    first = max(0, seen - 3000)                            # tokens before it attend no entry of that page
    assert np.isfinite(host(out)[0, :first]).all() and np.isinf(host(out)[0, N - 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(3, 2), (9, 8), (31, 8)])
def test_gpu_unattended_values_have_no_part(sv, N, G):
    """Infinities and NaN in the values and keys of tokens that a token does not attend."""
    rng = np.random.default_rng(6)
    a = Batch((70, 0, 64, 129), N, 2, G, 128, 16, seed=3)
    tree = random_tree(rng, 4, N)
    for b in range(4):
        p, s = oracle.place(a.table, b, int(a.prefix[b]) + N - 1, 16)      # the last token: a leaf
        a.v[p, :, s, 1::2] = math.inf
        a.v[p, 0, s, 4] = math.nan
        if b == 2:
            a.k[p, :, s] = math.nan
    num = np.full(4, N)
    for parents in (None, tree):
        out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), None, dev(parents))
        out, lse = host(out), host(lse)
        assert np.isfinite(out[:, :N - 1]).all() and np.isfinite(lse[:, :N - 1]).all()
        k, v = np.nan_to_num(host(a.k), posinf=0), np.nan_to_num(host(a.v), posinf=0)
        want, _, mag = oracle.attention(host(a.q), k, v, a.table, a.prefix, num, parents, a.scale)
        tol = 2.0 ** -8 * (mag + np.abs(want)) * 1.01 + 1e-4 * mag
        assert (np.abs(out - want)[:, :N - 1] <= tol[:, :N - 1]).all()
        assert np.isinf(out[[0, 1, 3], N - 1][:, :, 1::2]).all()           # its own infinity is its own
        assert np.isnan(out[[0, 1, 3], N - 1, :G, 4]).all()
        assert np.isnan(out[2, N - 1]).all() and np.isnan(lse[2, N - 1]).all()
        assert np.isfinite(out[[0, 1, 3], N - 1][:, G:, 0::2]).all()


@pytest.mark.gpu
def test_gpu_attention_row_errors(sv):
    a = Batch((40, 40, 40, 40, 40, 40), 3, 2, 4, 128, 16, seed=4)
    prefix = a.prefix.copy()
    num = np.array([3, 4, -1, 3, 2, 3], np.int32)
    prefix[3] = a.table.shape[1] * 16 - 2                  # one more entry than the table holds
    a.table[4, 1] = len(a.k)                               # a page past the end
    a.table[5, 2] = -1
    tree = np.array([[-1, 0, 1]] * 6, np.int32)
    for parents in (None, tree):
        out, lse = sv.attend(a.q, a.cache(sv), dev(prefix), dev(num), dev(parents))
        check_attention(a, out, lse, prefix, num, parents)
    for bad in ([0, 0, 1], [-1, 1, 1], [-1, 0, -1], [-1, 2, 0]):
        tree[0] = bad
        out, lse = sv.attend(a.q, a.cache(sv), dev(prefix), dev(num), dev(tree))
        check_attention(a, out, lse, prefix, num, tree)


@pytest.mark.gpu
def test_gpu_attention_extreme_scores(sv):
    """Scores of hundreds, and a key that outweighs all others by far: the running maximum holds."""
    a = Batch((200, 64), 2, 1, 4, 128, 16, seed=8)
    a.k *= 8
    a.q *= 8
    for b, j in ((0, 199), (1, 0)):
        p, s = oracle.place(a.table, b, j, 16)
        a.k[p, :, s] = a.q[b, 0, :1]
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix))
    check_attention(a, out, lse, a.prefix, np.array([2, 2]), None)


@pytest.mark.gpu
def test_gpu_far_pages(sv):
    """Offsets past 32 bits: pages that lie over 2^32 bytes into the cache."""
    S, H, D, P = 16, 8, 128, (1 << 17) + 9                  # 4.3 GB of keys, as much of values
    a = Batch((50, 20), 3, H, 2, D, S, seed=2)
    big = [torch.zeros((P, H, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w = torch.zeros((P, H, S), device="cuda")
    n = len(a.k)
    for x, y in zip(big, (a.k, a.v)):
        x[P - n:] = y
    table = a.table.astype(np.int64) + P - n
    c = sv.PagedCache(*big, dev(np.minimum(table, 1 << 30)), w)
    out, lse = sv.attend(a.q, c, dev(a.prefix))
    check_attention(a, out, lse, a.prefix, np.array([3, 3]), None)
    sv.spec_verify_kv_weights(a.q, lse, c, dev(a.prefix))
    want = oracle.weights(host(a.q), host(lse), np.nan_to_num(host(a.k)), np.zeros(a.weight.shape), a.table, a.prefix, [3, 3], None, a.scale)
    assert np.allclose(host(w[P - n:]), want, rtol=1e-4, atol=1e-7) and float(w[:P - n].abs().sum()) == 0
    olen = dev([0, 0])
    sv.spec_verify_kv_append(a.k_new, a.v_new, c, dev(a.prefix), None, None, olen)
    k, v, _, n_out = oracle.append(host(a.k), host(a.v), None, host(a.k_new), host(a.v_new), a.table, a.prefix, [3, 3], None)
    assert np.array_equal(host(big[0][P - n:]), k, equal_nan=True)
    assert np.array_equal(host(big[1][P - n:]), v, equal_nan=True)
    w[P - n:] = a.weight
    sv.spec_verify_kv_evict(c, dev([53, 23]), 22, 5, olen)
    k, v, w2, n_out = oracle.evict(k, v, host(a.weight), a.table, [53, 23], 22, 5)
    assert np.array_equal(host(big[0][P - n:]), k, equal_nan=True) and olen.tolist() == n_out.tolist()
    assert np.array_equal(host(w[P - n:]), w2)


# ------------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("prefix,N,H,G,D,S,dtype,nhd", ATTEND)
def test_gpu_weights(sv, prefix, N, H, G, D, S, dtype, nhd):
    rng = np.random.default_rng(N * 17 + D)
    a = Batch(prefix, N, H, G, D, S, dtype, nhd, seed=N + D)
    B = len(prefix)
    for path in (None, np.array([np.sort(rng.permutation(N)) for _ in range(B)], np.int32)):
        num = rng.integers(-1, N + 1, B).astype(np.int32)
        num[-1] = N
        _, lse, _ = oracle.attention(host(a.q), host(a.k), host(a.v), a.table, a.prefix, np.full(B, N), None, a.scale)
        lse = torch.as_tensor(lse, dtype=torch.float32).cuda()
        before = a.weight.clone()
        sv.spec_verify_kv_weights(a.q, lse, a.cache(sv), dev(a.prefix), dev(num), dev(path))
        want = oracle.weights(host(a.q), host(lse), host(a.k), host(before), a.table, a.prefix, num, path, a.scale)
        got, old = host(a.weight), host(before)
        # Each term: its score's error, the exponential's 2^-22, the exponent's own rounding (values of
        # some tens: 2^-24 of them, twice); the sum: N G terms in fp32.
        rel = score_error(a) + 2.0 ** -22 + 2.0 ** -23 * (np.abs(host(lse)).max() + 40) + N * G * 2.0 ** -24
        tol = rel * (want - old) + 2.0 ** -23 * want
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.gpu
def test_gpu_weights_errors(sv):
    a = Batch((40, 40, 40, 40), 3, 2, 4, 64, 16, seed=4)
    prefix = np.array([-1, a.table.shape[1] * 16 - 1, 40, 40], np.int32)
    path = np.array([[0, 1, 2], [0, 1, 2], [0, 3, 1], [0, 2, -1]], np.int32)
    num = np.array([3, 3, 2, 2], np.int32)
    a.table[3, 1] = -5                                      # passed over
    lse = torch.full((4, 3, 8), 3.0, device="cuda")
    before = host(a.weight)
    sv.spec_verify_kv_weights(a.q, lse, a.cache(sv), dev(prefix), dev(num), dev(path))
    want = oracle.weights(host(a.q), host(lse), host(a.k), before, a.table, prefix, num, path, a.scale)
    assert np.allclose(host(a.weight), want, rtol=1e-5, atol=0)


EVICT = [
    # lengths, budget, recent, Hkv, D, page, dtype, nhd
    ((40, 33, 32, 31, 0, 200), 32, 4, 2, 128, 16, "bf16", False),
    ((500, 129, 1000), 128, 0, 3, 64, 32, "f16", True),
    ((500, 129, 1000), 128, 128, 1, 256, 16, "bf16", False),
    ((3000, 2049), 2048, 100, 2, 128, 16, "bf16", True),
    ((2, 5), 1, 0, 8, 128, 256, "f16", False),
    ((2, 5), 1, 1, 1, 64, 16, "bf16", False),
    (tuple(range(60, 160)), 63, 7, 4, 128, 64, "bf16", False),
]


def check_evict(sv, a, lengths, budget, recent):
    before = [host(x) for x in (a.k, a.v, a.weight)]
    olen = torch.full((len(lengths),), 77, dtype=torch.int32, device="cuda")
    sv.spec_verify_kv_evict(a.cache(sv), dev(lengths), budget, recent, olen)
    *want, n = oracle.evict(*before, a.table, lengths, budget, recent)
    assert olen.tolist() == n.tolist()
    for x, w in zip((a.k, a.v, a.weight), want):
        assert np.array_equal(host(x), w, equal_nan=True)      # behind the budget too: left as it was


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["random", "equal", "few values", "special"])
@pytest.mark.parametrize("lengths,budget,recent,H,D,S,dtype,nhd", EVICT)
def test_gpu_evict(sv, lengths, budget, recent, H, D, S, dtype, nhd, weights):
    a = Batch(lengths, 1, H, 1, D, S, dtype, nhd, seed=budget + recent, poison=False)
    if weights == "equal":
        a.weight.fill_(0.5)
    elif weights == "few values":
        a.weight.mul_(4).floor_()
    elif weights == "special":
        r = a.weight.clone()
        a.weight[r < 0.2] = 0.0
        a.weight[(r >= 0.2) & (r < 0.3)] = -0.0
        a.weight[(r >= 0.3) & (r < 0.4)] = math.inf
        a.weight[(r >= 0.4) & (r < 0.5)] = -1.0
        a.weight[(r >= 0.5) & (r < 0.6)] = math.nan
        a.weight[(r >= 0.6) & (r < 0.7)] = 1e-42
    check_evict(sv, a, np.array(lengths), budget, recent)


@pytest.mark.gpu
def test_gpu_evict_row_errors(sv):
    a = Batch((100, 100, 100, 100), 1, 2, 1, 64, 16, seed=1, poison=False)
    a.table[1, 5] = len(a.k)
    check_evict(sv, a, np.array([-3, 90, a.table.shape[1] * 16 + 1, 100]), 50, 10)


@pytest.mark.gpu
def test_gpu_evict_few_heads_over_many_blocks(sv):
    """One row and head whose columns are split over a cluster, repeated: the same result each time."""
    first = None
    for _ in range(5):
        a = Batch((9000,), 1, 1, 1, 128, 16, seed=12, poison=False)
        a.weight.mul_(50).floor_()
        olen = dev([0])
        sv.spec_verify_kv_evict(a.cache(sv), dev([9000]), 4000, 33, olen)
        got = [x.clone() for x in (a.k, a.v, a.weight)]
        if first is None:
            first = got
            b = Batch((9000,), 1, 1, 1, 128, 16, seed=12, poison=False)
            b.weight.mul_(50).floor_()
            check_evict(sv, b, np.array([9000]), 4000, 33)
        assert all(torch.equal(x, y) for x, y in zip(got, first))


# ------------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("prefix,N,H,G,D,S,dtype,nhd", ATTEND)
def test_gpu_append(sv, prefix, N, H, G, D, S, dtype, nhd):
    rng = np.random.default_rng(N + D)
    B = len(prefix)
    for path in (None, np.array([np.sort(rng.permutation(N)) for _ in range(B)], np.int32)):
        a = Batch(prefix, N, H, G, D, S, dtype, nhd, seed=N + D)
        num = rng.integers(-1, N + 1, B).astype(np.int32)
        num[-1] = N
        want = oracle.append(host(a.k), host(a.v), host(a.weight), host(a.k_new), host(a.v_new), a.table, a.prefix, num, path)
        olen = torch.full((B,), 77, dtype=torch.int32, device="cuda")
        sv.spec_verify_kv_append(a.k_new, a.v_new, a.cache(sv), dev(a.prefix), dev(num), dev(path), olen)
        for x, w in zip((a.k, a.v, a.weight), want):
            assert np.array_equal(host(x), w, equal_nan=True)
        assert olen.tolist() == want[3].tolist()


@pytest.mark.gpu
def test_gpu_append_row_errors(sv):
    a = Batch((40, 40, 40, 40, 40, 40), 3, 2, 4, 64, 16, seed=4, extra=2)
    prefix = np.array([-1, 40, 40, a.table.shape[1] * 16 - 2, 40, 47], np.int32)
    num = np.array([3, 4, -2, 3, 2, 2], np.int32)
    path = np.array([[0, 1, 2]] * 4 + [[0, 3, 0], [1, 2, -1]], np.int32)
    assert a.table[5, 3] == 1 << 30                        # entry 48 of the last row has no page
    before = [host(x) for x in (a.k, a.v, a.weight)]
    olen = torch.full((6,), 77, dtype=torch.int32, device="cuda")
    sv.spec_verify_kv_append(a.k_new, a.v_new, a.cache(sv), dev(prefix), dev(num), dev(path), olen)
    assert olen.tolist() == [-1] * 6
    for x, w in zip((a.k, a.v, a.weight), before):
        assert np.array_equal(host(x), w, equal_nan=True)


# ------------------------------------------------------------------------------------------------
# Together, captured, on another stream
# ------------------------------------------------------------------------------------------------

@pytest.mark.gpu
def test_gpu_rounds_together(sv):
    """Two rounds as they are used: append, attention, verification of drafts from its output, rollback,
    weights of what was kept, eviction to a budget; then a tree round with its kept path."""
    rng = np.random.default_rng(3)
    N, H, G, D, S, V, B = 5, 2, 4, 64, 16, 512, 6
    a = Batch((30, 0, 64, 100, 47, 90), N + 40, H, G, D, S, seed=5, poison=False)
    W = torch.randn((H * G * D, V), device="cuda") / 8
    a.weight.zero_()
    c = a.cache(sv)
    n = a.prefix.copy()
    k, v, w = (host(x) for x in (a.k, a.v, a.weight))
    for rnd in range(3):
        tree = random_tree(rng, B, N) if rnd == 2 else None
        new = torch.as_tensor(rng.standard_normal((B, N, (G + 2) * H, D)), dtype=torch.float32).to(a.t).cuda()
        a.q, kn, vn = new[:, :, :H * G], new[:, :, H * G:H * G + H], new[:, :, H * G + H:]
        olen = dev(np.zeros(B))
        sv.spec_verify_kv_append(kn, vn, c, dev(n), None, None, olen)
        k, v, w, on = oracle.append(k, v, w, host(kn), host(vn), a.table, n, [N] * B, None)
        assert olen.tolist() == on.tolist()
        out, lse = sv.attend(a.q, c, dev(n), None, dev(tree))
        check_attention(a, out, lse, n, np.full(B, N), tree)
        logits = (out.float().reshape(B, N, -1) @ W).contiguous()
        path = None
        if tree is None:
            draft = torch.randn((B, N - 1, V), device="cuda")
            tok, num, _ = sv.verify(logits, draft, draft.argmax(-1).to(torch.int32), None,
                                    torch.full((B,), 0.5, device="cuda"), torch.rand((B, N + 1), device="cuda"))
        else:
            toks = torch.randint(0, V, (B, N), dtype=torch.int32, device="cuda")
            for b in range(B):                          # one child of the root is the target's choice
                toks[b, 1] = logits[b, 0].argmax()
            path, num, _, _ = sv.verify_tree(logits, toks, dev(tree))
            sv.spec_verify_kv_append(kn, vn, c, dev(n), num, path, olen)
            k, v, w, on = oracle.append(k, v, w, host(kn), host(vn), a.table, n, num.tolist(), path.cpu().numpy())
            assert (num > 1).any() and olen.tolist() == on.tolist()
        keep = torch.zeros_like(num)
        sv.spec_verify_kv_rollback(dev(n), None, num, None, keep, None, gamma_max=N - 1)
        assert keep.tolist() == (n + np.array(num.tolist())).tolist()
        sv.spec_verify_kv_weights(a.q, lse, c, dev(n), num, path)
        w = oracle.weights(host(a.q), host(lse), k, w, a.table, n, num.tolist(), None if path is None else path.cpu().numpy(), a.scale)
        assert np.allclose(host(a.weight), w, rtol=1e-4, atol=1e-6)
        # The probabilities of each kept token sum to 1 over its entries.
        w = host(a.weight)                               # the eviction decides on the stored weights
        sv.spec_verify_kv_evict(c, keep, 60, 12, olen)
        k, v, w, on = oracle.evict(k, v, w, a.table, keep.tolist(), 60, 12)
        for x, y in zip((a.k, a.v, a.weight), (k, v, w)):
            assert np.array_equal(host(x), y)
        assert olen.tolist() == on.tolist() and max(on) == 60
        n = on.copy()


@pytest.mark.gpu
def test_gpu_captured_and_streams(sv):
    """The calls in a CUDA graph (replayed on new lengths and contents) and on a side stream."""
    a = Batch((30, 200, 64), 4, 2, 4, 128, 16, seed=6, extra=3)
    c = a.cache(sv)
    pre, num = dev(a.prefix), dev([4, 4, 4])
    sv.attend(a.q, c, pre, num)
    side = torch.cuda.Stream()
    graph, outs = torch.cuda.CUDAGraph(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        outs = sv.attend(a.q, c, pre, num)
        sv.spec_verify_kv_weights(a.q, outs[1], c, pre, num)
    for prefix, m in (((30, 200, 64), (4, 3, 0)), ((0, 150, 9), (1, 4, 2))):
        pre.copy_(dev(prefix))
        num.copy_(dev(m))
        before = a.weight.clone()
        graph.replay()
        check_attention(a, *outs, np.array(prefix), np.array(m), None)
        want = oracle.weights(host(a.q), host(outs[1]), host(a.k), host(before), a.table, prefix, m, None, a.scale)
        assert np.allclose(host(a.weight), want, rtol=1e-4, atol=1e-7)
    side.wait_stream(torch.cuda.current_stream())
    out, lse = sv.attend(a.q, c, pre, num, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, outs[0]) and torch.equal(lse, outs[1])


@pytest.mark.gpu
def test_gpu_workspace_of_any_contents(sv):
    """Calls of several sizes on one workspace that holds anything: the same results."""
    ws = None
    for prefix, N, H, G, D in (((900, 3), 1, 1, 2, 64), ((2000, 1000, 7), 9, 4, 8, 128), ((300,) * 40, 1, 2, 4, 256),
                               ((64,), 65, 1, 4, 128)):
        a = Batch(prefix, N, H, G, D, 16, seed=N)
        c = a.cache(sv)
        if ws is None:
            ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")
        assert sv.spec_verify_paged_attention_workspace_size(N, H * G, c) <= ws.numel()
        B = len(prefix)
        out = torch.empty((B, N, H * G, D), dtype=a.t, device="cuda")
        lse = torch.empty((B, N, H * G), device="cuda")
        sv.spec_verify_paged_attention(a.q, c, dev(a.prefix), None, None, out, lse, ws)
        check_attention(a, out, lse, a.prefix, np.full(B, N), None)
        ws.random_(0, 256)
        out2 = torch.empty_like(out)
        sv.spec_verify_paged_attention(a.q, c, dev(a.prefix), None, None, out2, None, ws)
        assert torch.equal(out, out2)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,D", [(1, 4, 128), (9, 4, 64), (31, 8, 128), (5, 2, 256)])
def test_gpu_other_strides(sv, N, G, D):
    """Keys and values interleaved in one tensor with room between slots, a key head of one, queries with
    gaps between tokens: every call reads and writes its own elements alone."""
    for H in (1, 3):
        a = Batch((60, 0, 129), N, H, G, D, 32, seed=N)
        both = torch.full((len(a.k), 32, H + 1, 3, D), 7.0, dtype=a.t, device="cuda")
        k, v = both[:, :, :H, 0].transpose(1, 2), both[:, :, :H, 2].transpose(1, 2)
        k.copy_(a.k)
        v.copy_(a.v)
        a.k, a.v = k, v
        wide = torch.zeros((3, N, H * G + 2, D), dtype=a.t, device="cuda")
        wide[:, :, :H * G] = a.q
        a.q = wide[:, :, :H * G]
        c = a.cache(sv)
        out, lse = sv.attend(a.q, c, dev(a.prefix))
        check_attention(a, out, lse, a.prefix, np.full(3, N), None)
        before = host(a.weight)
        sv.spec_verify_kv_weights(a.q, lse, c, dev(a.prefix))
        want = oracle.weights(host(a.q), host(lse), host(a.k), before, a.table, a.prefix, [N] * 3, None, a.scale)
        assert np.allclose(host(a.weight), want, rtol=1e-4, atol=1e-7)
        want = oracle.append(host(a.k), host(a.v), host(a.weight), host(a.k_new), host(a.v_new), a.table, a.prefix, [N] * 3, None)
        sv.spec_verify_kv_append(a.k_new, a.v_new, c, dev(a.prefix))
        for x, w in zip((a.k, a.v, a.weight), want):
            assert np.array_equal(host(x), w, equal_nan=True)
        a.k.nan_to_num_(0.5)
        a.v.nan_to_num_(0.25)
        check_evict(sv, a, a.prefix + N, 40, 7)
        assert (both[:, :, H:] == 7).all() and (both[:, :, :, 1] == 7).all()


@pytest.mark.gpu
def test_gpu_shared_pages(sv):
    """Rows with a common prefix on the same pages: read by all, their weights take every row's part."""
    a = Batch((90, 90, 90), 4, 2, 4, 128, 16, seed=11)
    a.table[1, :4] = a.table[0, :4]
    a.table[2, :5] = a.table[0, :5]
    c = a.cache(sv)
    out, lse = sv.attend(a.q, c, dev(a.prefix))
    check_attention(a, out, lse, a.prefix, np.full(3, 4), None)
    before = host(a.weight)
    sv.spec_verify_kv_weights(a.q, lse, c, dev(a.prefix))
    want = oracle.weights(host(a.q), host(lse), host(a.k), before, a.table, a.prefix, [4] * 3, None, a.scale)
    assert np.allclose(host(a.weight), want, rtol=1e-4, atol=1e-7)


@pytest.mark.gpu
def test_gpu_calls_at_once(sv):
    """Calls in flight on three streams, each with its own workspace, give what they give alone."""
    batches = [Batch(p, N, H, G, D, 16, seed=N) for p, N, H, G, D in
               (((3000, 50, 700), 1, 2, 8, 128), ((900, 2000), 9, 2, 4, 64), ((64,) * 30, 31, 1, 8, 128))]
    caches = [b.cache(sv) for b in batches]
    alone = [sv.attend(b.q, c, dev(b.prefix)) for b, c in zip(batches, caches)]
    prefix = [dev(b.prefix) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for b, c, p, s in zip(batches, caches, prefix, streams):
            got.append(sv.attend(b.q, c, p, stream=s))
    torch.cuda.synchronize()
    for x, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[x % 3][0]) and torch.equal(lse, alone[x % 3][1])


@pytest.mark.gpu
def test_gpu_captured_append_and_evict(sv):
    """Append along a path and eviction in one graph, replayed on new contents and lengths."""
    a = Batch((100, 40, 70), 6, 2, 2, 64, 16, seed=13, poison=False, extra=1)
    c = a.cache(sv)
    pre, num = dev(a.prefix), dev([6, 6, 6])
    path = np.array([[0, 2, 3, -1, -1, -1], [0, 1, 2, 3, 4, 5], [0, 5, -1, -1, -1, -1]], np.int32)
    length, kept = dev([0] * 3), dev([0] * 3)
    d_path = dev(path)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sv.spec_verify_kv_append(a.k_new, a.v_new, c, pre, num, d_path, length)
        sv.spec_verify_kv_evict(c, length, 60, 9, kept)
    for prefix, m in (((100, 40, 70), (3, 6, 2)), ((60, 59, 3), (3, 1, 2))):
        pre.copy_(dev(prefix))
        num.copy_(dev(m))
        a.weight.uniform_()
        k, v, w, n = oracle.append(host(a.k), host(a.v), host(a.weight), host(a.k_new), host(a.v_new), a.table, prefix, m, path)
        k, v, w, on = oracle.evict(k, v, w, a.table, n.tolist(), 60, 9)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((a.k, a.v, a.weight), (k, v, w)):
            assert np.array_equal(host(x), y)
        assert length.tolist() == n.tolist() and kept.tolist() == on.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("H,D", [(1, 64), (2, 128)])
def test_gpu_evict_long_rows(sv, H, D):
    """Rows longer than a block holds keys of: the cluster selects together; equal weights across its runs."""
    lengths = np.array([40000, 16385, 20000])
    a = Batch(lengths, 1, H, 1, D, 128, seed=D, poison=False)
    a.weight.mul_(3000).floor_()
    for b, n in ((1, 16385),):                                   # one row of equal weights alone
        for p in range(-(-n // 128)):
            a.weight[int(a.table[b, p])] = 1.0
    old = [x.clone() for x in (a.k, a.v, a.weight)]
    olen = dev([0] * 3)
    budget, recent = 12001, 300
    sv.spec_verify_kv_evict(a.cache(sv), dev(lengths), budget, recent, olen)
    assert olen.tolist() == [budget] * 3
    for b, n in enumerate(lengths):
        ids = torch.as_tensor(a.table[b, :-(-int(n) // 128)].astype(np.int64), device="cuda")
        rows = lambda x: x[ids].transpose(0, 1).flatten(1, 2)[:, :int(n)]
        w = host(rows(old[2]))
        for h in range(H):
            keep = torch.as_tensor(oracle.kept_entries(w[h], budget, recent), device="cuda")
            for x, o in zip((a.k, a.v, a.weight), old):
                assert torch.equal(rows(x)[h, :budget], rows(o)[h][keep])
                assert torch.equal(rows(x)[h, budget:], rows(o)[h, budget:])


def test_overlap_refusals(L):
    """Arrays that share a part of their memory: refused as whole ones are (SV_ERR_OVERLAP)."""
    c = cache_struct()
    pre = FAKE + (5 << 20)
    assert calls(L, c, olen=pre + 4)["evict"] == 9 and calls(L, c, olen=pre - 4)["evict"] == 9
    got = calls(L, c, olen=pre + 4)
    assert got["append"] == 9
    assert calls(L, c, par=FAKE + (10 << 20), olen=FAKE + (10 << 20) + 4 * 17)["append"] == 9
    q, size = FAKE + (4 << 20), 2 * (9 * 32 * 128 * 2)
    assert calls(L, c, out=q)["attend"] == 9
    assert calls(L, c, out=q + size - 16)["attend"] == 9 and calls(L, c, out=q - size + 16)["attend"] == 9
    assert calls(L, c, lse=q + 64)["attend"] == 9


def test_cache_on_the_host():
    """Every call of the binding refuses a cache in host memory."""
    import speculative_decoding_verification_55_gb300 as sv
    sv.build_library()
    k = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    c = sv.PagedCache(k, k.clone(), torch.zeros((3, 2), dtype=torch.int32), torch.zeros((5, 2, 16)))
    q = torch.zeros((3, 4, 8, 64), dtype=torch.bfloat16)
    n = torch.zeros(3, dtype=torch.int32)
    lse = torch.zeros((3, 4, 8))
    for call in (lambda: sv.attend(q, c, n), lambda: sv.spec_verify_kv_weights(q, lse, c, n),
                 lambda: sv.spec_verify_kv_append(q[:, :, :2], q[:, :, :2], c, n),
                 lambda: sv.spec_verify_kv_evict(c, n, 4, 1, n.clone()),
                 lambda: sv.spec_verify_paged_attention(q, c, n, None, None, q.clone(), lse, torch.zeros(1 << 20))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.gpu
def test_gpu_evict_from_threads(sv):
    """Evictions of caches that need different amounts of shared memory, from host threads at once."""
    from concurrent.futures import ThreadPoolExecutor
    jobs = []
    for x, n in enumerate((70, 700, 5000, 20000)):
        a = Batch((n, n // 2), 1, 2, 1, 64, 16, seed=x, poison=False)
        jobs.append((a, a.cache(sv), dev([n, n // 2]), dev([0, 0]), n // 3, torch.cuda.Stream()))
    want = [oracle.evict(host(a.k), host(a.v), host(a.weight), a.table, n.tolist(), budget, 5)
            for a, c, n, o, budget, s in jobs]
    torch.cuda.synchronize()

    def run(job):
        a, c, n, o, budget, s = job
        for _ in range(30):                    # the first evicts, the others find rows in their budget
            sv.spec_verify_kv_evict(c, n, budget, 5, o, stream=s)
            with torch.cuda.stream(s):
                n.copy_(o)

    with ThreadPoolExecutor(4) as pool:
        list(pool.map(run, jobs))
    torch.cuda.synchronize()
    for (a, c, n, o, budget, s), (k, v, w, on) in zip(jobs, want):
        assert o.tolist() == on.tolist()
        for x, y in zip((a.k, a.v, a.weight), (k, v, w)):
            assert np.array_equal(host(x), y)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
def test_gpu_attention_large_trees_long_tables(sv, D, dtype):
    """More than 128 query rows a key head and an item for every SM in tables with room for long rows: two query
    tiles at once, of which many rows fill one alone."""
    rng = np.random.default_rng(8)
    prefix = rng.integers(0, 400, 170)
    a = Batch(prefix, 17, 1, 11, D, 16, dtype, seed=D, extra=120)
    num = rng.integers(0, 18, 170).astype(np.int32)
    tree = random_tree(rng, 170, 17)
    tree[5, 3] = 3                                         # a row in error
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num), dev(tree))
    if num[5] > 3:
        assert np.isnan(host(out)[5, :num[5]]).all() and np.isnan(host(lse)[5, :num[5]]).all()
    tree[5] = [-1] + [0] * 16
    keep = np.arange(170) != 5
    want, got = sv.attend(a.q, a.cache(sv), dev(a.prefix), dev(num), dev(tree)), (out, lse)
    for x, y in zip(got, want):
        assert torch.equal(x[dev(np.flatnonzero(keep)).long()], y[dev(np.flatnonzero(keep)).long()])
    check_attention(a, *want, a.prefix, num, tree)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (9, 4), (31, 8)])
def test_gpu_attention_one_workspace_other_lengths(sv, N, G):
    """Few rows, one graph replayed on lengths that leave rows short, without tokens and in error: nothing of an
    earlier call's parts is joined."""
    a = Batch((5000, 3000, 4000), N, 2, G, 128, 16, seed=N, poison=False)
    c, pre, num = a.cache(sv), dev(a.prefix), dev([N] * 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = sv.attend(a.q, c, pre, num)
    for prefix, m in (((5000, 3000, 4000), (N, N, N)), ((5000, 20, 4000), (0, N, N + 1)), ((0, 3000, 90), (1, 0, N)),
                      ((5000, 3000, 4000), (N, N, N))):
        pre.copy_(dev(prefix))
        num.copy_(dev(m))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(a, out, lse, np.array(prefix), np.array(m), None)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,dtype", [(1, 4, "bf16"), (1, 8, "f16"), (3, 5, "bf16"), (9, 4, "bf16"), (9, 4, "f16")])
def test_gpu_values_before_the_round_that_are_not_finite(sv, N, G, dtype):
    """Infinities and NaN in the last entries before the round, which every token attends."""
    prefix = (100, 111, 64, 97)
    for back in (1, 2, 7, 15):
        a = Batch(prefix, N, 2, G, 128, 16, dtype, seed=back)
        for b, n in enumerate(prefix):
            p, s = oracle.place(a.table, b, n - back, 16)
            a.v[p, 0, s, 3] = math.inf
            a.v[p, 0, s, 64] = -math.inf
            a.v[p, 1, s, 17] = math.nan
        out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix))
        got = host(out)
        assert np.isposinf(got[:, :, :G, 3]).all() and np.isneginf(got[:, :, :G, 64]).all()
        assert np.isnan(got[:, :, G:, 17]).all() and np.isfinite(host(lse)).all()
        got[:, :, :G, 3] = got[:, :, :G, 64] = got[:, :, G:, 17] = 0.0
        a.v[a.v.isinf()] = 0.0
        for b, n in enumerate(prefix):
            p, s = oracle.place(a.table, b, n - back, 16)
            a.v[p, 1, s, 17] = 0.0
        want, _ = sv.attend(a.q, a.cache(sv), dev(a.prefix))
        want = host(want)
        want[:, :, :G, 3] = want[:, :, :G, 64] = want[:, :, G:, 17] = 0.0
        assert np.array_equal(got, want)                   # nothing else is changed


def test_attend_from_threads_on_one_stream(monkeypatch):
    """Calls of attend from several host threads share a stream's workspace: one is done with its launches before the
    next has the workspace (no GPU: the call itself is stood in for)."""
    import threading
    import time
    from concurrent.futures import ThreadPoolExecutor
    from speculative_decoding_verification_55_gb300 import _cache
    k = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    c = _cache.PagedCache(k, k.clone(), torch.zeros((3, 2), dtype=torch.int32))
    q, n = torch.zeros((3, 4, 8, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    shared, inside, most, failing = torch.zeros(64, dtype=torch.uint8), [], [], threading.Event()

    def workspace(*args):
        inside.append(1)
        return shared

    def launches(*args):
        time.sleep(0.002)
        most.append(len(inside))
        inside.pop()
        if failing.is_set():
            raise RuntimeError("refused")

    monkeypatch.setattr(_cache, "_on_gpu", lambda device: None)
    monkeypatch.setattr(_cache, "_attend_workspace", workspace)
    monkeypatch.setattr(_cache, "_attention", launches)
    with ThreadPoolExecutor(4) as pool:
        list(pool.map(lambda x: _cache.attend(q, c, n), range(40)))
    assert most == [1] * 40
    failing.set()                                          # a refused call leaves the workspace to others
    for _ in range(2):
        with pytest.raises(RuntimeError, match="refused"):
            _cache.attend(q, c, n)


@pytest.mark.gpu
def test_gpu_attend_from_threads_on_one_stream(sv):
    """The same on the GPU: threads on the default stream, batches whose items have many parts."""
    from concurrent.futures import ThreadPoolExecutor
    jobs = []
    for prefix, N, H, G, D in (((9000,), 1, 2, 8, 128), ((4000, 900), 9, 2, 4, 64), ((700, 64, 3000), 31, 1, 8, 128)):
        a = Batch(prefix, N, H, G, D, 16, seed=N)
        c, n = a.cache(sv), dev(a.prefix)
        jobs.append((a, c, n, sv.attend(a.q, c, n)))
    torch.cuda.synchronize()

    def run(x):
        a, c, n, (out, lse) = jobs[x % 3]
        got = [sv.attend(a.q, c, n) for _ in range(60)]
        return all(torch.equal(o, out) and torch.equal(s, lse) for o, s in got)

    with ThreadPoolExecutor(6) as pool:
        assert all(pool.map(run, range(6)))


def test_overlap_refusals_of_every_array(L):
    """An array that a call writes shares memory with one that it reads, or with another it writes."""
    M = 1 << 20
    table, pre, num, par, out, lse, ws, olen = (FAKE + x * M for x in (3, 5, 11, 12, 6, 7, 8, 9))
    c = cache_struct()
    base = dict(num=num, par=par)
    # Two rows of five pages: 40 bytes of page table; 7 pages of 8 heads of 16 slots: 3584 bytes of weights.
    for at in (table + 36, table - 4, FAKE + 2 * M + 3580, FAKE + 64, FAKE + M + 7 * 8 * 16 * 128 * 2 - 4):
        got = calls(L, c, olen=at, **base)
        assert (got["append"], got["evict"]) == (9, 9), hex(at)
    for at in (pre, num + 4, par + 4 * 17):
        assert calls(L, c, olen=at, **base)["append"] == 9
    assert calls(L, c, olen=FAKE + 4 * M, **base)["append"] == 9      # the tokens
    size = 2 * 9 * 32 * 128 * 2                            # of the queries and the output, one row after the other
    for at in (table - 16, table, pre, num, par, FAKE + 2 * M, FAKE + M, FAKE + M - size + 16, FAKE + 4 * M + size - 16, lse, ws):
        assert calls(L, c, out=at, **base)["attend"] == 9, hex(at)
    for at in (table + 36, pre + 4, num, par + 4 * 17, FAKE + 16, out + size - 4, ws + 512):
        assert calls(L, c, lse=at, **base)["attend"] == 9, hex(at)
    for at in (table & ~255, pre, num, par, FAKE + 4 * M, FAKE + M):
        assert calls(L, c, ws=at, **base)["attend"] == 9, hex(at)
    for name, at in (("q", 64), ("lse", 3580), ("pre", 0), ("num", 4), ("par", 3584 - 4 * 18)):
        kw = {**base, name: FAKE + 2 * M + at}
        assert calls(L, c, **kw)["weigh"] == 9, name
    assert calls(L, cache_struct(page_table=FAKE + 2 * M + 4), **base)["weigh"] == 9
    # The extent of pages with large strides is not cut off at 64 bits.
    far = cache_struct(num_pages=(1 << 31) - 1, page_stride=(1 << 38) - 8)
    assert calls(L, far, **base)["attend"] == 9


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,rows", [(1, 4, 1), (1, 4, 3), (9, 4, 1), (9, 4, 3), (1, 4, 90)])
def test_gpu_infinities_in_a_part_that_weighs_nothing(sv, N, G, rows):
    """Infinite values in blocks' parts of a row whose maxima lie so far below another part's that their weight is 0
    in fp32: what comes of them is not finite, whichever block had them."""
    a = Batch((12000,) * rows, N, 1, G, 64, 128, seed=N, poison=False)
    a.q[:] = 1.0
    a.k.clamp_(-0.1, 0.1)
    for b in range(rows):
        p, s = oracle.place(a.table, b, 128 * 40, 128)
        a.k[p, :, s] = 40.0                                # its score is 320, the others' below 1
        for t in range(41, 93):
            p, s = oracle.place(a.table, b, 128 * t + 1, 128)
            a.v[p, 0, s, t - 41] = math.inf
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix))
    got = host(out)
    assert not np.isfinite(got[..., :52]).any() and np.isfinite(got[..., 52:]).all()
    assert np.isfinite(host(lse)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("top", [14.0, 17.0, 18.5])
@pytest.mark.parametrize("rows,n,N,G", [(1, 60000, 1, 2), (1, 60000, 9, 4), (1, 60000, 31, 8), (320, 3000, 1, 4),
                                        (320, 3000, 4, 4), (160, 3000, 9, 4), (80, 3000, 31, 8)])
def test_gpu_halves_of_small_probabilities(sv, rows, n, N, G, top):
    """One entry far above equal ones, whose probabilities lie among a half's smallest numbers: they keep their
    precision. A probability and the output are each rounded by half a step, e relative, and the sums are fp32 (1e-5).
    Probabilities are kept times 2^15, or 2^7 where a key head has more than 16 query rows. A half's smallest step is
    2^-24, half of it 2^-40 or 2^-32 of the largest probability, for each entry; the output's own is 2^-24."""
    a = Batch((n,) * rows, N, 1, G, 64, 128, "f16", seed=N, poison=False)
    a.q[:] = 0.0
    a.q[..., 0] = 1.0
    a.k[:] = 0.0
    a.v[:] = 1.0
    for b in range(rows):
        p, s = oracle.place(a.table, b, 77, 128)
        a.k[p, :, s, 0] = top
        a.v[p, :, s] = 0.0
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), scale=1.0)
    e = 2.0 ** -11
    for i in range(N):
        rest = (n + i) * math.exp(-top)
        want = rest / (1 + rest)
        err = np.abs(host(out)[:, i] - want).max()
        assert err <= want * (2 * e + 1e-5) * (1 + e) + (n + i) * 2.0 ** (-40 if N * G <= 16 else -32) + 2.0 ** -25, (err / want, i)
        assert np.abs(host(lse)[:, i] - (top + math.log1p(rest))).max() <= 2.0 ** -22 * (top + 2)


@pytest.mark.gpu
def test_gpu_tables_wider_than_their_rows(sv):
    """A batch in a table with room for rows far longer than all its pages hold is worked on as in one that fits."""
    a = Batch((500, 900, 130, 1000, 77, 640, 300, 800), 31, 4, 8, 128, 16, seed=1, poison=False)
    fits = sv.attend(a.q, a.cache(sv), dev(a.prefix))
    check_attention(a, *fits, a.prefix, np.full(8, 31), None)
    table = np.full((8, 4096), 1 << 30, np.int32)
    table[:, :a.table.shape[1]] = a.table
    a.table = table
    wide = sv.attend(a.q, a.cache(sv), dev(a.prefix))
    assert torch.equal(wide[0], fits[0]) and torch.equal(wide[1], fits[1])


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,D", [(31, 8, 128), (65, 7, 64), (9, 16, 128)])
def test_gpu_attention_large_trees_in_a_large_pool(sv, N, G, D):
    """A few rows in tables and among pages with room for more keys and values than L2 holds: two query tiles at once,
    in parts."""
    a = Batch((3000, 129, 0), N, 1, G, D, 16, seed=N)
    pages = (800 << 20) // (16 * D * 4)
    at = pages - len(a.k)
    big = [torch.zeros((pages, 1, 16, D), dtype=a.t, device="cuda") for _ in range(2)]
    for x, y in zip(big, (a.k, a.v)):
        x[at:] = y
    table = np.full((3, 65536), 1 << 30, np.int64)
    table[:, :a.table.shape[1]] = np.where(a.table < pages, a.table.astype(np.int64) + at, 1 << 30)
    c = sv.PagedCache(*big, dev(table))
    tree = random_tree(np.random.default_rng(N), 3, N)
    num = np.array([N, N - 3, N], np.int32)
    for parents in (None, tree):
        out, lse = sv.attend(a.q, c, dev(a.prefix), dev(num), dev(parents))
        check_attention(a, out, lse, a.prefix, num, parents)


WIDE_HEADS = [
    # prefix lengths, N, Hkv, group, D, page, dtype, nhd: more than 128 query rows a key head of 256
    ((40, 257, 0, 1000), 33, 2, 8, 256, 16, "bf16", False),
    ((63, 64, 700), 65, 1, 3, 256, 64, "f16", True),
    ((300, 5), 9, 1, 128, 256, 32, "f16", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,N,H,G,D,S,dtype,nhd", WIDE_HEADS)
def test_gpu_heads_of_256_in_several_query_tiles(sv, prefix, N, H, G, D, S, dtype, nhd):
    test_gpu_attention(sv, prefix, N, H, G, D, S, dtype, nhd)
    test_gpu_weights(sv, prefix, N, H, G, D, S, dtype, nhd)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,H,D,S,budget,recent", [
    (tuple(range(16500, 20000, 90)), 8, 64, 128, 9001, 200),      # a block a row and head: keys not held
    ((140000, 500, 131073), 2, 64, 16, 70001, 77),                # clusters whose runs' keys are not held
    ((300000, 262145, 70), 1, 64, 16, 200003, 0),                 # nor page numbers
    ((1 << 20,), 1, 64, 16, 999999, 1000), ((1 << 20,), 1, 128, 16, 12345, 0),   # the longest rows
    (tuple(range(66000, 69900, 300)), 8, 64, 16, 66100, 30),      # page numbers not held, two blocks an SM
])
def test_gpu_evict_of_rows_that_shared_memory_does_not_hold(sv, lengths, H, D, S, budget, recent):
    """Rows whose order keys or page numbers are read again from memory; equal weights across runs."""
    g = torch.Generator(device="cuda").manual_seed(budget)
    used = [-(-n // S) for n in lengths]
    ids = torch.randperm(sum(used) + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(used)), 1 << 30, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    shape = (len(ids), H, S, D)
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(shape[:3], generator=g, device="cuda").mul_(500).floor_()
    old = [x.clone() for x in (k, v, w)]
    olen = dev([0] * len(lengths))
    sv.spec_verify_kv_evict(sv.PagedCache(k, v, table, w), dev(lengths), budget, recent, olen)
    assert olen.tolist() == [min(n, budget) for n in lengths]
    for b, n in enumerate(lengths):
        row = lambda x: x[table[b, :used[b]].long()].transpose(0, 1).flatten(1, 2)[:, :n]   # noqa: E731
        for h in range(H):
            keep = torch.ones(n, dtype=torch.bool, device="cuda")
            if n > budget:
                order = torch.sort(row(old[2])[h, :n - recent], descending=True, stable=True)[1]
                keep[order[budget - recent:]] = False
            for x, o in zip((k, v, w), old):
                assert torch.equal(row(x)[h, :budget], row(o)[h][keep])
                assert torch.equal(row(x)[h, budget:], row(o)[h, budget:])


@pytest.mark.gpu
@pytest.mark.parametrize("N,G,S", [(1, 4, 16), (9, 4, 128)])
def test_gpu_the_longest_row(sv, N, G, S):
    """A row of 1,048,576 entries, the most that there may be, beside a short one: attention and weights against 64 bits.
    Half a step of the probabilities and of the output, and 1e-5 for scores, exponentials and sums."""
    n, D = (1 << 20) - N, 64
    g = torch.Generator(device="cuda").manual_seed(N)
    pages = (1 << 20) // S
    k, v = (torch.randn((pages + 1, 1, S, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, N, G, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).repeat(2, 1)
    table[1, 0] = pages
    w = torch.zeros((pages + 1, 1, S), device="cuda")
    c = sv.PagedCache(k, v, table, w)
    prefix = dev([n, 3])
    out, lse = sv.attend(q, c, prefix)
    sv.spec_verify_kv_weights(q, lse, c, prefix)
    K, V = (x[table[0].long(), 0].reshape(-1, D).double() for x in (k, v))
    s = (q[0].double().reshape(N * G, D) @ K.T / 8).reshape(N, G, -1)
    s.masked_fill_(torch.arange(1 << 20, device="cuda") > n + torch.arange(N, device="cuda")[:, None, None], -math.inf)
    want_lse = torch.logsumexp(s, -1)
    p = torch.exp(s - want_lse[..., None])
    want, mag = p @ V, p @ V.abs()
    e = 2.0 ** -8
    assert ((out[0].double() - want).abs() <= e * want.abs() + (e + 1e-5) * mag).all()
    assert (lse[0].double() - want_lse).abs().max() <= 1e-5
    got = w[table[0].long(), 0].reshape(-1).double()
    assert ((got - p.sum((0, 1))).abs() <= 1e-4 * p.sum((0, 1))).all()
    assert abs(float(w.double().sum()) - 2 * N * G) <= 1e-4 * N * G and torch.isfinite(out[1]).all()


@pytest.mark.gpu
def test_gpu_weights_along_a_path_that_names_a_token_twice(sv):
    a = Batch((40, 7, 130), 5, 2, 4, 64, 16, seed=2)
    path = np.array([[0, 0, 3, 3, 3], [4, 4, 4, 4, 4], [1, 0, 1, 0, 2]], np.int32)
    lse = torch.full((3, 5, 8), 2.0, device="cuda")
    before = host(a.weight)
    sv.spec_verify_kv_weights(a.q, lse, a.cache(sv), dev(a.prefix), None, dev(path))
    want = oracle.weights(host(a.q), host(lse), host(a.k), before, a.table, a.prefix, [5] * 3, path, a.scale)
    assert np.allclose(host(a.weight), want, rtol=1e-5, atol=0)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (9, 4), (31, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gpu_scores_of_tens_of_millions(sv, N, G, dtype):
    """One entry whose score is far beyond all others and beyond what fp32 has fractions for: its value, its score. Its
    probability and the output are each rounded by half a step; the lse by two roundings, a product and a logarithm."""
    B, D = 12, 128
    a = Batch((200,) * B, N, 1, G, D, 16, dtype, seed=N, poison=False)
    a.q[:] = 1500.0
    a.k[:] = 0.0
    a.scale = 0.09
    for b in range(B):
        p, s = oracle.place(a.table, b, 17 * b, 16)
        a.k[p, :, s] = 1000.0 + 117.0 * b                  # exact in fp32: the sum of 128 products, up to 4.4e8
    out, lse = sv.attend(a.q, a.cache(sv), dev(a.prefix), scale=a.scale)
    for b in range(B):
        p, s = oracle.place(a.table, b, 17 * b, 16)
        v, e = host(a.v[p, 0, s]), torch.finfo(a.t).eps / 2
        assert (np.abs(host(out)[b] - v) <= 2 * e * (1 + e) * np.abs(v) + 1e-6).all(), b
        want = 0.09 * 128 * float(a.q[0, 0, 0, 0]) * float(a.k[p, 0, s, 0])
        assert np.abs(host(lse)[b] / want - 1).max() <= 2.0 ** -22
