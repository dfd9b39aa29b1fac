"""Shaping of a round's logits (penalties, biases, masks) and the token counts it reads: oracle pins and refusals on
the CPU, GPU parity against the fp64 oracle.

Tolerance of a shaped logit: a division or product, a product and two differences, and a sum for each bias of its token,
each off by at most 2^-24 of the magnitudes that went in (the oracle's `size`), then half a step of the logits' type.
Logits that nothing concerns are compared bit for bit, counts exactly.
"""
import numpy as np
import pytest

from oracle import logits_oracle as oracle

torch = pytest.importorskip("torch")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------
# Oracle pins (CPU)
# ------------------------------------------------------------------------------------------------

def test_oracle_penalties_by_hand():
    z = np.array([[[2.0, -2.0, 1.0, 0.0, 5.0]] * 3])
    counts = np.array([[0, 3, -32768, -32767, 0]], np.int16)      # 1: three times; 2: prompt; 3: prompt and once
    out, changed, _ = oracle.shape(z, np.array([2]), np.array([[4, 0]]), None, counts, [2.0], [0.5], [0.25])
    assert out[0, 0].tolist() == [2.0, -4.0 - 1.5 - 0.25, 0.5, 0.0 - 0.5 - 0.25, 5.0]
    assert out[0, 1].tolist() == out[0, 0].tolist()[:4] + [2.5 - 0.75]
    assert out[0, 2].tolist() == z[0, 2].tolist() and not changed[0, 2].any()
    assert changed[0, 0].tolist() == [False, True, True, True, False]


def test_oracle_tree_bias_mask_by_hand():
    z = np.zeros((1, 4, 3))
    parents = np.array([[-1, 0, 0, 1]])
    tokens = np.array([[0, 1, 0, 1]])
    out, _, _ = oracle.shape(z, None, tokens, parents, None, None, [1.0], None)
    assert out[0].tolist() == [[-1, 0, 0], [-1, -1, 0], [-2, 0, 0], [-1, -2, 0]]
    out, _, _ = oracle.shape(z, None, None, None, None, None, None, None, [[2, 7, 2, -1]], [[1.0, 9.0, 0.5, 9.0]],
                             np.array([[[0b110]]]))
    assert out[0].tolist() == [[-np.inf, 0, 1.5]] * 4
    bad, changed, _ = oracle.shape(z, None, tokens, np.array([[-1, 0, 3, 1]]), None, None, [1.0], None)
    assert not changed.any()


def test_oracle_counts_by_hand():
    c = np.array([[0, 32766, -1, 5]], np.int16)
    got = oracle.count(c, np.array([[1, 1, 2, 0, 0, 9, -1, 3]]), np.array([7]))
    assert got.tolist() == [[2, 32767, -1, 5]]
    assert oracle.count(c, np.array([[0, 1]]), None, True).tolist() == [[-32768, -2, -1, 5]]
    assert oracle.count(c, np.array([[0, 1]]), np.array([-1])).tolist() == c.tolist()


# ------------------------------------------------------------------------------------------------
# Refusals (CPU: no call gets as far as the device)
# ------------------------------------------------------------------------------------------------

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m.lib()


def shape_status(L, **kw):
    a = dict(z=FAKE, num=FAKE + (1 << 30), tok=FAKE + (2 << 30), T=8, par=FAKE + (3 << 30), cnt=FAKE + (4 << 30),
             rep=FAKE + (5 << 30), fre=FAKE + (6 << 30), pre=FAKE + (7 << 30), bt=FAKE + (8 << 30), bi=FAKE + (9 << 30),
             K=16, mask=FAKE + (10 << 30), mp=8, B=4, N=8, V=1000, dt=1)
    a.update(kw)
    return L.spec_verify_shape_logits(a["z"], a["num"], a["tok"], a["T"], a["par"], a["cnt"], a["rep"], a["fre"],
                                      a["pre"], a["bt"], a["bi"], a["K"], a["mask"], a["mp"], a["B"], a["N"], a["V"],
                                      a["dt"], None)


@pytest.mark.parametrize("change,status", [
    (dict(z=None), 1), (dict(bt=None), 1), (dict(bi=None), 1), (dict(tok=None), 1),
    (dict(dt=2), 3), (dict(dt=9), 3),
    (dict(B=0), 2), (dict(N=0), 2), (dict(N=66), 2), (dict(V=0), 2), (dict(V=(1 << 24) + 1), 2), (dict(T=7), 2),
    (dict(T=6, par=None), 2), (dict(K=1025), 2), (dict(K=-1), 2), (dict(mp=2), 2),
    (dict(z=FAKE + 1), 5), (dict(dt=0, z=FAKE + 2), 5), (dict(num=FAKE + (1 << 30) + 2), 5),
    (dict(cnt=FAKE + (4 << 30) + 1), 5), (dict(bi=FAKE + (9 << 30) + 1), 5), (dict(mask=FAKE + (10 << 30) + 2), 5),
    (dict(cnt=FAKE + 2 * 4 * 8 * 1000 - 2), 9), (dict(rep=FAKE), 9), (dict(mask=FAKE + 64), 9),
    (dict(tok=FAKE - 4 * 4 * 8 + 4), 9),
])
def test_shape_refusals(L, change, status):
    assert shape_status(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(t=None), 1), (dict(c=None), 1), (dict(B=0), 2), (dict(M=0), 2), (dict(V=0), 2), (dict(V=(1 << 24) + 1), 2),
    (dict(B=(1 << 20) + 1), 2), (dict(M=(1 << 30) + 1), 2), (dict(t=FAKE + 2), 5), (dict(n=FAKE + (1 << 20) + 1), 5),
    (dict(c=FAKE + (1 << 30) + 1), 5), (dict(c=FAKE + 8), 9), (dict(n=FAKE + (1 << 30) + 8), 9),
])
def test_count_refusals(L, change, status):
    a = dict(t=FAKE, n=FAKE + (1 << 20), c=FAKE + (1 << 30), B=4, M=9, V=1000)
    a.update(change)
    assert L.spec_verify_count_tokens(a["t"], a["n"], a["c"], 0, a["B"], a["M"], a["V"], None) == status


def test_binding_refusals():
    """The binding's own checks, on CPU tensors (no call is made)."""
    import speculative_decoding_verification_55_gb300 as sv
    z = torch.zeros((2, 3, 40))
    i32 = torch.int32
    with pytest.raises(ValueError, match="logits"):
        sv.spec_verify_shape_logits(z[:, :, ::2])
    with pytest.raises(ValueError, match="logits"):
        sv.spec_verify_shape_logits(z[0])
    with pytest.raises(TypeError, match="logits"):
        sv.spec_verify_shape_logits(z.half())
    with pytest.raises(ValueError, match="go together"):
        sv.spec_verify_shape_logits(z, bias=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="mask"):
        sv.spec_verify_shape_logits(z, mask=torch.zeros((2, 2, 2), dtype=i32))
    with pytest.raises(ValueError, match="mask"):
        sv.spec_verify_shape_logits(z, mask=torch.zeros((2, 3, 1), dtype=i32))
    with pytest.raises(TypeError, match="counts"):
        sv.spec_verify_shape_logits(z, counts=torch.zeros((2, 40), dtype=i32))
    with pytest.raises(ValueError, match="repetition"):
        sv.spec_verify_shape_logits(z, repetition=torch.ones(3))
    with pytest.raises(ValueError, match="tokens"):
        sv.spec_verify_shape_logits(z, tokens=torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_shape_logits(z)
    with pytest.raises(TypeError, match="counts"):
        sv.spec_verify_count_tokens(torch.zeros((2, 3), dtype=i32), None, torch.zeros((2, 40), dtype=i32))
    with pytest.raises(ValueError, match="num"):
        sv.spec_verify_count_tokens(torch.zeros((2, 3), dtype=i32), torch.zeros(3, dtype=i32),
                                    torch.zeros((2, 40), dtype=torch.int16))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_count_tokens(torch.zeros((2, 3), dtype=i32), None, torch.zeros((2, 40), dtype=torch.int16))


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


def trees(rng, B, N):
    p = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        p[:, i] = np.maximum(0, i - 1 - rng.integers(0, 5, B))
    return p


def inputs(rng, B, N, V, dtype, tree=False, mask="some", positions=None, K=12, history=40):
    """A call's arguments in NumPy, every kind of row and token among them; logits in a type's values."""
    a = {}
    z = (rng.standard_normal((B, N, V)) * 4).astype(np.float32)
    flat = z.reshape(-1)
    odd = rng.integers(0, flat.size, min(200, flat.size))
    flat[odd] = rng.choice(np.array([np.inf, -np.inf, 0.0, -0.0, 3e38, -3e38], np.float32), odd.size)
    a["logits"] = torch.from_numpy(z).to(TYPES[dtype])
    a["num"] = rng.integers(0, N + 1, B).astype(np.int32)
    a["num"][: min(B, 3)] = np.array([N, 0, N], np.int32)[: min(B, 3)]
    if B > 6:
        a["num"][3:6] = [-1, N + 1, 1]
    few = min(V, 60)                           # tokens repeat: in the text, in the round, and each other
    a["tokens"] = rng.integers(0, few, (B, N)).astype(np.int32)
    a["tokens"][rng.random((B, N)) < 0.1] = -1
    a["tokens"][rng.random((B, N)) < 0.1] = V
    a["parents"] = trees(rng, B, N) if tree else None
    if tree and B > 7:
        a["parents"][6, N // 2] = N            # not a tree where the row has that many nodes
    c = np.zeros((B, V), np.uint16)
    for b in range(B):
        np.add.at(c[b], np.append(rng.integers(0, few, history), rng.integers(0, V, history)), 1)
        c[b, rng.integers(0, V, history)] |= 1 << 15
    c[0, V - 1] = 0xffff                       # 32767 times, and in the prompt
    a["counts"] = c.view(np.int16)
    a["repetition"] = rng.uniform(0.7, 1.6, B).astype(np.float32)
    a["frequency"] = rng.uniform(-0.2, 0.8, B).astype(np.float32)
    a["presence"] = rng.uniform(-0.2, 0.8, B).astype(np.float32)
    a["bias_tokens"] = np.concatenate([rng.integers(0, few, (B, K // 2)), rng.integers(-1, V + 1, (B, K - K // 2))], 1).astype(np.int32)
    a["bias"] = (rng.standard_normal((B, K)) * 3).astype(np.float32)
    W, P = -(-V // 32), positions or N
    if mask == "some":                         # rows of random words, of all ones, of zeros, and with few ones
        m = rng.integers(-2 ** 31, 2 ** 31, (B, P, W)).astype(np.int32)
        m[0::4] = -1
        m[1::4] = 0
        m[1::4, :, W // 2] = 1 << 5
        m[3::4, :, : W // 2] = -1
        a["mask"] = m
    else:
        a["mask"] = None
    return a


ORDER = ("num", "tokens", "parents", "counts", "repetition", "frequency", "presence", "bias_tokens", "bias", "mask")
NAMES = dict(num="num_positions", parents="tree_parents")


def on_gpu(a):
    return {NAMES.get(k, k): None if a[k] is None else torch.from_numpy(a[k]).cuda() for k in ORDER}


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


def check(got, before, a, extra=8):
    z = before.double().numpy()
    want, changed, size = oracle.shape(z, *(a[k] for k in ORDER))
    half = torch.finfo(before.dtype).eps / 2
    same = torch.from_numpy(~changed)
    assert torch.equal(bits(got)[same], bits(before)[same])
    g = got.double().numpy()
    # What lies beyond the type's largest number by half a step has become an infinity.
    most = torch.finfo(before.dtype).max
    inside = changed & np.isfinite(want) & (np.abs(want) <= most)
    slack = extra * 2.0 ** -24 * size[inside]
    assert np.all(np.abs(g[inside] - want[inside]) <= half * (np.abs(want[inside]) + slack) + slack)
    rest = changed & ~inside & ~np.isnan(want)
    finite = rest & np.isfinite(want)
    assert np.all(np.abs(g[finite]) >= most) and np.all(np.sign(g[finite]) == np.sign(want[finite]))
    assert np.array_equal(g[rest & ~finite], want[rest & ~finite])
    assert np.isnan(g[changed & np.isnan(want)]).all()


CASES = [  # B, N, V, dtype, tree, mask, positions
    (1, 1, 1, "f32", False, "some", None), (1, 1, 8, "bf16", False, "some", None), (9, 5, 33, "bf16", False, "some", None),
    (9, 5, 40, "f32", True, "some", None), (9, 4, 1001, "bf16", True, "some", 1), (9, 4, 1001, "f32", False, "none", None),
    (12, 6, 2048, "bf16", False, "some", None), (9, 9, 2056, "bf16", False, "some", 1), (9, 65, 520, "f32", True, "some", None),
    (9, 65, 777, "bf16", False, "some", None), (9, 7, 32000, "bf16", False, "none", None), (8, 5, 32000, "f32", False, "some", None),
    (5, 31, 10008, "bf16", True, "some", None), (9, 2, 32001, "f32", True, "some", None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,V,dtype,tree,mask,positions", CASES)
def test_shape_parity(sv, B, N, V, dtype, tree, mask, positions):
    rng = np.random.default_rng(B * 1000 + N * 10 + V)
    a = inputs(rng, B, N, V, dtype, tree, mask, positions)
    z = a["logits"].cuda()
    sv.spec_verify_shape_logits(z, **on_gpu(a))
    check(z.cpu(), a["logits"], a, 4 + a["bias"].shape[1])


@pytest.mark.gpu
@pytest.mark.parametrize("left", [
    ("tokens", "parents"), ("counts",), ("repetition", "frequency"), ("repetition", "frequency", "presence"),
    ("bias_tokens", "bias"), ("mask", "num"), ("repetition", "frequency", "presence", "bias_tokens", "bias"),
    ("repetition", "frequency", "presence", "mask"), ("repetition", "frequency", "presence", "bias_tokens", "bias", "mask"),
    ("tokens", "parents", "counts", "mask"),
])
@pytest.mark.parametrize("V", [1000, 1003])
def test_shape_parts(sv, left, V):
    """Each part of a call alone, and each left out; what a call with nothing to do leaves alone."""
    a = inputs(np.random.default_rng(V), 9, 6, V, "bf16", True)
    for k in left:
        a[k] = None
    z = a["logits"].cuda()
    sv.spec_verify_shape_logits(z, **on_gpu(a))
    check(z.cpu(), a["logits"], a, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,V,K,tree", [(6, 6, 162, 276, False), (4, 46, 256, 236, True), (3, 9, 2050, 1024, False), (2, 65, 70, 1024, True)])
def test_shape_many_special_tokens(sv, B, N, V, K, tree):
    """More biases than tokens, most of the tokens in the round: each named many times."""
    rng = np.random.default_rng(V)
    a = inputs(rng, B, N, V, "f32", tree, "some", None, K, 20)
    a["tokens"] = rng.integers(-1, V + 1, (B, N)).astype(np.int32)
    a["num"][:] = N
    z = a["logits"].cuda()
    sv.spec_verify_shape_logits(z, **on_gpu(a))
    check(z.cpu(), a["logits"], a, 4 + K)


@pytest.mark.gpu
def test_shape_nan(sv):
    """NaN is barred like anything else, stays where nothing concerns it, and stays NaN where something does."""
    z = torch.full((2, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    before = z.clone()
    mask = torch.full((2, 1, 2), -2, dtype=torch.int32, device="cuda")          # bars tokens 0 and 32
    counts = torch.zeros((2, 64), dtype=torch.int16, device="cuda")
    counts[:, 9] = 1
    sv.spec_verify_shape_logits(z, counts=counts, frequency=torch.ones(2, device="cuda"), mask=mask)
    barred = torch.zeros(64, dtype=torch.bool, device="cuda")
    barred[[0, 32]] = True
    assert bool((z[..., barred] == -float("inf")).all())
    barred[9] = True
    assert torch.equal(bits(z)[..., ~barred], bits(before)[..., ~barred])
    assert bool(z[..., 9].isnan().all())


@pytest.mark.gpu
def test_shape_many_groups_and_odd_places(sv):
    """Rows long and many enough for four groups a thread; logits and counts that are not on 16-byte boundaries."""
    rng = np.random.default_rng(5)
    a = inputs(rng, 80, 2, 128256, "bf16", False, "some", 1, K=40)
    want = a["logits"].cuda()
    sv.spec_verify_shape_logits(want, **on_gpu(a))
    for b in (0, 1, 2, 40, 79):                # (the oracle takes a while for all)
        one = {k: None if a[k] is None else a[k][b:b + 1] for k in ("logits",) + ORDER}
        check(want[b:b + 1].cpu(), one["logits"], one, 44)
    g = on_gpu(a)
    for off in (1, 4):
        room = torch.empty(a["logits"].numel() + off, dtype=torch.bfloat16, device="cuda")
        z = room[off:].view(a["logits"].shape)
        z.copy_(a["logits"])
        sv.spec_verify_shape_logits(z, **g)
        assert torch.equal(bits(z), bits(want))
    c = torch.empty(g["counts"].numel() + 1, dtype=torch.int16, device="cuda")[1:].view(g["counts"].shape)
    c.copy_(g["counts"])
    z = a["logits"].cuda()
    sv.spec_verify_shape_logits(z, **dict(g, counts=c))
    assert torch.equal(bits(z), bits(want))


@pytest.mark.gpu
def test_shape_beyond_32_bits(sv):
    """A batch of more than 2^31 logits: its last row is what that row alone is."""
    B, N, V = 1100, 8, 256000
    rng = np.random.default_rng(6)
    a = inputs(rng, 1, N, V, "bf16")
    g = on_gpu(a)
    big = {k: None if x is None else x.expand(B, *x.shape[1:]).contiguous() for k, x in g.items()}
    z = torch.zeros((B, N, V), dtype=torch.bfloat16, device="cuda")
    z[0], z[-1] = a["logits"][0], a["logits"][0]
    sv.spec_verify_shape_logits(z, **big)
    check(z[-1:].cpu(), a["logits"], a, 16)
    assert torch.equal(bits(z[0]), bits(z[-1]))


def counted(rng, B, M, V, num="some"):
    few = min(V, 30)
    tokens = np.where(rng.random((B, M)) < 0.7, rng.integers(0, few, (B, M)), rng.integers(-1, V + 1, (B, M))).astype(np.int32)
    counts = rng.integers(0, 4, (B, V)).astype(np.uint16)
    counts[:, ::3] |= 1 << 15
    counts[:, : min(V, 4)] = [32766, 0xfffe, 32767, 0][: min(V, 4)]
    n = rng.integers(0, M + 1, B).astype(np.int32)
    if B > 4:
        n[:4] = [-1, 0, M, M + 1]
    return tokens, None if num is None else n, counts.view(np.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("B,M,V", [(1, 1, 1), (7, 9, 33), (64, 65, 1001), (5, 5000, 100), (3, 1025, 128256), (1024, 9, 32000),
                                   (2, 200000, 9000)])
def test_count_parity(sv, B, M, V, prompt):
    rng = np.random.default_rng(M + V)
    for num in ("some", None):
        tokens, n, counts = counted(rng, B, M, V, num)
        got = torch.from_numpy(counts).cuda()
        sv.spec_verify_count_tokens(torch.from_numpy(tokens).cuda(), None if n is None else torch.from_numpy(n).cuda(), got, prompt)
        assert np.array_equal(got.cpu().numpy(), oracle.count(counts, tokens, n, prompt))


@pytest.mark.gpu
def test_count_leaves_its_surroundings(sv):
    """Counts in the middle of an allocation, at an odd place: their neighbours stay."""
    room = torch.full((3 * 7 + 2,), 77, dtype=torch.int16, device="cuda")
    counts = room[1:-1].view(3, 7)
    counts.zero_()
    tokens = torch.tensor([[0, 6, 6], [6, 0, 0], [6, 6, 6]], dtype=torch.int32, device="cuda")
    sv.spec_verify_count_tokens(tokens, None, counts)
    sv.spec_verify_count_tokens(tokens[:, :1].contiguous(), None, counts, prompt=True)
    assert counts.cpu().tolist() == [[1 - 32768, 0, 0, 0, 0, 0, 2], [2, 0, 0, 0, 0, 0, 1 - 32768], [0, 0, 0, 0, 0, 0, 3 - 32768]]
    assert room[0].item() == 77 and room[-1].item() == 77


@pytest.mark.gpu
def test_shape_and_count_captured(sv):
    """A graph of both calls, replayed on new contents and on another stream, does what the calls do."""
    rng = np.random.default_rng(8)
    a = inputs(rng, 9, 5, 1000, "bf16")
    g = on_gpu(a)
    z, counts0 = a["logits"].cuda(), g["counts"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_verify_shape_logits(z, **g)
        sv.spec_verify_count_tokens(g["tokens"], g["num_positions"], g["counts"])
    for seed in (1, 2):
        b = inputs(np.random.default_rng(seed), 9, 5, 1000, "bf16")
        n = on_gpu(b)
        want, want_counts = b["logits"].cuda(), n["counts"].clone()
        sv.spec_verify_shape_logits(want, **n)
        sv.spec_verify_count_tokens(n["tokens"], n["num_positions"], want_counts)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            z.copy_(b["logits"])
            for k, x in n.items():
                if x is not None:
                    g[k].copy_(x)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(z), bits(want)) and torch.equal(g["counts"], want_counts)
    assert not torch.equal(counts0, g["counts"])


@pytest.mark.gpu
def test_masked_round_verifies(sv):
    """What a verification emits from shaped logits is allowed, and its counts are those of the emitted tokens."""
    B, G, V = 40, 4, 1000
    g = torch.Generator(device="cuda").manual_seed(3)
    target = torch.randn((B, G + 1, V), generator=g, device="cuda").to(torch.bfloat16)
    draft = torch.randn((B, G, V), generator=g, device="cuda").to(torch.bfloat16)
    allowed = torch.rand((B, 1, V), generator=g, device="cuda") < 0.02
    allowed[..., 5] = True
    words = torch.zeros((B, 1, 32), dtype=torch.int32, device="cuda")
    padded = torch.nn.functional.pad(allowed, (0, 24))
    for k in range(32):
        words |= padded[..., k::32].int() << k
    counts = torch.zeros((B, V), dtype=torch.int16, device="cuda")
    penalty = torch.full((B,), 1.2, device="cuda")
    length = torch.arange(B, device="cuda", dtype=torch.int32) % (G + 1)
    ids = torch.rand((B, G, V), generator=g, device="cuda").masked_fill_(~allowed, 0).argmax(-1).int()
    temperature = (torch.arange(B, device="cuda") % 2).float()
    seen = np.zeros((B, V), np.int64)
    for _ in range(3):
        t, d = target.clone(), draft.clone()
        sv.spec_verify_shape_logits(t, length + 1, ids, None, counts, penalty, mask=words)
        sv.spec_verify_shape_logits(d, length, ids, None, counts, penalty, mask=words)
        u = torch.rand((B, G + 2), generator=g, device="cuda")
        tokens, num, _ = sv.verify(t, d, ids, length, temperature, u)
        assert int(num.min()) >= 1
        sv.spec_verify_count_tokens(tokens, num, counts)
        out = tokens.cpu().numpy()
        for b in range(B):
            for x in out[b, : int(num[b])]:
                seen[b, x] += 1
                assert bool(allowed[b, 0, x])
    assert np.array_equal(counts.cpu().numpy(), seen)
