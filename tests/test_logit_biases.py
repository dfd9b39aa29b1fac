"""Several biases of one token: they go onto its logit one after the other, in their order, in fp32.

The calls below have biases and penalties whose fp32 results are exact by construction or are computed here by the same
additions, so logits are compared bit for bit.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


def in_order(z, tokens, bias):
    """The logits [B, N, V] fp32 plus each row's biases, one after the other in fp32."""
    z = z.copy()
    with np.errstate(over="ignore"):
        for b in range(z.shape[0]):
            for t, x in zip(tokens[b], bias[b]):
                if 0 <= t < z.shape[2]:
                    z[b, :, t] = z[b, :, t] + np.float32(x)
    return z


def bits(x):
    return x.cpu().view(torch.int16 if x.element_size() == 2 else torch.int32)


def shaped(sv, z, bias_tokens, bias, dtype, **rest):
    """z: fp32 values of the type."""
    got = torch.from_numpy(z).to(TYPES[dtype]).cuda()
    sv.spec_verify_shape_logits(got, bias_tokens=torch.from_numpy(bias_tokens).cuda(), bias=torch.from_numpy(bias).cuda(), **rest)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 33])
def test_biases_that_cancel(sv, V, dtype):
    """Beside 100,000,000 a 1 is lost, as in the same fp32 additions; three numbers of 2^127 whose last sum is in range."""
    z = np.zeros((2, 3, V), np.float32)
    z[..., 3], z[..., 5], z[..., 7] = 1.0, -2.0 ** 127, 4.0
    tokens = np.array([[3, 5, 9, 3, 5, 7], [5, 3, 7, 5, -1, 3]], np.int32)
    bias = np.array([[1e8, 2.0 ** 127, 2.5, -1e8, 2.0 ** 127, 0.5], [2.0 ** 127, 1e8, 1.0, 2.0 ** 127, 7.0, -1e8]], np.float32)
    got = shaped(sv, z, tokens, bias, dtype)
    assert (got[..., 3] == 0).all() and (got[..., 5] == 2.0 ** 127).all()
    assert torch.equal(bits(got), bits(torch.from_numpy(in_order(z, tokens, bias)).to(TYPES[dtype])))


@pytest.mark.parametrize("tree", [False, True])
def test_biases_after_the_penalties(sv, tree):
    """A token of the text, of the round, and of neither, each with biases that cancel: the penalised logit goes first."""
    z = np.full((1, 3, 24), 2.0, np.float32)
    tokens = np.array([[4, 11, 20, 4, 11, 20, 2]], np.int32)
    bias = np.array([[1e8, 2.0 ** 24, 1e8, -1e8, -2.0 ** 24, -1e8, 0.25]], np.float32)
    counts = np.zeros((1, 24), np.int16)
    counts[0, 4] = 1
    drafts = torch.tensor([[11, 11, 11]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda") if tree else None
    got = shaped(sv, z, tokens, bias, "f32", tokens=drafts, tree_parents=parents, counts=torch.from_numpy(counts).cuda(),
                repetition=torch.full((1,), 2.0, device="cuda"), presence=torch.full((1,), 2.0, device="cuda"))
    assert (got[0, :, 4] == 0).all() and (got[0, :, 20] == 0).all() and (got[0, :, 2] == 2.25).all()
    # 2 / 2 - 2 = -1 where the round has said it, and 2^24 - 1 is an fp32 number; else 2.
    said = [tree, True, True]
    assert got[0, :, 11].tolist() == [-1.0 if s else 2.0 for s in said]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,V,K", [(6, 6, 162, 276), (3, 9, 2050, 1024), (2, 65, 8, 1024), (2, 4, 5000, 300), (1, 1, 1, 9)])
def test_many_biases_of_many_sizes(sv, B, N, V, K, dtype):
    rng = np.random.default_rng(V + K)
    z = torch.from_numpy((rng.standard_normal((B, N, V)) * 4).astype(np.float32)).to(TYPES[dtype]).float().numpy()
    tokens = rng.integers(-1, min(V, 200) + 1, (B, K)).astype(np.int32)
    bias = (rng.standard_normal((B, K)) * 2.0 ** rng.integers(-20, 20, (B, K))).astype(np.float32)
    got = shaped(sv, z, tokens, bias, dtype)
    assert torch.equal(bits(got), bits(torch.from_numpy(in_order(z, tokens, bias)).to(TYPES[dtype])))
