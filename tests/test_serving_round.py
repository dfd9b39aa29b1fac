"""Rounds of a batch on one prompt, step by step against the same rounds on pages of each row's own: append, shared
attention, shaping, verification, counts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_55_gb300 as m
    m.build_library()
    return m


@pytest.mark.gpu
def test_gpu_rounds_of_one_prompt_step_by_step(sv):
    """Two roundings of the attention's output (2^-8 of it, about 0.4% of the logits' spread of 1) may move a logit over a
    border when logits are rounded to whole numbers: about 2 * 0.004 of them. With 10 logits a row that depend on the
    attention, nine rows of ten have the same rounded logits; these have to have the same tokens, numbers and counts."""
    B, N, H, G, D, S, V, live = 40, 5, 2, 4, 64, 16, 512, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    front, rows = 96, 700                      # (room for fronts to be worth it)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.zeros((B, rows), **i32)
    table[:, :6] = torch.arange(6, device="cuda")
    own = 20                                   # pages of a row's own; the columns behind them are never reached
    table[:, 6:6 + own] = 6 + torch.arange(B * own, device="cuda").view(B, -1)
    pages = 6 + B * rows                       # (more than are used: room for fronts)
    k, v = (torch.randn((pages, H, S, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    shared = sv.PagedCache(k, v, table)
    used = table[:, :6 + own].long()
    apart = sv.PagedCache(k[used].flatten(0, 1).contiguous(), v[used].flatten(0, 1).contiguous(),
                          torch.arange(B * (6 + own), **i32).view(B, -1))
    n = front + 3 + torch.arange(B, **i32) % 5
    common, start = torch.full((B,), front, **i32), torch.tensor([0, B], **i32)
    head = torch.zeros((H * G * D, V), device="cuda")
    head[:, :live] = torch.randn((H * G * D, live), generator=g, device="cuda")
    rest = torch.randint(-3, 4, (V,), generator=g, device="cuda").float()
    counts = [torch.zeros((B, V), dtype=torch.int16, device="cuda") for _ in range(2)]
    prompt = torch.randint(0, V, (B, 30), generator=g, **i32)
    for c in counts:
        sv.spec_verify_count_tokens(prompt, None, c, prompt=True)
    emitted = np.zeros((B, V), np.int64)
    penalty, frequency = torch.full((B,), 1.25, device="cuda"), torch.full((B,), 0.5, device="cuda")
    temperature = (torch.arange(B, device="cuda") % 3 != 0).float()
    kept = several = 0
    for _ in range(6):
        qkv = torch.randn((B, N, H * G + 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        drafts = torch.randint(0, 12, (B, N - 1), generator=g, **i32)
        length = torch.arange(B, **i32) % N
        draft = 2 * torch.randn((B, N - 1, V), generator=g, device="cuda").to(torch.bfloat16)
        u = torch.rand((B, N + 1), generator=g, device="cuda")
        ends = []
        for cache, c, attend in ((shared, counts[0], lambda *x: sv.attend_shared(x[0], x[1], x[2], common, start, x[3])),
                                 (apart, counts[1], sv.attend)):
            sv.spec_verify_kv_append(qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:], cache, n, length + 1)
            out, lse = attend(qkv[:, :, :H * G], cache, n, length + 1)
            x = out.flatten(2).float()
            spread = x.square().sum(-1, keepdim=True).sqrt() + 1e-6
            logits = torch.round(torch.matmul((x / spread).double(), head.double()).float() + rest).to(torch.bfloat16)
            t, d = logits.clone(), draft.clone()
            sv.spec_verify_shape_logits(t, length + 1, drafts, None, c, penalty, frequency)
            sv.spec_verify_shape_logits(d, length, drafts, None, c, penalty, frequency)
            tokens, num, _ = sv.verify(t, d, drafts, length, temperature, u)
            sv.spec_verify_count_tokens(tokens, num, c)
            ends.append((out.float(), lse, logits, t, d, tokens, num))
        (o1, z1, l1, t1, d1, k1, m1), (o2, z2, l2, t2, d2, k2, m2) = ends
        assert float((o1 - o2).abs().max()) <= 2.0 ** -7 * float(o2.abs().max()) and float((z1 - z2).abs().max()) <= 1e-5
        assert int(m1.min()) >= 1 and int(m2.min()) >= 1
        inside = torch.arange(N, device="cuda")[None] <= length[:, None]
        same = ((l1 == l2).all(-1) | ~inside).all(1)
        kept += int(same.sum())
        several += int((m1[same] > 1).sum())
        assert torch.equal(torch.where(inside[..., None], t1, 0)[same], torch.where(inside[..., None], t2, 0)[same])
        assert torch.equal(d1, d2)             # the drafter's logits do not depend on the attention
        assert torch.equal(m1[same], m2[same]) and torch.equal(k1[same], k2[same])
        assert torch.equal(counts[0][same], counts[1][same])
        out = k1.cpu().numpy()
        for b, m in enumerate(m1.tolist()):
            for x in out[b, :m]:
                emitted[b, x] += 1
        assert np.array_equal(counts[0].cpu().numpy() & 32767, emitted)
        new = torch.empty_like(n)
        sv.spec_verify_kv_rollback(n, length, m1, None, new, None, gamma_max=N - 1)
        assert torch.equal(new, n + m1)
        counts[1][~same] = counts[0][~same]    # rows on the other side of a border go on from the same text
        n = new
    said = torch.zeros((B, V), dtype=torch.bool, device="cuda").scatter_(1, prompt.long(), True)
    assert torch.equal(counts[0] < 0, said)
    assert kept >= 0.75 * 6 * B and several > 0
