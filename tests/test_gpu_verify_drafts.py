"""pkvqk_verify_drafts against the oracle's whole-number verdict: every output is equal.

Sums are formed in whole multiples of 2^-44 on both sides, so there is no tolerance.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _softmax(rng, *shape, peak=3.0):
    x = peak * rng.normal(size=shape)
    x = np.exp(x - x.max(-1, keepdims=True))
    return x / x.sum(-1, keepdims=True)


def _probs(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dtype]).cuda()


def _inputs(rng, B, K, V, dtype, lookup=False):
    p = _softmax(rng, B, K + 1, V)
    q = p[:, :K] * np.exp(0.5 * rng.normal(size=(B, K, V)))
    q /= q.sum(-1, keepdims=True)
    drafts = np.array([[rng.choice(V, p=q[b, i]) for i in range(K)] for b in range(B)],
                      np.int32).reshape(B, K)
    u = rng.random((B, K + 1)).astype(np.float32)
    return (_probs(p, dtype), None if lookup else _probs(q, dtype), torch.from_numpy(drafts).cuda(),
            torch.from_numpy(u).cuda())


def _run(lib, p, q, drafts, u, lens=None, seq_lens=None, **more):
    B, K = drafts.shape
    tokens = torch.full((B, K + 1), -77, dtype=torch.int32, device="cuda")
    n = torch.full((B,), -77, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = None if seq_lens is None else torch.full_like(seq_lens, -77)
    lib.verify_drafts(p, q, drafts, u, tokens, n, draft_lens=lens, seq_lens=seq_lens,
                      kept_lens=kept, status_flags=flags, **more)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), n.cpu().numpy(), flags.item(), kept


def _check(lib, p, q, drafts, u, lens=None, flags=0):
    seq_lens = torch.arange(drafts.shape[0], dtype=torch.int32, device="cuda") + 300
    tokens, n, f, kept = _run(lib, p, q, drafts, u, lens, seq_lens)
    ref, ref_n = oracle.verify_drafts(
        p.double().cpu().numpy(), None if q is None else q.double().cpu().numpy(),
        drafts.cpu().numpy(), u.cpu().numpy(), None if lens is None else lens.cpu().numpy())
    assert np.array_equal(n, ref_n), (n, ref_n)
    assert np.array_equal(tokens, ref), (tokens, ref)
    K = drafts.shape[1]
    have = np.full(len(n), K) if lens is None else np.clip(lens.cpu().numpy(), 0, K)
    assert np.array_equal(kept.cpu().numpy(), seq_lens.cpu().numpy() - (have - n))
    assert f == flags
    return tokens, n


# vocabularies below, at and past a CTA's least share, odd ones (scalar loads), and ones
# whose last warps have nothing
@pytest.mark.parametrize("V", [1, 2, 7, 100, 1024, 2048, 4099, 16384, 32768, 50001, 65536, 131072])
@pytest.mark.parametrize("dtype,lookup", [("fp32", False), ("fp32", True), ("bf16", False),
                                          ("fp16", True)])
def test_vocabularies(lib, V, dtype, lookup):
    rng = np.random.default_rng(V)
    B, K = 3, 4
    _check(lib, *_inputs(rng, B, K, V, dtype, lookup))


@pytest.mark.parametrize("B,K", [(1, 1), (1, 0), (2, 31), (2, 32), (2, 33), (1, 255), (77, 3),
                                 (160, 2), (400, 1)])
def test_batches_and_drafts(lib, B, K):
    _check(lib, *_inputs(np.random.default_rng(B + K), B, K, 1500, "fp32"))


def test_ragged_drafts(lib):
    rng = np.random.default_rng(5)
    p, q, drafts, u = _inputs(rng, 8, 5, 3000, "fp32")
    lens = torch.tensor([0, 1, 2, 3, 4, 5, -3, 99], dtype=torch.int32, device="cuda")
    _check(lib, p, q, drafts, u, lens)
    # rows past a sequence's drafts are not read
    p2, q2 = p.clone(), q.clone()
    for b, n in enumerate([0, 1, 2, 3, 4, 5, 0, 5]):
        p2[b, n + 1:] = float("nan")
        q2[b, n:] = float("nan")
    a, b = _run(lib, p, q, drafts, u, lens), _run(lib, p2, q2, drafts, u, lens)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and b[2] == 0


def test_every_draft_kept_and_none(lib):
    rng = np.random.default_rng(6)
    p, q, drafts, u = _inputs(rng, 6, 4, 5000, "fp32")
    u[:, :4] = 0.0                             # 0 < p: kept
    tokens, n = _check(lib, p, q, drafts, u)
    assert (n == 4).all()
    p.scatter_(2, drafts.long()[..., None], 0.0)        # u q < 0 is false: refused
    _, n = _check(lib, p, q, drafts, u)
    assert (n == 0).all()


@pytest.mark.parametrize("u", [0.0, 2.0 ** -149, 0.25, 0.5, 1 - 2.0 ** -24, 1.0, 7.0, -1.0,
                               float("nan"), float("inf"), float("-inf")])
def test_ends_of_the_draw(lib, u):
    """Weights that are whole parts of 1, so that a uniform falls on a border itself."""
    V = 4096
    p = torch.full((2, 1, V), 1.0 / V, device="cuda")
    p[1, 0, :17] = 0.0
    p[1, 0, -9:] = 0.0
    drafts = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    uu = torch.full((2, 1), u, device="cuda")
    tokens, _ = _check(lib, p, None, drafts, uu)
    assert 17 <= tokens[1, 0] < V - 9          # a token without weight is never drawn


def test_draws_follow_the_target(lib):
    """All of a grid of uniforms: each token exactly as often as its weight says."""
    V, m = 64, 512                             # the weights below sum to less
    w = torch.randint(0, 9, (V,), generator=torch.Generator().manual_seed(1)).float()
    w[0] += m - w.sum()
    p = (w / m).cuda().expand(m, 1, V)
    u = ((torch.arange(m) + 0.5) / m).cuda()[:, None].contiguous()
    tokens, _, _, _ = _run(lib, p, None, torch.empty(m, 0, dtype=torch.int32, device="cuda"), u)
    assert np.array_equal(np.bincount(tokens[:, 0], minlength=V), w.numpy().astype(int))


def test_nothing_left_of_the_target(lib):
    rng = np.random.default_rng(7)
    p, _, drafts, u = _inputs(rng, 4, 2, 3000, "fp32")
    q = p[:, :2].clone()
    q[1] = 1.0                                 # p < q everywhere: p itself
    p[2, 0] = 0.0
    p[2, 0, 5] = 1.0                           # a certain draft that p gives all its weight
    u[:, :2] = 1.0
    _check(lib, p, q, drafts, u)
    drafts[2, 0] = 5
    _check(lib, p, None, drafts, u)


def test_bad_probabilities_and_tokens(lib):
    rng = np.random.default_rng(8)
    p, q, drafts, u = _inputs(rng, 6, 3, 5000, "fp32")
    u[:, :3] = 0.0
    drafts[:, 2] = -1                          # reached by every sequence, and refused
    dirty = p.clone()
    dirty[0, 2, 7] = float("nan")
    dirty[1, 2, 8] = -0.5
    dirty[2, 2, 9] = 3.0                       # counts as 1
    dirty[3, 2, 10] = float("inf")             # counts as 1
    _check(lib, dirty, q, drafts, u, flags=lib.FLAG_BAD_VALUE | lib.FLAG_BAD_TOKEN)
    drafts[:, 2] = 5000
    _check(lib, p, None, drafts, u, flags=lib.FLAG_BAD_TOKEN)
    # a bad draft that is not reached says nothing
    drafts[:, 0] = p[:, 0].argmin(-1).int()
    p.scatter_(2, drafts[:, :1].long().expand(-1, 4)[..., None].clamp(max=4999), 0.0)
    _, n = _check(lib, p, q, drafts, u)
    assert (n == 0).all()
    # a row without any weight
    p[4] = 0.0
    tokens, _ = _check(lib, p, q, drafts, u, flags=lib.FLAG_BAD_VALUE)
    assert tokens[4].tolist() == [-1] * 4


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_rows_and_alignment(lib, dtype):
    """Rows of wider tensors, starting on and off 16-byte boundaries, give the same."""
    rng = np.random.default_rng(9)
    B, K, V = 3, 2, 4096
    p, q, drafts, u = _inputs(rng, B, K, V, dtype)
    want = _run(lib, p, q, drafts, u)
    for shift in (0, 1, 8):
        wide = torch.full((B, K + 3, V + 24), float("nan"), dtype=TYPES[dtype], device="cuda")
        wide[:, :K + 1, shift:shift + V] = p
        wide_q = torch.full((K, B, V + 16), float("nan"), dtype=TYPES[dtype], device="cuda")
        wide_q[:, :, :V] = q.transpose(0, 1)
        got = _run(lib, wide[:, :, shift:shift + V], wide_q.transpose(0, 1)[:, :, :V], drafts, u)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0


def test_lengths_in_place_on_a_side_stream_and_in_a_graph(lib):
    rng = np.random.default_rng(10)
    p, q, drafts, u = _inputs(rng, 8, 4, 20000, "fp32")
    want = _run(lib, p, q, drafts, u)
    lens = torch.full((8,), 500, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(8, 5, dtype=torch.int32, device="cuda")
    n = torch.zeros(8, dtype=torch.int32, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        lib.verify_drafts(p, q, drafts, u, tokens, n, seq_lens=lens, kept_lens=lens)
    torch.cuda.current_stream().wait_stream(s)
    for i in range(1, 3):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(tokens.cpu().numpy(), want[0])
        assert np.array_equal(lens.cpu().numpy(), 500 - i * (4 - want[1]))
