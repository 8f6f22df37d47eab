"""GPU parity of pkvqk_norm_rope_append_q8 in calls large enough for the kernel's narrow
form (four CTAs an SM), on both sides of the threshold between the forms."""

import os
import re

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import bf16_ulp_distance, bits
from tests._q8 import CLASSES, Q8, check_appended, code_bytes
from tests.test_gpu_q8_append import _before, _check, _exact, _run, _table

pytestmark = pytest.mark.gpu

_SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_qk_gb300", "csrc", "norm_rope_append_q8.cu")
with open(_SRC, encoding="utf-8") as f:
    MANY_TOKENS = int(re.search(r"constexpr int kManyTokens = (\d+);", f.read()).group(1))


def _problem(Hq, Hkv, bs, new, priors, seed, extra=2):
    lens = [c + n for c, n in zip(priors, new)]
    nb = sum(-(-n // bs) for n in lens) + extra
    p = workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, new, nb, seed, "cuda")
    # values of very different size from token to token: groups grow
    g = torch.Generator(device="cuda").manual_seed(seed)
    p.v = (p.v.float() * torch.randn(p.T, Hkv, 1, device="cuda", generator=g).exp2()).bfloat16()
    return p


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for x, y in zip(a.args(), b.args()))


# (Hq, Hkv, page, new tokens, prior contexts): whole groups, runs that start inside a
# group and end in the next window, many short sequences (several runs a window); one to
# three waves of CTAs; a part of one head vector (1 + 2 x 1), heads that no part divides
CASES = [
    (16, 8, 16, [1600, 37, 700], [0, 5, 16]),
    (32, 4, 256, [1100, 1200], [3, 255]),
    (14, 2, 48, [9] * 240, [7] * 240),
    (4, 4, 16, [1, 2, 16, 17, 31, 33] * 21, [0, 15, 8, 1, 30, 2] * 21),
    (1, 1, 16, [2048], [9]),
    (3, 3, 32, [5000], [0]),
    (9, 3, 16, [5] * 1100, [0, 13, 14, 27, 6] * 220),
]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"Hq{c[0]}-Hkv{c[1]}-B{len(c[3])}-bs{c[2]}")
def test_many_tokens(lib, fmt, case):
    Hq, Hkv, bs, new, priors = case
    p = _problem(Hq, Hkv, bs, new, priors, 70)
    assert p.T >= MANY_TOKENS
    n = int(p.seq_lens_host.max())
    table = _table(lib, p, n)
    results = []
    for positions in (n, n // 2, 0):         # all angles from the table, some, none
        c = Q8(p, fmt, 7, unused=None)
        before = _before(c)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full_like(p.q, float("nan"))
        _run(lib, p, c, q_out=q_out, table=table, n=positions, flags=flags)
        torch.cuda.synchronize()
        assert flags.item() == 0
        results.append((c, q_out))
    _check(p, results[0][0], before, results[0][1], what=f"{fmt} {case[:3]}")
    for c, q_out in results[1:]:             # the same bits
        assert torch.equal(q_out, results[0][1]) and _same(c, results[0][0])


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("tokens", [MANY_TOKENS - 1, MANY_TOKENS, MANY_TOKENS + 1])
def test_around_the_threshold(lib, fmt, tokens):
    p = _problem(8, 2, 16, [tokens], [7], 71)
    c = Q8(p, fmt, 8, unused=None)
    before = _before(c)
    q_out = torch.empty_like(p.q)
    _run(lib, p, c, q_out=q_out)
    torch.cuda.synchronize()
    _check(p, c, before, q_out, what=f"{tokens}")


def _pieces(lib, p, c, q_out, step):
    for a in range(0, p.T, step):
        s = slice(a, a + step)
        lib.norm_rope_append_q8(p.q[s], p.k[s], p.v[s], p.positions[s], p.slot_mapping[s],
                                p.gamma_q, p.gamma_k, p.theta, p.eps, *c.args(), q_out=q_out[s])


@pytest.mark.parametrize("fmt", CLASSES)
def test_one_call_and_several_small_ones(lib, fmt):
    """Cut between groups: the same q, V and scales bit for bit; K's codes too but where
    a value lies within 2^-20 of the middle between two (a subnormal e4m3 code's within
    2^-20 of the group's largest code)."""
    p = _problem(4, 2, 16, [2304], [0], 72)
    one, several = (Q8(p, fmt, 9, unused=None) for _ in range(2))
    q1, q2 = torch.empty_like(p.q), torch.empty_like(p.q)
    _run(lib, p, one, q_out=q1)
    _pieces(lib, p, several, q2, 768)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2)
    assert torch.equal(one.v.view(torch.uint8), several.v.view(torch.uint8))
    assert torch.equal(one.vs, several.vs) and torch.equal(one.ks, several.ks)
    x, y = (oracle.q8_values(code_bytes(c.k), fmt) for c in (one, several))
    at = np.argwhere(x != y)
    if at.size:
        k = np.zeros(x.shape)
        slots = p.slot_mapping.cpu().numpy()
        k[slots // 16, slots % 16] = _exact(p)[1]
        s = one.ks.double().cpu().numpy()
        for b, o, h, d in at:
            z, mid = k[b, o, h, d] / s[b, 0, h], (x[b, o, h, d] + y[b, o, h, d]) / 2
            assert abs(z - mid) <= max(abs(z), 448 * 2.0 ** -10 if fmt == "e4m3" else 0) * 2.0 ** -20


@pytest.mark.parametrize("fmt", CLASSES)
def test_padding_bad_slots_and_non_finite_values(lib, fmt):
    p = _problem(8, 2, 16, [20] * 110, [20] * 110, 73, extra=0)
    c = Q8(p, fmt, 8, unused=None)
    c.vs[:, :, 0] = float("nan")             # scales that no append wrote
    c.ks[3] = 0.0
    slots = p.slot_mapping.clone()
    slots[0:20] = -1                         # a padded sequence, a window and more
    slots[1000:1060] = -5                    # three, windows of padding alone
    slots[-1] = p.num_blocks * 16 + 3        # too large
    p.v[100, 0, 3] = float("inf")
    p.v[101, 1, 0] = float("nan")
    p.v[500] = 3e38                          # beyond the largest scale
    p.v[501] = 2.0 ** -120
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(p.q)
    _run(lib, p, c, slots=slots, q_out=q_out, table=_table(lib, p, 40), n=40, flags=flags)
    torch.cuda.synchronize()
    assert p.T >= MANY_TOKENS
    assert flags.item() == lib.FLAG_BAD_SLOT | lib.FLAG_BAD_VALUE
    q, k, v = _exact(p)
    s = slots.cpu().numpy()
    check_appended(k, s, *before["k"], code_bytes(c.k), c.ks.cpu().numpy(), fmt, "k")
    check_appended(np.nan_to_num(v, nan=0.0, posinf=np.inf), s, *before["v"], code_bytes(c.v),
                   c.vs.cpu().numpy(), fmt, "v")
    assert bf16_ulp_distance(bits(q_out), oracle.f64_to_bf16_bits(q)).max() <= 1


@pytest.mark.parametrize("fmt", CLASSES)
def test_slots_given_twice_leave_other_groups_right(lib, fmt):
    p = _problem(8, 2, 32, [2200], [0], 74)
    slots = p.slot_mapping.clone()
    own = slots[600:640].clone()
    slots[600:640] = own[0]                  # one slot forty times, over three windows
    gone = torch.unique(own // 16)
    c = Q8(p, fmt, 4, unused=None)
    before = _before(c)
    _run(lib, p, c, slots=slots, q_out=torch.empty_like(p.q))
    torch.cuda.synchronize()
    # every other group holds what a call without those tokens writes
    want = slots.cpu().numpy().copy()
    want[np.isin(want // 16, gone.cpu().numpy())] = -1
    _, k, v = _exact(p)
    for exact, codes, scales, (c0, s0) in ((k, c.k, c.ks, before["k"]), (v, c.v, c.vs, before["v"])):
        c1, s1 = code_bytes(codes).copy(), scales.cpu().numpy().copy()
        g = gone.cpu().numpy()
        for dst, src in ((c1.reshape(-1, 16, 2, 128), c0.reshape(-1, 16, 2, 128)),
                         (s1.reshape(-1, 2), s0.reshape(-1, 2))):
            dst[g] = src[g]
        check_appended(exact, want, c0, s0, c1, s1, fmt)


def test_strided_tensors_and_interleaved_caches_captured_and_replayed(lib):
    """q, k, v as slices of one projection, K and V interleaved with the heads outside the
    slots, scales with their own strides, on a side stream from a graph."""
    p = _problem(8, 2, 32, [2100, 33], [50, 1], 75)
    g = torch.Generator(device="cuda").manual_seed(76)
    fused = torch.randn(p.T, 12, 128, device="cuda", generator=g).bfloat16()
    p.q, p.k, p.v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    c = Q8(p, "int8", 5, unused=None)
    nb, bs, H, D = c.k.shape
    both = torch.zeros(nb, 2, H, bs, D, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, H, nb, bs // 16, device="cuda")
    kv = []
    for i, (x, s) in enumerate(((c.k, c.ks), (c.v, c.vs))):
        view, sview = both[:, i].transpose(1, 2), scales[i].permute(1, 2, 0)
        view.copy_(x)
        sview.copy_(s)
        kv.append((view, sview))
    (c.k, c.ks), (c.v, c.vs) = kv
    start = both.clone(), scales.clone()
    before = _before(c)
    q_out = torch.empty(p.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    _run(lib, p, c, q_out=q_out)
    torch.cuda.synchronize()
    _check(p, c, before, q_out)
    want = both.clone(), scales.clone(), q_out.clone()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        _run(lib, p, c, q_out=q_out)
    for _ in range(2):
        both.copy_(start[0])
        scales.copy_(start[1])
        q_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(both, want[0]) and torch.equal(scales, want[1])
        assert torch.equal(q_out, want[2])
