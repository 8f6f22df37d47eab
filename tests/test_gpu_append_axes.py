"""GPU parity of pkvqk_norm_rope_append_axes against the fp64 oracle: q_hat / k_hat within
1 bf16 ulp, v rows and every cache slot that no token maps to bit-exact, and text tokens
(one position on every axis) the bits of pkvqk_norm_rope_append.
"""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import ULP_TOL, bf16_ulp_distance, bits

pytestmark = pytest.mark.gpu


def _problem(Hq, Hkv, bs, lens, q_len, seed):
    pages = sum(-(-n // bs) for n in lens)
    return workloads.make_problem("axes", Hq, Hkv, 128, bs, lens, q_len, pages + 3, seed, "cuda")


def _positions(rng, axes, T, top):
    return torch.from_numpy(rng.integers(0, top, size=(axes, T))).cuda()


def _table(lib, positions, theta):
    t = torch.empty(lib.rope_table_bytes(positions), dtype=torch.uint8, device="cuda")
    lib.rope_table_build(t, positions, theta)
    return t


def _check(lib, p, pos, axes, table_positions=0, slots=None, in_place=False):
    slots = p.slot_mapping if slots is None else slots
    q, kc, vc = p.q.clone(), p.k_cache.clone(), p.v_cache.clone()
    q_out = q if in_place else torch.full_like(q, float("nan"))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = _table(lib, table_positions, p.theta) if table_positions else None
    lib.norm_rope_append_axes(q, p.k, p.v, pos, axes, slots, p.gamma_q, p.gamma_k, p.theta, p.eps,
                              kc, vc, q_out=None if in_place else q_out, rope_table=table,
                              table_positions=table_positions, status_flags=flags)
    torch.cuda.synchronize()
    qh, kco, vco = oracle.norm_rope_append_axes(
        bits(p.q), bits(p.k), bits(p.v), pos.cpu().numpy(), axes, slots.cpu().numpy(),
        bits(p.gamma_q), bits(p.gamma_k), p.theta, p.eps, bits(p.k_cache), bits(p.v_cache),
        p.block_size)
    assert bf16_ulp_distance(bits(q_out), qh).max() <= ULP_TOL
    assert bf16_ulp_distance(bits(kc), kco).max() <= ULP_TOL
    assert np.array_equal(bits(vc), vco)
    untouched = ~np.any(vco != bits(p.v_cache), axis=(2, 3))
    assert np.array_equal(bits(kc)[untouched], bits(p.k_cache)[untouched])
    if not in_place:
        assert torch.equal(q, p.q)
    return flags.item(), q_out, kc


SECTIONS = [((16, 24, 24), False), ((24, 20, 20), True), ((64,), False), ((1, 62, 1), False),
            ((21, 21, 22), True), ((30, 34), False), ((10, 20, 30, 4), True), ((0, 64), False)]


@pytest.mark.parametrize("table", [0, 300, 5000], ids=["computed", "some-in-table", "table"])
@pytest.mark.parametrize("sections,interleaved", SECTIONS)
def test_sections(lib, sections, interleaved, table):
    p = _problem(16, 8, 16, [17, 1, 40], 1, 31)
    pos = _positions(np.random.default_rng(sum(sections) + table), len(sections), p.T, 5000)
    if table == 300:
        pos[:, ::2] %= 300                     # every other token lies in the table whole
    _check(lib, p, pos, lib.rope_axes(sections, interleaved=interleaved), table)


@pytest.mark.parametrize("Hq,Hkv,bs", [(32, 4, 256), (8, 1, 32), (14, 2, 96), (12, 4, 64),
                                        (40, 8, 16)])
def test_heads(lib, Hq, Hkv, bs):
    p = _problem(Hq, Hkv, bs, [19, 300], 7, 32)
    pos = _positions(np.random.default_rng(Hq), 3, p.T, 40000)
    _check(lib, p, pos, lib.rope_axes((16, 24, 24)))
    _check(lib, p, pos, lib.rope_axes((24, 20, 20), interleaved=True), 40000)


@pytest.mark.parametrize("T", [1023, 1024, 1500])
@pytest.mark.parametrize("table", [0, 2000])
def test_many_tokens(lib, T, table):
    p = _problem(16, 8, 16, [T], T, 33)
    pos = _positions(np.random.default_rng(T), 3, T, 2000)
    for axes in (lib.rope_axes((16, 24, 24)), lib.rope_axes((24, 20, 20), interleaved=True)):
        _check(lib, p, pos, axes, table)


def test_in_place_and_negative_and_far_positions(lib):
    p = _problem(16, 8, 16, [5, 33], 1, 34)
    pos = torch.tensor([[2000000, -5], [-1, 1 << 20], [0, 77777]], device="cuda")
    _check(lib, p, pos, lib.rope_axes((16, 24, 24)), 1000, in_place=True)


def test_padding_and_bad_slots(lib):
    p = _problem(16, 8, 16, [5, 33, 8], 1, 35)
    slots = p.slot_mapping.clone()
    slots[0], slots[2] = -1, p.num_blocks * 16
    f, _, _ = _check(lib, p, _positions(np.random.default_rng(1), 3, 3, 99),
                     lib.rope_axes((16, 24, 24)), slots=slots)
    assert f == lib.FLAG_BAD_SLOT


@pytest.mark.parametrize("table", [0, 9000])
def test_text_tokens_have_the_plain_bits(lib, table):
    p = _problem(16, 8, 16, [9000, 33, 8], 5, 36)
    pos = p.positions[None].expand(3, -1)
    q, kc, vc = p.q.clone(), p.k_cache.clone(), p.v_cache.clone()
    lib.norm_rope_append(q, p.k, p.v, p.positions, p.slot_mapping, p.gamma_q, p.gamma_k, p.theta,
                         p.eps, kc, vc)
    for axes in (lib.rope_axes((16, 24, 24)), lib.rope_axes((20, 22, 22), interleaved=True)):
        _, q2, kc2 = _check(lib, p, pos, axes, table)   # the axes share one row: stride 0
        assert torch.equal(q2, q) and torch.equal(kc2, kc)


def test_strided_views(lib):
    """q, k, v views of one fused buffer, K and V views of one allocation, and positions
    rows of a wider tensor."""
    p = _problem(16, 8, 16, [5, 33, 100], 1, 37)
    T = p.T
    qkv = torch.cat((p.q, p.k, p.v), 1)
    p.q, p.k, p.v = qkv[:, :16], qkv[:, 16:24], qkv[:, 24:]
    both = torch.stack((p.k_cache, p.v_cache), 1).contiguous()
    wide = torch.zeros(3, T + 9, dtype=torch.int64, device="cuda")
    wide[:, 4:4 + T] = _positions(np.random.default_rng(2), 3, T, 3000)
    kc, vc = both[:, 0], both[:, 1]
    q_out = torch.empty(T, 20, 128, dtype=torch.bfloat16, device="cuda")[:, 2:18]
    axes = lib.rope_axes((16, 24, 24))
    before = both.clone()
    lib.norm_rope_append_axes(p.q, p.k, p.v, wide[:, 4:4 + T], axes, p.slot_mapping, p.gamma_q,
                              p.gamma_k, p.theta, p.eps, kc, vc, q_out=q_out)
    torch.cuda.synchronize()
    qh, kco, vco = oracle.norm_rope_append_axes(
        bits(p.q), bits(p.k), bits(p.v), wide[:, 4:4 + T].cpu().numpy(), axes,
        p.slot_mapping.cpu().numpy(), bits(p.gamma_q), bits(p.gamma_k), p.theta, p.eps,
        bits(before[:, 0]), bits(before[:, 1]), 16)
    assert bf16_ulp_distance(bits(q_out), qh).max() <= ULP_TOL
    assert bf16_ulp_distance(bits(kc), kco).max() <= ULP_TOL
    assert np.array_equal(bits(vc), vco)


def test_on_a_side_stream_and_in_a_graph(lib):
    p = _problem(16, 8, 16, [300, 33, 100], 4, 38)
    pos = _positions(np.random.default_rng(3), 3, p.T, 3000)
    axes = lib.rope_axes((16, 24, 24))
    want, want_q = p.k_cache.clone(), torch.empty_like(p.q)
    v = p.v_cache.clone()
    args = (pos, axes, p.slot_mapping, p.gamma_q, p.gamma_k, p.theta, p.eps)
    lib.norm_rope_append_axes(p.q, p.k, p.v, *args, want, v, q_out=want_q)
    got, got_q = p.k_cache.clone(), torch.empty_like(p.q)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        lib.norm_rope_append_axes(p.q, p.k, p.v, *args, got, v, q_out=got_q)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        got.copy_(p.k_cache)
        got_q.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_q, want_q)
