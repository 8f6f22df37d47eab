"""The scored attention calls, the append with axes and the verdict on drafts where sizes and
circumstances are unusual: caches and probabilities whose offsets pass 32 bits, the longest
chunk, pages that sequences share, calls at the same time, and captured prefills.
"""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import ULP_TOL, assert_attention_close, bf16_ulp_distance, bits

pytestmark = pytest.mark.gpu


def _slopes(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)


def test_offsets_past_32_bits_in_the_cache(lib):
    """A cache of 2.6 G elements a tensor whose last pages are used."""
    nb, bs, hkv, hq = 160000, 16, 8, 16
    lens = [45, 300]
    p = workloads.make_problem("far", hq, hkv, 128, bs, lens, 3, 24, 41, "cuda")
    kc, vc = (torch.empty(nb, bs, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    shift = nb - 24
    kc[shift:], vc[shift:] = p.k_cache, p.v_cache
    table = torch.where(p.block_tables >= 0, p.block_tables + shift, p.block_tables)
    slots = p.slot_mapping + shift * bs
    assert slots.min() * hkv * 128 > 2 ** 31
    axes = lib.rope_axes((16, 24, 24))
    pos = p.positions[None].expand(3, -1)
    q = torch.empty_like(p.q)
    lib.norm_rope_append_axes(p.q, p.k, p.v, pos, axes, slots, p.gamma_q, p.gamma_k, p.theta,
                              p.eps, kc, vc, q_out=q)
    torch.cuda.synchronize()
    qh, kco, vco = oracle.norm_rope_append_axes(
        bits(p.q), bits(p.k), bits(p.v), pos.cpu().numpy(), axes, p.slot_mapping.cpu().numpy(),
        bits(p.gamma_q), bits(p.gamma_k), p.theta, p.eps, bits(p.k_cache), bits(p.v_cache), bs)
    assert bf16_ulp_distance(bits(q), qh).max() <= ULP_TOL
    assert bf16_ulp_distance(bits(kc[shift:]), kco).max() <= ULP_TOL
    assert np.array_equal(bits(vc[shift:]), vco)
    rules = dict(softcap=8.0, window=200)
    ref, ref_lse = oracle.scored_attention(bits(q), bits(kc[shift:]), bits(vc[shift:]),
                                           p.block_tables_host, lens, bs, [3, 3], **rules)
    for f in (lib.paged_decode_scored, lib.paged_prefill_scored):
        out = torch.empty(6, hq, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(6, hq, device="cuda")
        f(q, kc, vc, table, p.seq_lens, out, q_len=3, lse_out=lse, **rules)
        torch.cuda.synchronize()
        assert_attention_close(bits(out), ref, lse.cpu().numpy(), ref_lse)


def test_offsets_past_32_bits_in_the_probabilities(lib):
    B, K, V = 140, 15, (1 << 20) - 1
    p = torch.zeros(B, K + 1, V, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, K, V, dtype=torch.bfloat16, device="cuda")
    assert p.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.softmax(3 * torch.randn(K + 1, V, device="cuda", generator=g), -1)
    p[-1] = rows.bfloat16()
    q[-1] = torch.softmax(rows[:K].log() + 0.5 * torch.randn(K, V, device="cuda", generator=g),
                          -1).bfloat16()
    drafts = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    drafts[-1] = torch.multinomial(q[-1, :, ::16].float(), 1, generator=g)[:, 0].int() * 16
    u = torch.rand(B, K + 1, device="cuda", generator=g)
    for first in (0.0, 1.0):                   # down to the last row, and at the first
        u[-1, :K] = first
        tokens = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
        n = torch.empty(B, dtype=torch.int32, device="cuda")
        lib.verify_drafts(p, q, drafts, u, tokens, n)
        torch.cuda.synchronize()
        want, want_n = oracle.verify_drafts(p[-1:].double().cpu().numpy(),
                                            q[-1:].double().cpu().numpy(),
                                            drafts[-1:].cpu().numpy(), u[-1:].cpu().numpy())
        assert np.array_equal(tokens[-1:].cpu().numpy(), want)
        assert n[-1].item() == want_n[0]
        assert (tokens[:-1, 0] == -1).all() and (n[:-1] == 0).all()


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (4, 1)])
def test_longest_chunk(lib, Hq, Hkv):
    """16384 tokens at once, with rules that hide nothing, beside the plain call."""
    T = 16384
    p = workloads.make_problem("long", Hq, Hkv, 128, 64, [T], T, T // 64, 42, "cuda")
    got = []
    for f, more in ((lib.paged_prefill, {}),
                    (lib.paged_prefill_scored, dict(window=T, softcap=2.0 ** 20)),
                    (lib.paged_prefill_scored, dict(first_keys=torch.zeros(
                        T, dtype=torch.int32, device="cuda")))):
        out = torch.empty(T, Hq, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, Hq, device="cuda")
        f(p.q, p.k_cache, p.v_cache, p.block_tables, p.seq_lens, out, q_len=T, lse_out=lse, **more)
        torch.cuda.synchronize()
        got.append((out, lse))
    for out, lse in got[1:]:
        # P rounded to bf16 on both sides: as far apart as twice either is off
        assert (out.float() - got[0][0].float()).abs().max() <= 4e-2
        assert (lse - got[0][1]).abs().max() <= 2e-3


def test_pages_shared_by_sequences(lib):
    """One prompt's pages in every sequence's table, and a page twice in one."""
    p = workloads.make_problem("shared", 16, 8, 128, 16, [200, 200, 200], 1, 45, 43, "cuda")
    table = p.block_tables.clone()
    table[1:, :10] = table[0, :10]
    table[2, 4] = table[2, 3]
    host = table.cpu().numpy()
    rules = dict(softcap=6.0, slopes=_slopes(16))
    ref, ref_lse = oracle.scored_attention(bits(p.q), bits(p.k_cache), bits(p.v_cache), host,
                                           [200] * 3, 16, [1] * 3, softcap=6.0,
                                           slopes=_slopes(16).cpu().numpy())
    out = torch.empty(3, 16, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 16, device="cuda")
    lib.paged_decode_scored(p.q, p.k_cache, p.v_cache, table, p.seq_lens, out, lse_out=lse, **rules)
    torch.cuda.synchronize()
    assert_attention_close(bits(out), ref, lse.cpu().numpy(), ref_lse)


def _prefill_calls(lib, n):
    """n independent prefills of several places a SM, as functions of a stream."""
    calls = []
    for i in range(n):
        lens = [500 + 37 * i, 130, 801, 64 + i, 700, 333]
        p = workloads.make_problem("many", 16, 8, 128, 16, lens, lens, 170, 44 + i, "cuda")
        S = 1 + i % 2
        rules = (dict(softcap=5.0), dict(window=90, slopes=_slopes(16)), dict(window=33))[i % 3]
        out = torch.zeros(p.T, 16, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(p.T, 16, device="cuda")
        ws = torch.empty(max(256, lib.prefill_workspace_bytes(1, p.T, 16, 128, S)),
                         dtype=torch.uint8, device="cuda")

        def call(stream, p=p, S=S, rules=rules, out=out, lse=lse, ws=ws):
            lib.paged_prefill_varlen_scored(p.q, p.cu_seqlens, int(p.q_lens_host.max()), p.k_cache,
                                            p.v_cache, p.block_tables, p.seq_lens, out,
                                            num_splits=S, lse_out=lse, workspace=ws,
                                            stream=stream, **rules)

        calls.append((call, out, lse))
    return calls


def test_prefills_at_the_same_time(lib):
    """On streams of their own, over one another: the bits of one after the other."""
    calls = _prefill_calls(lib, 4)
    want = []
    for call, out, lse in calls:
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for _, out, lse in calls:
            out.zero_()
            lse.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for (call, _, _), s in zip(calls, streams):
                call(s)
        torch.cuda.synchronize()
        for (_, out, lse), (o, l) in zip(calls, want):
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_captured_prefills(lib):
    """Two calls, one behind the other, in a graph that is replayed."""
    calls = _prefill_calls(lib, 2)
    want = []
    for call, out, lse in calls:
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        for call, _, _ in calls:
            call(s)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for _, out, lse in calls:
            out.zero_()
            lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        for (_, out, lse), (o, l) in zip(calls, want):
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_verdicts_at_the_same_time(lib):
    """Calls of different sizes on streams of their own."""
    g = torch.Generator(device="cuda").manual_seed(3)
    calls = []
    for B, K, V in ((1, 4, 32768), (9, 2, 100003), (64, 3, 5000), (2, 7, 131072)):
        p = torch.softmax(torch.randn(B, K + 1, V, device="cuda", generator=g) * 3, -1)
        q = torch.softmax(p[:, :K].log() + torch.randn(B, K, V, device="cuda", generator=g), -1)
        d = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).int()
        u = torch.rand(B, K + 1, device="cuda", generator=g)
        calls.append([(p, q, d, u), torch.empty(B, K + 1, dtype=torch.int32, device="cuda"),
                      torch.empty(B, dtype=torch.int32, device="cuda"), torch.cuda.Stream()])
    want = []
    for args, tokens, n, _ in calls:
        lib.verify_drafts(*args, tokens, n)
        torch.cuda.synchronize()
        want.append((tokens.clone(), n.clone()))
    for _ in range(5):
        for args, tokens, n, s in calls:
            lib.verify_drafts(*args, tokens, n, stream=s)
        torch.cuda.synchronize()
        for (_, tokens, n, _), (t, m) in zip(calls, want):
            assert torch.equal(tokens, t) and torch.equal(n, m)
            tokens.zero_()
        torch.cuda.synchronize()
