"""GPU parity of pkvqk_paged_prefill_q8 / _varlen_q8 (and of the decode entry point
above 16 rows per kv head, which runs there) against the fp64 oracle on the
cache's values; tolerances in tests/_q8.py."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import bits, compact_cache
from tests._q8 import CLASSES, Q8, check_attention

pytestmark = pytest.mark.gpu


def _prefill(lib, p, c, num_splits=1, hint=None, scale=0.0, flags=None, q=None):
    q = p.q if q is None else q
    out = torch.full((p.B, p.q_len, p.Hq, p.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.B, p.q_len, p.Hq), float("nan"), device="cuda")
    n = lib.prefill_workspace_bytes(p.B, p.q_len, p.Hq, p.D, num_splits)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    lib.paged_prefill_q8(q, *c.args(), p.block_tables, p.seq_lens, out, q_len=p.q_len,
                         num_splits=num_splits,
                         max_seq_len_hint=p.max_seq_len if hint is None else hint, scale=scale,
                         lse_out=lse, workspace=ws, status_flags=flags)
    torch.cuda.synchronize()
    return out, lse


def _problem(Hq, Hkv, q_len, bs, priors, seed, extra=3):
    lens = [c + q_len for c in priors]
    nb = sum(-(-n // bs) for n in lens) + extra
    return workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, q_len, nb, seed, "cuda")


# (Hq, Hkv, new tokens, page, priors): one row to several CTAs a kv head, with and
# without a second row tile, ragged ones, groups that are no power of two (rows find
# their token by a division), pages that are no power of two, one key to many tiles
CASES = [
    (16, 8, 1, 16, [0, 126, 127, 128, 700]),
    (32, 4, 40, 32, [250, 1]),
    (16, 16, 130, 64, [0, 700]),
    (16, 8, 150, 256, [300, 5]),
    (16, 8, 50, 48, [61, 190]),
    (12, 4, 90, 16, [100, 0]),
    (14, 2, 70, 96, [333, 0]),
    (8, 1, 40, 16, [1500, 3]),
    (16, 8, 300, 192, [90]),
]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"Hq{c[0]}-Hkv{c[1]}-T{c[2]}-bs{c[3]}")
def test_prefill_matches_oracle(lib, fmt, case):
    Hq, Hkv, q_len, bs, priors = case
    p = _problem(Hq, Hkv, q_len, bs, priors, 60 + q_len)
    c = Q8(p, fmt, 13 + bs)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _prefill(lib, p, c, flags=flags)
    assert flags.item() == 0
    check_attention(p, c, out, lse, f"{fmt} {case}")


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("S", [2, 5])
def test_prefill_splits_match_oracle(lib, fmt, S):
    p = _problem(16, 8, 96, 16, [1500, 40, 0], 31 + S)
    c = Q8(p, fmt, 14)
    out, lse = _prefill(lib, p, c, S)
    check_attention(p, c, out, lse, f"{fmt} S={S}")
    out, lse = _prefill(lib, p, c, S, hint=200)      # the last split takes the rest
    check_attention(p, c, out, lse, f"{fmt} S={S} short hint")


@pytest.mark.parametrize("fmt", CLASSES)
def test_prefill_scales_far_apart(lib, fmt):
    p = _problem(16, 8, 80, 16, [300, 0], 5)
    c = Q8(p, fmt, 6)
    g = np.random.default_rng(9)
    shape = tuple(c.vs.shape)
    c.vs.copy_(torch.from_numpy(2.0 ** g.integers(-60, 1, shape)).float())
    c.ks.copy_(torch.from_numpy(2.0 ** g.integers(-40, -5, shape)).float())
    out, lse = _prefill(lib, p, c)
    check_attention(p, c, out, lse, fmt)


def test_prefill_peaked_scores_raise_the_reference(lib):
    """Keys that grow along the sequence: the running reference rises in many tiles
    and in both halves, P and O are rescaled."""
    p = _problem(16, 8, 64, 16, [900, 200], 7)
    c = Q8(p, "int8", 8)
    nb, ng, H = c.ks.shape
    pos = np.zeros((nb, ng))
    for b in range(p.B):
        for n in range(0, int(p.seq_lens_host[b]), 16):
            pos[p.block_tables_host[b, n // 16], 0] = n // 16
    c.ks.mul_(torch.from_numpy(2.0 ** np.minimum(pos // 8, 6)).float().cuda()[..., None])
    c.poison_unused()
    out, lse = _prefill(lib, p, c, scale=0.5)
    check_attention(p, c, out, lse, scale=0.5)


def test_prefill_rows_without_keys(lib):
    p = _problem(16, 8, 20, 16, [40, 20, 30], 3)
    lens = torch.tensor([0, 5, 50], dtype=torch.int32)
    p.seq_lens, p.seq_lens_host = lens.cuda(), lens.numpy().astype(np.int64)
    c = Q8(p, "e4m3", 4)
    out, lse = _prefill(lib, p, c)
    check_attention(p, c, out, lse)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    assert torch.all(out[1, :15] == 0) and torch.all(torch.isneginf(lse[1, :15]))


def test_prefill_q_rows_of_any_magnitude(lib):
    p = _problem(12, 4, 50, 16, [60, 200], 9)        # a group that is no power of two
    for p in (p, _problem(16, 8, 50, 16, [60, 200], 9)):   # and one that is
        q = p.q.clone()
        q[3] = 0
        q[4] *= 2.0 ** -100
        q[60, 2] *= 2.0 ** torch.linspace(-30, 0, 128, device="cuda").round().bfloat16()
        c = Q8(p, "e4m3", 10)
        out, lse = _prefill(lib, p, c, q=q)
        check_attention(p, c, out, lse, q=q)


def test_prefill_bad_block_ids_read_as_zeros_and_are_reported(lib):
    p = _problem(16, 8, 30, 16, [400, 400], 11)
    c = Q8(p, "e4m3", 12, unused=None)
    ref = Q8(p, "e4m3", 12, unused=None)
    bad = p.block_tables_host.copy()
    for b, page, to in ((0, 2, p.num_blocks), (1, 17, -3), (0, 20, 1 << 30)):
        ref.k.view(torch.uint8)[int(bad[b, page])] = 0
        ref.v.view(torch.uint8)[int(bad[b, page])] = 0
        bad[b, page] = to
    p.block_tables = torch.from_numpy(bad).cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _prefill(lib, p, c, flags=flags)
    assert flags.item() == lib.FLAG_BAD_BLOCK_ID
    check_attention(p, ref, out, lse)


def test_prefill_strided_and_interleaved_caches(lib):
    p = _problem(8, 4, 40, 32, [100, 40], 13)
    c = Q8(p, "int8", 14)
    want, want_lse = _prefill(lib, p, c)
    nb, bs, H, D = c.k.shape
    both = torch.zeros(nb, 2, H, bs, D, dtype=torch.int8, device="cuda")
    for i, x in enumerate((c.k, c.v)):
        both[:, i].transpose(1, 2).copy_(x)
    c.k, c.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    scales = torch.zeros(2, H, nb, bs // 16, device="cuda")
    for i, s in enumerate((c.ks, c.vs)):
        scales[i].permute(1, 2, 0).copy_(s)
    c.ks, c.vs = scales[0].permute(1, 2, 0), scales[1].permute(1, 2, 0)
    fused = torch.randn(80, 16, 128, device="cuda").bfloat16()
    fused[:, 4:12] = p.q
    out, lse = _prefill(lib, p, c, q=fused[:, 4:12])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("S", [1, 3, 0])
def test_decode_above_16_rows_per_kv_head(lib, S):
    """Verify of 5 tokens at GQA-8: 40 rows per kv head."""
    p = _problem(32, 4, 5, 16, [9, 300, 700], 23)
    c = Q8(p, "e4m3", 24)
    out = torch.empty(p.B, 5, 32, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(p.B, 5, 32, device="cuda")
    n = lib.decode_workspace_bytes(p.B, 5, 32, 128, S)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    lib.paged_decode_q8(p.q, *c.args(), p.block_tables, p.seq_lens, out, q_len=5, num_splits=S,
                        max_seq_len_hint=p.max_seq_len, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    check_attention(p, c, out, lse, f"S={S}")


def _check_varlen(p, c, out, lse, what=""):
    kv, vv = c.values("k"), c.values("v")
    cu = np.concatenate([[0], np.cumsum(p.q_lens_host)])
    qb = bits(p.q)
    for b in range(p.B):
        n = int(p.q_lens_host[b])
        if n == 0:
            continue
        kb, vb, table, lens = compact_cache(p, [b], kv, vv)
        rows = slice(int(cu[b]), int(cu[b + 1]))
        q = qb[rows][None]
        ref, ref_lse = oracle.paged_attention(q, kb, vb, table, lens, p.block_size, q_len=n)
        mag, _ = oracle.paged_attention(q, kb, vb & 0x7FFF, table, lens, p.block_size, q_len=n)
        got = out[rows].double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -11 + 2.0 ** -14) * mag[0]
        assert (np.abs(got - ref[0]) <= tol).all(), f"{what} sequence {b}"
        assert np.abs(lse[rows].double().cpu().numpy() - ref_lse[0]).max() <= 2.0 ** -11


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("S", [1, 3])
def test_varlen_matches_oracle_and_leaves_rows_past_the_end(lib, fmt, S):
    """A sequence without new tokens among the others; rows of out past total_q keep
    what they held."""
    lens, new = [40, 77, 300, 9, 130], [40, 0, 33, 9, 130]
    p = workloads.make_problem("q8", 16, 8, 128, 16, lens, new, 60, 25, "cuda")
    c = Q8(p, fmt, 26)
    total = p.T
    out = torch.full((total + 8, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total + 8, 16), 7.0, device="cuda")
    n = lib.prefill_workspace_bytes(1, total, 16, 128, S)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    lib.paged_prefill_varlen_q8(p.q, p.cu_seqlens, p.q_len, *c.args(), p.block_tables, p.seq_lens,
                                out[:total], num_splits=S, max_seq_len_hint=p.max_seq_len,
                                lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(out[total:] == 7) and torch.all(lse[total:] == 7)
    _check_varlen(p, c, out, lse, f"{fmt} S={S}")


def test_serving_chain_prefill_then_decode_steps_captured(lib):
    """A prompt appended and prefilled in two chunks (the second one starts inside a
    group), then three decode steps, eager and from one captured graph a step: the
    same bits; the last step against the oracle over the final cache."""
    Hq, Hkv, bs = 16, 8, 16
    chunks = [37, 90, 1, 1, 1]
    total = sum(chunks)
    nb = -(-total // bs) + 1

    def run(graphs):
        g = torch.Generator(device="cuda").manual_seed(31)
        k = torch.empty(nb, bs, Hkv, 128, dtype=torch.float8_e4m3fn, device="cuda")
        k.view(torch.uint8).fill_(0x7F)              # never written: NaN codes
        v = k.clone()
        ks = torch.full((nb, 1, Hkv), float("nan"), device="cuda")
        vs = ks.clone()
        table = torch.arange(nb, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
        gam = torch.ones(128, device="cuda", dtype=torch.bfloat16)
        outs, at = [], 0
        for n in chunks:
            q, kk, vv = (torch.randn(n, h, 128, device="cuda", generator=g).bfloat16()
                         for h in (Hq, Hkv, Hkv))
            pos = torch.arange(at, at + n, device="cuda")
            slots = table[0, pos // bs].long() * bs + pos % bs
            at += n
            lens = torch.tensor([at], dtype=torch.int32, device="cuda")
            qh = torch.empty_like(q)
            out = torch.empty(1, n, Hq, 128, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(1, n, Hq, device="cuda")

            def step():
                lib.norm_rope_append_q8(q, kk, vv, pos, slots, gam, gam, 1e6, 1e-6, k, v, ks, vs,
                                        q_out=qh)
                if n > 1:
                    lib.paged_prefill_q8(qh, k, v, ks, vs, table, lens, out, q_len=n,
                                         max_seq_len_hint=at, lse_out=lse)
                else:
                    lib.paged_decode_q8(qh, k, v, ks, vs, table, lens, out, max_seq_len_hint=at,
                                        lse_out=lse)

            if graphs:
                s, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s), torch.cuda.graph(gr, stream=s):
                    step()
                gr.replay()
            else:
                step()
            torch.cuda.synchronize()
            outs.append((qh, out, lse))
        return outs, (k, v, ks, vs), table

    eager, cache, table = run(False)
    graph, cache2, _ = run(True)
    for a, b in zip(eager, graph):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for x, y in zip(cache, cache2):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    p = workloads.make_problem("q8", Hq, Hkv, 128, bs, [total], 1, nb, 1, "cuda")
    p.block_tables_host, p.block_tables = table.cpu().numpy(), table
    c = Q8(p, "e4m3", 1, unused=None)
    c.k, c.v, c.ks, c.vs = cache
    qh, out, lse = eager[-1]
    check_attention(p, c, out, lse, "last step", q=qh)


def test_prefill_benchmark_shape_sampled_rows(lib):
    """4 x 2048 fresh tokens at the benchmark's launch; some rows of each sequence."""
    p = workloads.chunked_prefill(device="cuda", batch=2, chunk=2048, lo=0, hi=0)
    c = Q8(p, "e4m3", 33, unused=None)
    out, lse = _prefill(lib, p, c)
    kv, vv = c.values("k"), c.values("v")
    q = bits(p.q).reshape(2, 2048, 16, 128)
    for b in range(2):
        for t in (0, 1, 127, 128, 1000, 2047):
            kb, vb, table, _ = compact_cache(p, [b], kv, vv)
            args = (table, np.array([t + 1]), p.block_size)
            ref, ref_lse = oracle.paged_attention(q[b:b + 1, t:t + 1], kb, vb, *args)
            mag, _ = oracle.paged_attention(q[b:b + 1, t:t + 1], kb, vb & 0x7FFF, *args)
            got = out[b, t].double().cpu().numpy()
            tol = 2.0 ** -8 * np.abs(ref[0, 0]) + (2.0 ** -11 + 2.0 ** -14) * mag[0, 0]
            assert (np.abs(got - ref[0, 0]) <= tol).all(), (b, t)
            assert np.abs(lse[b, t].double().cpu().numpy() - ref_lse[0, 0]).max() <= 2.0 ** -11


@pytest.mark.parametrize("fmt", CLASSES)
def test_prefill_tiny_rows_over_groups_of_the_smallest_scale(lib, fmt):
    """Score factors that underflow (2^-110 rows, 2^-64 scales): masked keys stay
    masked, the others weigh the same."""
    p = _problem(16, 8, 40, 16, [130, 0], 21)
    c = Q8(p, fmt, 22)
    used = ~torch.isnan(c.ks)
    c.ks[used] = 2.0 ** -64
    q = p.q.clone()
    q[5:20] *= 2.0 ** -110
    out, lse = _prefill(lib, p, c, q=q)
    check_attention(p, c, out, lse, fmt, q=q)
