"""GPU parity of pkvqk_paged_decode_q8 (decode and verify over an 8-bit cache)
against the fp64 oracle on the cache's values; tolerances in tests/_q8.py."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._q8 import CLASSES, Q8, check_attention, code_bytes, from_bytes

pytestmark = pytest.mark.gpu


def _decode(lib, p, c, num_splits=1, hint=None, scale=0.0, flags=None, q=None, **kw):
    q = p.q if q is None else q
    out = torch.full((p.B, p.q_len, p.Hq, p.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.B, p.q_len, p.Hq), float("nan"), device="cuda")
    hint = p.max_seq_len if hint is None else hint
    S = num_splits
    if S < 0:
        S = lib.choose_num_splits(p.B, p.Hkv, p.q_len * p.Hq // p.Hkv, max(hint, 1),
                                  p.total_tokens, p.block_size)
    n = lib.decode_workspace_bytes(p.B, p.q_len, p.Hq, p.D, S)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    lib.paged_decode_q8(q, *c.args(), p.block_tables, p.seq_lens, out, q_len=p.q_len,
                        num_splits=S, max_seq_len_hint=hint, scale=scale, lse_out=lse,
                        workspace=ws, status_flags=flags, **kw)
    torch.cuda.synchronize()
    return out, lse


def _problem(Hq, Hkv, q_len, bs, lens, seed, extra=2):
    nb = max(1, sum(-(-n // bs) for n in lens)) + extra
    return workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, q_len, nb, seed, "cuda")


# (Hq, Hkv, q_len, page, lengths): rows per kv head 1 to 16, 8/4/2/1 heads a CTA,
# pages whose size is not a power of two, tiles cut by the sequence's end
SHAPES = [
    (16, 8, 1, 16, [1, 15, 16, 17, 200, 333]),
    (8, 8, 1, 16, [40, 7]),
    (32, 4, 1, 32, [100, 31, 1]),
    (28, 4, 1, 48, [97, 48]),
    (12, 4, 1, 96, [200, 5]),
    (14, 2, 1, 64, [130, 64]),
    (8, 1, 1, 256, [300, 256, 2]),
    (9, 3, 1, 16, [50, 21]),
    (16, 8, 5, 16, [9, 300, 77, 5]),
    (16, 8, 8, 16, [64, 8]),
    (16, 1, 1, 16, [77, 3]),
    (4, 2, 7, 32, [40, 33]),
    (10, 2, 3, 16, [19, 120]),
]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("shape", SHAPES,
                         ids=lambda s: f"Hq{s[0]}-Hkv{s[1]}-T{s[2]}-bs{s[3]}")
@pytest.mark.parametrize("S", [1, 3, 0])
def test_decode_matches_oracle(lib, fmt, shape, S):
    Hq, Hkv, q_len, bs, lens = shape
    p = _problem(Hq, Hkv, q_len, bs, lens, 50 + q_len + bs)
    c = Q8(p, fmt, 11 + bs)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _decode(lib, p, c, S, flags=flags)
    assert flags.item() == 0
    check_attention(p, c, out, lse, f"{fmt} {shape} S={S}")


@pytest.mark.parametrize("S", [1, 2, 0])
def test_sequences_without_keys_and_shorter_than_their_new_tokens(lib, S):
    """seq_len 0, and seq_len < q_len: rows without a visible key are 0 and -inf."""
    p = _problem(16, 8, 4, 16, [40, 20, 30], 3)
    lens = torch.tensor([0, 2, 30], dtype=torch.int32)
    p.seq_lens, p.seq_lens_host = lens.cuda(), lens.numpy().astype(np.int64)
    c = Q8(p, "e4m3", 4)
    out, lse = _decode(lib, p, c, S)
    check_attention(p, c, out, lse, f"S={S}")
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    assert torch.all(out[1, :2] == 0) and torch.all(torch.isneginf(lse[1, :2]))
    assert torch.all(torch.isfinite(lse[1, 2:]))


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("S", [1, 3])
def test_scales_far_apart(lib, fmt, S):
    """V scales over 2^-60 .. 2^0 and K scales over 2^-40 .. 2^-6: groups whose values
    vanish beside others still count in the softmax."""
    p = _problem(16, 8, 2, 16, [200, 40], 5)
    c = Q8(p, fmt, 6)
    g = np.random.default_rng(9)
    shape = tuple(c.vs.shape)
    c.vs.copy_(torch.from_numpy(2.0 ** g.integers(-60, 1, shape)).float())
    c.ks.copy_(torch.from_numpy(2.0 ** g.integers(-40, -5, shape)).float())
    out, lse = _decode(lib, p, c, S)
    check_attention(p, c, out, lse, f"{fmt} S={S}")


def test_scales_that_are_no_powers_of_two_and_scales_of_zero(lib):
    """The attention takes any scale in range; 0 counts as 2^-64.  Checked against the
    same cache with the scale folded into float64 values."""
    p = _problem(16, 8, 1, 16, [100, 33], 7)
    c = Q8(p, "int8", 8, unused=None)
    c.ks.mul_(1.37)
    c.vs.mul_(0.71)
    c.vs[:, :, 3] = 0
    out, lse = _decode(lib, p, c)
    k, v = ((oracle.q8_values(code_bytes(x), "int8")
             * np.repeat(s.double().cpu().numpy(), 16, axis=1)[..., None])
            for x, s in ((c.k, c.ks), (c.v, c.vs)))
    q = p.q.double().cpu().numpy().reshape(2, 16, 128)
    for b in range(2):
        n = np.arange(int(p.seq_lens_host[b]))
        blk = p.block_tables_host[b, n // 16]
        for h in range(16):
            s = k[blk, n % 16, h // 2] @ q[b, h] * 128 ** -0.5
            w = np.exp(s - s.max())
            ref = (w @ v[blk, n % 16, h // 2]) / w.sum()
            mag = (w @ np.abs(v[blk, n % 16, h // 2])) / w.sum()
            got = out[b, 0, h].double().cpu().numpy()
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 1e-15).all()
            assert abs(lse[b, 0, h].item() - (s.max() + np.log(w.sum()))) <= 2.0 ** -11


def test_q_rows_of_any_magnitude(lib):
    """Rows of 0, of 2^-100 and of 2^60 (with K to match), and elements far apart."""
    p = _problem(16, 8, 1, 16, [60, 17, 90], 9)
    q = p.q.clone()
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -100
    q[1, 2] *= 2.0 ** torch.linspace(-30, 0, 128, device="cuda").round().bfloat16()
    c = Q8(p, "e4m3", 10)
    out, lse = _decode(lib, p, c, q=q)
    check_attention(p, c, out, lse, q=q)
    q2 = (p.q.float() * 2.0 ** 60).bfloat16()
    for s in (c.ks,):
        s.mul_(2.0 ** -50)
    out, lse = _decode(lib, p, c, q=q2, scale=2.0 ** -13)
    check_attention(p, c, out, lse, q=q2, scale=2.0 ** -13)


@pytest.mark.parametrize("S", [2, 0])
def test_bad_block_ids_read_as_zeros_and_are_reported(lib, S):
    p = _problem(16, 8, 1, 16, [64, 64], 11)
    c = Q8(p, "e4m3", 12, unused=None)
    zero_k, zero_v = c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    bad = p.block_tables_host.copy()
    gone = bad[0, 2]
    bad[0, 2] = p.num_blocks + 5
    bad[1, 1] = -3
    for x in (zero_k, zero_v):
        x[int(gone)] = 0
        x[int(p.block_tables_host[1, 1])] = 0
    p.block_tables = torch.from_numpy(bad).cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _decode(lib, p, c, S, flags=flags)
    assert flags.item() == lib.FLAG_BAD_BLOCK_ID
    ref = Q8(p, "e4m3", 12, unused=None)
    ref.k, ref.v = zero_k.view(c.k.dtype), zero_v.view(c.v.dtype)
    check_attention(p, ref, out, lse, f"S={S}")


def test_strided_and_interleaved_caches(lib):
    """K and V in one allocation with the heads outside the slots, scales transposed,
    q as a slice of a fused projection."""
    p = _problem(8, 4, 1, 32, [100, 40, 33], 13)
    c = Q8(p, "int8", 14)
    want, want_lse = _decode(lib, p, c)
    nb, bs, H, D = c.k.shape
    both = torch.zeros(nb, 2, H, bs, D, dtype=torch.int8, device="cuda")
    for i, x in enumerate((c.k, c.v)):
        both[:, i].transpose(1, 2).copy_(x)
    c.k, c.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    scales = torch.zeros(2, H, nb, bs // 16, device="cuda")
    for i, s in enumerate((c.ks, c.vs)):
        scales[i].permute(1, 2, 0).copy_(s)
    c.ks, c.vs = scales[0].permute(1, 2, 0), scales[1].permute(1, 2, 0)
    fused = torch.randn(3, 16, 128, device="cuda").bfloat16()
    fused[:, 4:12] = p.q
    out, lse = _decode(lib, p, c, q=fused[:, 4:12])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("case", ["mixed", "verify", "uniform"])
def test_large_batches_on_the_chosen_schedule(lib, case):
    """The benchmark's shapes at full width, sampled sequences, the schedule that the
    heuristic picks (balanced for the mixed batch)."""
    p = {"mixed": lambda: workloads.decode_gqa8(device="cuda", batch=24, hi=4096),
         "verify": lambda: workloads.verify_causal(device="cuda", batch=12, lo=300, hi=1500),
         "uniform": lambda: workloads.decode_uniform(16, 2048, device="cuda")}[case]()
    c = Q8(p, "e4m3", 21, unused=None)
    out, lse = _decode(lib, p, c, -1)
    seqs = [0, p.B // 2, p.B - 1]
    check_attention(p, c, out, lse, case, seqs=seqs)


@pytest.mark.parametrize("S", [1, 3, 0])
def test_append_then_decode_captured_and_replayed(lib, S):
    """The serving step, append and decode on one side stream, eager and captured:
    the same bits, and the oracle's chain."""
    p = workloads.make_problem("q8", 16, 8, 128, 16, [30, 99, 400], 1, 40, 17, "cuda")
    state = []
    for _ in range(2):
        c = Q8(p, "e4m3", 18, unused=None)
        q = torch.empty_like(p.q)
        out = torch.empty(p.B, 1, p.Hq, p.D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(p.B, 1, p.Hq, device="cuda")
        n = lib.decode_workspace_bytes(p.B, 1, p.Hq, p.D, S)
        state.append((c, q, out, lse, torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")))

    def step(c, q, out, lse, ws):
        lib.norm_rope_append_q8(p.q, p.k, p.v, p.positions, p.slot_mapping, p.gamma_q, p.gamma_k,
                                p.theta, p.eps, *c.args(), q_out=q)
        lib.paged_decode_q8(q, *c.args(), p.block_tables, p.seq_lens, out, num_splits=S,
                            max_seq_len_hint=p.max_seq_len, lse_out=lse, workspace=ws)

    step(*state[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step(*state[1])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for i in (1, 2, 3):
        assert torch.equal(state[0][i], state[1][i])
    c, q, out, lse, _ = state[0]
    check_attention(p, c, out, lse, "chain", q=q)


def test_q8_decode_of_a_bf16_cache_s_values(lib):
    """The bf16 kernel on the same values: both within their own roundings."""
    p = _problem(16, 8, 1, 16, [500, 77], 19)
    c = Q8(p, "int8", 20, unused=None)
    out, lse = _decode(lib, p, c, 2)
    out_b, lse_b = torch.empty_like(out), torch.empty_like(lse)
    lib.paged_decode(p.q, c.values("k").cuda(), c.values("v").cuda(), p.block_tables, p.seq_lens,
                     out_b, num_splits=1, max_seq_len_hint=p.max_seq_len, lse_out=lse_b)
    torch.cuda.synchronize()
    assert (out.float() - out_b.float()).abs().max().item() <= 2e-2
    assert (lse - lse_b).abs().max().item() <= 1e-3


def test_codes_round_trip():
    b = np.arange(256, dtype=np.uint8).reshape(2, 128)
    assert np.array_equal(code_bytes(from_bytes(b, "int8")), b)


@pytest.mark.parametrize("fmt", CLASSES)
def test_decode_tiny_rows_over_groups_of_the_smallest_scale(lib, fmt):
    p = _problem(16, 8, 4, 16, [130, 4], 21)
    c = Q8(p, fmt, 22)
    used = ~torch.isnan(c.ks)
    c.ks[used] = 2.0 ** -64
    q = p.q.clone()
    q[1:6] *= 2.0 ** -110
    out, lse = _decode(lib, p, c, 1, q=q)
    check_attention(p, c, out, lse, fmt, q=q)


def test_two_calls_at_once_on_two_streams(lib):
    """Decode and prefill calls that overlap, each with a workspace of its own."""
    p = _problem(16, 8, 5, 16, [3000, 900, 5, 40], 31)
    c = Q8(p, "int8", 32)
    want = {S: _decode(lib, p, c, S) for S in (0, 3)}
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = {}
    for S, s in zip((0, 3), streams):
        n = lib.decode_workspace_bytes(p.B, p.q_len, p.Hq, p.D, S)
        got[S] = (torch.empty(n, dtype=torch.uint8, device="cuda"),
                  torch.empty_like(want[S][0]), torch.empty_like(want[S][1]))
    torch.cuda.synchronize()
    for _ in range(20):
        for S, s in zip((0, 3), streams):
            ws, out, lse = got[S]
            with torch.cuda.stream(s):
                lib.paged_decode_q8(p.q, *c.args(), p.block_tables, p.seq_lens, out, q_len=p.q_len,
                                    num_splits=S, max_seq_len_hint=p.max_seq_len, lse_out=lse,
                                    workspace=ws)
    torch.cuda.synchronize()
    for S in (0, 3):
        assert torch.equal(got[S][1].view(torch.int16), want[S][0].view(torch.int16))
        assert torch.equal(got[S][2], want[S][1])


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("S", [1, 2, 0])
def test_odd_tiles_at_a_cut_inside_a_sequence(lib, fmt, S):
    """Segments of an odd number of 16-key tiles: what follows the last one belongs to
    the next split, and is counted once."""
    p = _problem(16, 8, 1, 16, [16 * 7, 16 * 3 + 5, 16, 16 * 11 + 1], 33)
    c = Q8(p, fmt, 34)
    out, lse = _decode(lib, p, c, S, hint=16 * 6)    # splits of 3 pages
    check_attention(p, c, out, lse, f"{fmt} S={S}")
    p = _problem(8, 2, 4, 16, [16 * 7, 16 * 3 + 5], 35)
    c = Q8(p, fmt, 36)
    out, lse = _decode(lib, p, c, S, hint=16 * 6)
    check_attention(p, c, out, lse, f"{fmt} S={S} GQA-4")
