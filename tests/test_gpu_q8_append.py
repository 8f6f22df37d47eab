"""GPU parity of pkvqk_norm_rope_append_q8 against the fp64 oracle: q within one
bf16 ulp, the scale rule, every code the nearest one, and nothing else touched."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import bf16_ulp_distance, bits
from tests._q8 import CLASSES, Q8, check_appended, code_bytes

pytestmark = pytest.mark.gpu


def _table(lib, p, positions):
    t = torch.empty(lib.rope_table_bytes(positions), dtype=torch.uint8, device="cuda")
    lib.rope_table_build(t, positions, p.theta)
    return t


def _exact(p):
    """float64 q^, k^ and v of a problem's tokens."""
    pos = p.positions.cpu().numpy()[:, None]
    eps, theta = np.float64(np.float32(p.eps)), np.float64(np.float32(p.theta))

    def hat(x, g):
        w = oracle.bf16_bits_to_f64
        return oracle.rope_neox(oracle.rms_norm(w(bits(x)), w(bits(g)), eps), pos, theta)

    return hat(p.q, p.gamma_q), hat(p.k, p.gamma_k), oracle.bf16_bits_to_f64(bits(p.v))


def _run(lib, p, c, slots=None, q_out=None, table=None, n=0, flags=None, **kw):
    lib.norm_rope_append_q8(p.q, p.k, p.v, p.positions, p.slot_mapping if slots is None else slots,
                            p.gamma_q, p.gamma_k, p.theta, p.eps, *c.args(), q_out=q_out,
                            rope_table=table, table_positions=n, status_flags=flags, **kw)


def _check(p, c, before, q_out, slots=None, what=""):
    q, k, v = _exact(p)
    assert bf16_ulp_distance(bits(q_out), oracle.f64_to_bf16_bits(q)).max() <= 1, what
    slots = (p.slot_mapping if slots is None else slots).cpu().numpy()
    for name, exact, codes, scales in (("k", k, c.k, c.ks), ("v", v, c.v, c.vs)):
        check_appended(exact, slots, *before[name], code_bytes(codes), scales.cpu().numpy(),
                       c.fmt, f"{what} {name}")


def _before(c):
    return {"k": (code_bytes(c.k).copy(), c.ks.cpu().numpy().copy()),
            "v": (code_bytes(c.v).copy(), c.vs.cpu().numpy().copy())}


# (Hq, Hkv, new tokens, page, prior contexts): one token, runs that start and end
# inside groups, runs across two windows of 16 tokens, many windows, head counts
# that no part divides, odd page sizes
SHAPES = [
    (16, 8, 1, 16, [0, 1, 15, 16, 31, 200]),
    (16, 8, 5, 16, [0, 13, 14, 27, 100, 15, 16]),
    (32, 4, 16, 64, [3, 64, 0]),
    (14, 2, 17, 48, [15, 1]),
    (8, 1, 33, 96, [30, 0, 7]),
    (3, 3, 100, 32, [5]),
    (12, 4, 300, 256, [200, 8]),
    (1, 1, 1, 16, [0]),
]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"Hq{s[0]}-Hkv{s[1]}-T{s[2]}-bs{s[3]}")
def test_append_matches_oracle(lib, fmt, shape):
    Hq, Hkv, new, bs, priors = shape
    lens = [c + new for c in priors]
    nb = sum(-(-n // bs) for n in lens) + 2
    p = workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, new, nb, 40 + new, "cuda")
    c = Q8(p, fmt, 7 + new, unused=None)
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(p.q, float("nan"))
    _run(lib, p, c, q_out=q_out, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 0
    _check(p, c, before, q_out, what=f"{fmt} {shape}")
    # angles from the table, q in place, the same bits
    n = max(lens)
    d = Q8(p, fmt, 7 + new, unused=None)
    q2 = p.q
    _run(lib, p, d, table=_table(lib, p, n), n=n)
    torch.cuda.synchronize()
    assert torch.equal(q2.view(torch.int16), q_out.view(torch.int16))
    for x, y in zip(c.args(), d.args()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_varlen_chunks_and_table_shorter_than_positions(lib, fmt):
    p = workloads.varlen_prefill(device="cuda", batch=5, lo=1, hi=90, prior_lo=0, prior_hi=50,
                                 seed=77)
    c = Q8(p, fmt, 3, unused=None)
    before = _before(c)
    q_out = torch.empty_like(p.q)
    _run(lib, p, c, q_out=q_out, table=_table(lib, p, 40), n=40)
    torch.cuda.synchronize()
    _check(p, c, before, q_out)


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_padding_and_slots_outside_the_cache(lib, fmt):
    p = workloads.make_problem("q8", 16, 8, 128, 16, [40, 40], 20, 8, 5, "cuda")
    c = Q8(p, fmt, 9, unused=None)
    slots = p.slot_mapping.clone()
    slots[:3] = -1                           # padding before a run
    slots[18:20] = -7                        # and behind it
    slots[25] = 8 * 16                       # too large: skipped and flagged
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(p.q)
    # the token after a gap in a group starts a run of its own there: the run before
    # the gap must not share its group
    slots[24] = -1
    keep = [i for i in range(26, 40) if slots[i] // 16 == slots[23] // 16]
    slots[keep] = -1
    _run(lib, p, c, slots=slots, q_out=q_out, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == lib.FLAG_BAD_SLOT
    _check(p, c, before, q_out, slots=slots)


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_token_by_token_follows_the_rule_each_step(lib, fmt):
    """A sequence that grows by one token a call, values growing: every step
    against the oracle's rule from the state before it."""
    rng = np.random.default_rng(1)
    p = workloads.make_problem("q8", 8, 2, 128, 32, [40], 40, 3, 6, "cuda")
    p.v = (p.v.float() * torch.from_numpy(2.0 ** rng.uniform(-3, 6, (40, 1, 1))).float().cuda()
           ).bfloat16()
    c = Q8(p, fmt, 2, unused=None)
    _, k, v = _exact(p)
    slots = p.slot_mapping.cpu().numpy()
    for t in range(40):
        before = _before(c)
        lib.norm_rope_append_q8(p.q[t:t + 1].clone(), p.k[t:t + 1], p.v[t:t + 1],
                                p.positions[t:t + 1], p.slot_mapping[t:t + 1], p.gamma_q,
                                p.gamma_k, p.theta, p.eps, *c.args())
        torch.cuda.synchronize()
        check_appended(k[t:t + 1], slots[t:t + 1], *before["k"], code_bytes(c.k),
                       c.ks.cpu().numpy(), fmt, f"step {t} k")
        check_appended(v[t:t + 1], slots[t:t + 1], *before["v"], code_bytes(c.v),
                       c.vs.cpu().numpy(), fmt, f"step {t} v")


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_extreme_and_non_finite_values(lib, fmt):
    p = workloads.make_problem("q8", 4, 2, 128, 16, [16, 3, 2, 9], 2, 8, 8, "cuda")
    p.v[0] = 0                               # a group of zeros beside tiny values
    p.v[1] = 2.0 ** -120
    p.v[2] = 3e38                            # beyond the largest scale: largest codes
    p.v[3, 0, 5] = float("inf")
    p.v[3, 1, 7] = float("-inf")
    p.v[4, 0, 0] = float("nan")
    c = Q8(p, fmt, 4, unused=None)
    # stored scales that no append wrote count as the smallest
    c.vs[:, :, 0] = float("nan")
    c.vs[:, :, 1] = -1.0
    c.ks[0] = 0.0
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run(lib, p, c, q_out=torch.empty_like(p.q), flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == lib.FLAG_BAD_VALUE
    _, k, v = _exact(p)
    slots = p.slot_mapping.cpu().numpy()
    check_appended(k, slots, *before["k"], code_bytes(c.k), c.ks.cpu().numpy(), fmt, "k")
    check_appended(np.nan_to_num(v, nan=0.0, posinf=np.inf, neginf=-np.inf), slots, *before["v"],
                   code_bytes(c.v), c.vs.cpu().numpy(), fmt, "v")


def test_append_strided_tensors_heads_inside_pages_and_interleaved_caches(lib):
    """q, k, v as slices of one fused projection; K and V codes interleaved in one
    allocation with the heads outside the slots; scales with their own strides."""
    p = workloads.make_problem("q8", 8, 2, 128, 32, [70, 33], 20, 6, 12, "cuda")
    fused = torch.randn(40, 12, 128, device="cuda").bfloat16()
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
    before = _before(c)
    q_out = torch.empty(40, 8, 128, dtype=torch.bfloat16, device="cuda")
    _run(lib, p, c, q_out=q_out)
    torch.cuda.synchronize()
    _check(p, c, before, q_out)


def test_append_on_a_side_stream_captured_and_replayed(lib):
    """Captured once, replayed on new contents: the eager call's bits."""
    p = workloads.make_problem("q8", 16, 8, 128, 16, [30, 99, 16], 3, 12, 15, "cuda")
    c, d = Q8(p, "e4m3", 6, unused=None), Q8(p, "e4m3", 6, unused=None)
    q0, k0 = p.q.clone(), p.k.clone()
    out_c, out_d = torch.empty_like(q0), torch.empty_like(q0)
    _run(lib, p, c, q_out=out_c)
    g = torch.cuda.CUDAGraph()
    start = [x.clone() for x in d.args()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        _run(lib, p, d, q_out=out_d)
    for _ in range(2):
        for x, y in zip(d.args(), start):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        out_d.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_c, out_d)
        for x, y in zip(c.args(), d.args()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # inputs changed in place: the replay reads them
    p.k.copy_(-k0)
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(c.k.view(torch.uint8), d.k.view(torch.uint8))


# many windows (the kernel's narrow form, for larger calls: test_gpu_q8_append_many.py):
# whole groups, runs that start inside a group and end in the next window, many short
# sequences (several runs a window), padding between them
MANY = [
    (16, 8, [1024, 37, 200], 16, [0, 5, 16]),
    (32, 4, [700, 700], 256, [3, 255]),
    (14, 2, [9] * 130, 48, [7] * 130),
    (4, 4, [1, 2, 16, 17, 31, 33] * 12, 16, [0, 15, 8, 1, 30, 2] * 12),
]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"Hq{c[0]}-Hkv{c[1]}-B{len(c[2])}-bs{c[3]}")
def test_append_of_many_tokens(lib, fmt, case):
    Hq, Hkv, new, bs, priors = case
    lens = [c + n for c, n in zip(priors, new)]
    nb = sum(-(-n // bs) for n in lens) + 2
    p = workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, new, nb, 70, "cuda")
    assert p.T >= 1024
    p.v = (p.v.float() * torch.randn(p.T, Hkv, 1, device="cuda").exp2()).bfloat16()   # grows
    n = max(lens)
    for table_positions in (n, n // 2):      # all angles from the table, some computed
        c = Q8(p, fmt, 7, unused=None)
        before = _before(c)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full_like(p.q, float("nan"))
        _run(lib, p, c, q_out=q_out, table=_table(lib, p, n), n=table_positions, flags=flags)
        torch.cuda.synchronize()
        assert flags.item() == 0
        _check(p, c, before, q_out, what=f"{fmt} {case[:2]} table {table_positions}")
    # without a table, the same bits
    d = Q8(p, fmt, 7, unused=None)
    q2 = p.q.clone()
    lib.norm_rope_append_q8(q2, p.k, p.v, p.positions, p.slot_mapping, p.gamma_q, p.gamma_k,
                            p.theta, p.eps, *d.args())
    torch.cuda.synchronize()
    assert torch.equal(q2, q_out)
    for x, y in zip(c.args(), d.args()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_of_many_tokens_padding_bad_slots_and_non_finite_values(lib):
    p = workloads.make_problem("q8", 8, 2, 128, 16, [40] * 60, 20, 200, 71, "cuda")
    c = Q8(p, "e4m3", 8, unused=None)
    slots = p.slot_mapping.clone()
    slots[0:20] = -1                         # a padded sequence
    slots[-1] = p.num_blocks * 16 + 3        # too large
    p.v[100, 0, 3] = float("inf")
    p.v[101, 1, 0] = float("nan")
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(p.q)
    _run(lib, p, c, slots=slots, q_out=q_out, table=_table(lib, p, 40), n=40, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == lib.FLAG_BAD_SLOT | lib.FLAG_BAD_VALUE
    q, k, v = _exact(p)
    s = slots.cpu().numpy()
    check_appended(k, s, *before["k"], code_bytes(c.k), c.ks.cpu().numpy(), "e4m3", "k")
    check_appended(np.nan_to_num(v, nan=0.0, posinf=np.inf), s, *before["v"], code_bytes(c.v),
                   c.vs.cpu().numpy(), "e4m3", "v")
    assert bf16_ulp_distance(bits(q_out), oracle.f64_to_bf16_bits(q)).max() <= 1


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_of_one_slot_given_twice_leaves_other_groups_right(lib, fmt):
    """More tokens than slots in a group: its contents are undefined, every other
    group's are those of a call without it."""
    p = workloads.make_problem("q8", 16, 8, 128, 32, [60], 60, 3, 8, "cuda")
    slots = torch.full((60,), -1, dtype=torch.int64)
    slots[0:16] = torch.arange(16)               # group 0
    slots[16:38] = 32 + torch.arange(22) % 16    # group 2, six slots twice
    slots[38:44] = 80 + torch.arange(6)          # group 5
    slots[50:60] = 20                            # group 1, one slot ten times
    c, d = (Q8(p, fmt, 4, unused=None) for _ in range(2))
    _run(lib, p, c, slots=slots.cuda(), q_out=torch.empty_like(p.q))
    once = slots.clone()
    once[16:38] = -1
    once[50:60] = -1
    before = _before(d)
    q_out = torch.empty_like(p.q)
    _run(lib, p, d, slots=once.cuda(), q_out=q_out)
    torch.cuda.synchronize()
    _check(p, d, before, q_out, slots=once)
    keep = [0, 3, 4, 5]                          # groups whose contents are defined
    for x, y in ((c.k, d.k), (c.v, d.v)):
        x, y = (t.view(torch.uint8).reshape(6, 16, 8, 128)[keep] for t in (x, y))
        assert torch.equal(x, y)
    for x, y in ((c.ks, d.ks), (c.vs, d.vs)):
        assert torch.equal(x.reshape(6, 8)[keep], y.reshape(6, 8)[keep])


@pytest.mark.parametrize("fmt", CLASSES)
def test_append_below_2048_tokens_gives_the_nearest_codes(lib, fmt):
    """1.2 million K values, some within an fp32 norm's error of the middle between two
    codes: each code is the float64 value's (subnormal e4m3 codes aside)."""
    p = workloads.make_problem("q8", 1, 8, 128, 16, [1200], 1200, 76, 17, "cuda")
    c = Q8(p, fmt, 5, unused=None)
    before = _before(c)
    _run(lib, p, c, q_out=torch.empty_like(p.q))
    torch.cuda.synchronize()
    k = _exact(p)[1]
    want, scales = oracle.q8_append(k, p.slot_mapping.cpu().numpy(), *before["k"], fmt)
    assert np.array_equal(scales, c.ks.double().cpu().numpy())
    got = oracle.q8_values(code_bytes(c.k), fmt)
    same = got == want
    if fmt == "e4m3":
        same |= np.maximum(np.abs(got), np.abs(want)) < 2.0 ** -6
    same |= np.isnan(got) & np.isnan(want)
    assert same.all(), f"{(~same).sum()} codes"
