"""Decode, verify and prefill attention under score rules against the fp64 oracle.

Tolerances, against the float64 value o of a row whose weights p sum to 1 over values v:
P is rounded to bf16 (relative 2^-8 a weight at most), so that the numerator is off by at
most 2^-8 sum p |v|, the sum of unrounded weights not at all; the output's own rounding
adds 2^-8 |o| <= 2^-8 sum p |v|.  Scores are off by what fp32 sums of exact products are
(128 terms: 128 * 2^-24 of sum |q k| scale), by tanh's 2e-7 of the cap, and by the bias'
rounding (2^-23 of its size); a score off by d moves a weight by d relative, and the sum by
d too: 2 d sum p |v|.  lse is off by d and by its own rounding.
"""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_qk_gb300 import workloads
from tests._parity import bits

pytestmark = pytest.mark.gpu

NAN = float("nan")


class Case:
    """Sequences of the given lengths whose last q_len (one, or one each) tokens are new."""

    def __init__(self, Hq, Hkv, bs, lens, q_len, seed, gain=1.0, dirty=True, extra=3):
        pages = sum(-(-n // bs) for n in lens)
        varlen = not np.isscalar(q_len)
        self.p = p = workloads.make_problem("scored", Hq, Hkv, 128, bs, lens, q_len, pages + extra,
                                            seed, "cuda")
        self.q_lens = list(q_len) if varlen else [q_len] * len(lens)
        self.varlen = varlen
        self.q = (p.q.float() * gain).bfloat16()
        self.kc, self.vc = p.k_cache.clone(), p.v_cache.clone()
        if dirty:                              # slots past the sequences' ends
            for b, n in enumerate(lens):
                if n % bs:
                    blk = int(p.block_tables_host[b, n // bs])
                    self.kc[blk, n % bs:] = NAN
                    self.vc[blk, n % bs:] = NAN
        self.rows = sum(self.q_lens)

    def tolerance(self, ref, scale, softcap, slopes):
        """(per-row bound of a score's error, bound factor of the output's)."""
        q = self.q.double().abs()
        k = self.p.k_cache.double().abs().amax((0, 1))          # [Hkv, D]
        G = self.p.Hq // self.p.Hkv
        dot = scale * (q * k.repeat_interleave(G, 0)[None]).sum(-1).cpu().numpy()
        d = 128 * 2.0 ** -24 * dot + 2e-7 * softcap * 2
        if slopes is not None:
            d = d + 2.0 ** -23 * slopes.double().abs().cpu().numpy()[None] * max(self.p.seq_lens_host)
        return d

    def check(self, lib, which, S, scale=0.0, hint=None, seqs=None, strided=False, **rules):
        p = self.p
        out = torch.full((self.rows + 2, p.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.rows + 2, p.Hq), 7.0, device="cuda")
        if "prefill" in which:
            size = lib.prefill_workspace_bytes(1, self.rows, p.Hq, 128, S)
        else:
            size = lib.decode_workspace_bytes(p.B, self.q_lens[0], p.Hq, 128, S)
        ws = torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        more = dict(num_splits=S, max_seq_len_hint=p.max_seq_len if hint is None else hint,
                    scale=scale, lse_out=lse, workspace=ws, status_flags=flags, **rules)
        if self.varlen:
            lib.paged_prefill_varlen_scored(self.q, p.cu_seqlens, max(self.q_lens), self.kc,
                                            self.vc, p.block_tables, p.seq_lens, out, **more)
        else:
            getattr(lib, which)(self.q, self.kc, self.vc, p.block_tables, p.seq_lens, out,
                                q_len=self.q_lens[0], **more)
        torch.cuda.synchronize()
        assert flags.item() == 0
        # rows behind the last sequence stay as they were
        assert (out[self.rows:] == 7.0).all() and (lse[self.rows:] == 7.0).all()
        host = {k: v.cpu().numpy() if torch.is_tensor(v) else v for k, v in rules.items()}
        sc = scale if scale > 0 else 128 ** -0.5
        ref, ref_lse = oracle.scored_attention(
            bits(self.q), bits(self.kc), bits(self.vc), p.block_tables_host, p.seq_lens_host,
            p.block_size, self.q_lens, scale=sc, seqs=seqs, **host)
        # sum p |v|, by the same weights over |v|
        mag, _ = oracle.scored_attention(
            bits(self.q), bits(self.kc), bits(self.vc) & 0x7FFF, p.block_tables_host,
            p.seq_lens_host, p.block_size, self.q_lens, scale=sc, seqs=seqs, **host)
        have = ~np.isnan(ref_lse)
        d = self.tolerance(ref, sc, rules.get("softcap", 0.0), rules.get("slopes"))
        got = oracle.bf16_bits_to_f64(bits(out[:self.rows]))
        got_lse = lse[:self.rows].cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(got_lse)[have], np.isneginf(ref_lse)[have])
        empty = np.isneginf(ref_lse)
        assert (got[empty] == 0).all()
        fine = have & ~empty
        bound = (2.0 ** -7 + 2 * d)[..., None] * mag + 1e-30
        over = np.abs(got - ref)[fine] / bound[fine]
        assert np.isfinite(got[fine]).all() and over.max(initial=0) <= 1, over.max()
        err = np.abs(got_lse - np.where(fine, ref_lse, 0))[fine] / \
            (d + 2.0 ** -22 * (1 + np.abs(np.where(fine, ref_lse, 0))))[fine]
        assert err.max(initial=0) <= 1, err.max()
        return out, lse


def _slopes(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)


def _first(rng, c, worst=False):
    """A first key for every row: somewhere before it, on it, or (worst) past it."""
    p = c.p
    first = []
    for b, n in enumerate(c.q_lens):
        for t in range(n):
            pos = int(p.seq_lens_host[b]) - n + t
            first.append(int(rng.integers(0, pos + 1 + (3 if worst else 0))))
    return torch.tensor(first, dtype=torch.int32, device="cuda")


RULES = {
    "none": {},
    "cap": dict(softcap=5.0),
    "cap-tight": dict(softcap=0.25),
    "cap-wide": dict(softcap=1000.0),
    "slopes": dict(slopes=True),
    "window": dict(window=40),
    "window-1": dict(window=1),
    "window-all": dict(window=2 ** 31 - 1),
    "prefix": dict(prefix=True),
    "documents": dict(first=True),
    "empty-rows": dict(worst=True),
    "all": dict(softcap=3.0, slopes=True, window=150, prefix=True, first=True),
}


def _rules(name, c, seed=0):
    r = dict(RULES[name])
    rng = np.random.default_rng(seed)
    if r.pop("slopes", False):
        r["slopes"] = _slopes(c.p.Hq)
    if r.pop("prefix", False):
        top = [int(n) + 5 for n in c.p.seq_lens_host]
        r["prefix_lens"] = torch.tensor([int(rng.integers(0, n)) for n in top], dtype=torch.int32,
                                        device="cuda")
    worst = r.pop("worst", False)
    if r.pop("first", False) or worst:
        r["first_keys"] = _first(rng, c, worst)
    return r


# rows per kv head: CUDA-core dots (1, 2), mma tiles (3 .. 16), the tcgen05 kernel
HEADS = [(8, 8, 1), (16, 8, 1), (32, 8, 1), (32, 4, 1), (14, 2, 1), (12, 4, 2), (16, 8, 5),
         (8, 1, 2), (6, 3, 1), (32, 4, 5), (16, 8, 16)]


@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("Hq,Hkv,T", HEADS)
def test_decode(lib, Hq, Hkv, T, rules):
    c = Case(Hq, Hkv, 16, [T, 45 + T, 300, 17 + T, 129], T, 71, gain=2.0)
    for S in (1, 3, 0):
        c.check(lib, "paged_decode_scored", S, **_rules(rules, c, S))


@pytest.mark.parametrize("bs", [16, 48, 96, 128, 256])
@pytest.mark.parametrize("rules", ["cap", "window", "empty-rows", "all"])
def test_decode_page_sizes(lib, bs, rules):
    for Hq, Hkv, T in ((16, 8, 1), (32, 4, 1), (16, 8, 3)):
        c = Case(Hq, Hkv, bs, [T, 700, 257, 256, 255 + T], T, 72)
        for S in (1, 4, 0):
            c.check(lib, "paged_decode_scored", S, **_rules(rules, c, bs))


@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("Hq,Hkv,T", [(16, 8, 40), (32, 4, 70), (14, 2, 33), (8, 1, 17), (4, 4, 300)])
def test_prefill(lib, Hq, Hkv, T, rules):
    c = Case(Hq, Hkv, 16, [T, T + 45, T + 300], T, 73, gain=2.0)
    for S in (1, 3):
        c.check(lib, "paged_prefill_scored", S, **_rules(rules, c, S))


@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("Hq,Hkv,bs", [(16, 8, 16), (32, 4, 64), (12, 4, 96), (2, 2, 256)])
def test_varlen_prefill(lib, Hq, Hkv, bs, rules):
    c = Case(Hq, Hkv, bs, [130, 300, 1, 40, 400, 257], [130, 200, 1, 7, 1, 129], 74, gain=2.0)
    for S in (1, 2):
        c.check(lib, "paged_prefill_varlen_scored", S, **_rules(rules, c, S))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 127, 128, 129, 500])
def test_windows_at_the_edges_of_pages_and_tiles(lib, window):
    for bs in (16, 64, 128):
        c = Case(16, 8, bs, [511, 512, 513, 640], 1, 75)
        for S in (1, 2, 0):
            c.check(lib, "paged_decode_scored", S, window=window)
        c = Case(8, 4, bs, [300, 384, 385], [150, 128, 129], 76)
        for S in (1, 3):
            c.check(lib, "paged_prefill_varlen_scored", S, window=window, softcap=4.0)


def test_nothing_outside_the_span_is_read(lib):
    """Keys before the first visible one are NaN and their whole pages have no block: the
    results do not notice, and no bad block is reported."""
    for which, Hq, Hkv, T in (("paged_decode_scored", 16, 8, 1), ("paged_decode_scored", 32, 8, 1),
                              ("paged_decode_scored", 16, 8, 4), ("paged_prefill_scored", 16, 8, 40)):
        c = Case(Hq, Hkv, 32, [600, 333, 480], T, 77)
        window = 100
        for b, n in enumerate((600, 333, 480)):
            low = n - T + 1 - window
            for key in range(low):
                blk = int(c.p.block_tables_host[b, key // 32])
                c.kc[blk, key % 32] = NAN
                c.vc[blk, key % 32] = NAN
            c.p.block_tables[b, :low // 32] = -7
        for S in (1, 3) + ((0,) if "decode" in which else ()):
            c.check(lib, which, S, window=window, softcap=6.0)


def test_infinities_and_nan_in_hidden_keys(lib):
    """Documents: the keys of an earlier document hold infinities."""
    for which, Hq, Hkv, T in (("paged_decode_scored", 16, 8, 1), ("paged_decode_scored", 32, 4, 1),
                              ("paged_prefill_scored", 16, 8, 40)):
        c = Case(Hq, Hkv, 16, [200, 333], T, 78)
        first = []
        for b, (n, cut) in enumerate(((200, 101), (333, 250))):
            first += [cut] * T
            for key in range(cut):
                blk = int(c.p.block_tables_host[b, key // 16])
                c.kc[blk, key % 16] = float("inf")
                c.vc[blk, key % 16] = float("-inf")
        c.check(lib, which, 1, first_keys=torch.tensor(first, dtype=torch.int32, device="cuda"),
                slopes=_slopes(Hq))


def test_hints_below_and_above_the_span(lib):
    c = Case(16, 8, 16, [700, 90, 1], 1, 79)
    for hint in (1, 50, 700, 4000, 0):
        c.check(lib, "paged_decode_scored", 5, hint=hint, softcap=5.0)
        c.check(lib, "paged_decode_scored", 5, hint=hint, window=77)


def test_scales_and_caps(lib):
    for Hq, Hkv, T, which in ((16, 8, 1, "paged_decode_scored"), (32, 4, 1, "paged_decode_scored"),
                              (16, 8, 33, "paged_prefill_scored")):
        c = Case(Hq, Hkv, 16, [T + 60, T + 200], T, 80, gain=3.0)
        for scale in (0.01, 0.3, 1.0):
            for cap in (2.0 ** -20, 0.1, 20.0, 2.0 ** 20):
                c.check(lib, which, 1, scale=scale, softcap=cap)


def test_steep_and_negative_slopes(lib):
    """Slopes at which one key holds all the weight, rising ones, and zeros."""
    for Hq, Hkv, T, which in ((16, 8, 1, "paged_decode_scored"), (32, 4, 1, "paged_decode_scored"),
                              (16, 8, 33, "paged_prefill_scored")):
        c = Case(Hq, Hkv, 16, [T + 60, T + 600], T, 81)
        s = torch.zeros(Hq, device="cuda")
        s[:4] = torch.tensor([30.0, -0.5, 1000.0, 1e-6])
        for S in (1, 2):
            c.check(lib, which, S, slopes=s)
            c.check(lib, which, S, slopes=s, softcap=2.0, window=50)


@pytest.mark.parametrize("Hq,Hkv,q_len,S", [(16, 8, 1, 2), (32, 4, 1, 0), (16, 8, 5, 6)])
def test_long_contexts(lib, Hq, Hkv, q_len, S):
    """Sampled sequences of long ones."""
    lens = [8192, 3001, 16384, 500, 9999, 20000]
    c = Case(Hq, Hkv, 16, lens, q_len, 82, gain=3.0)
    c.check(lib, "paged_decode_scored", S, seqs=[1, 5], softcap=30.0)
    c.check(lib, "paged_decode_scored", S, seqs=[0, 5], slopes=_slopes(Hq))
    c.check(lib, "paged_decode_scored", S, seqs=[2, 3, 5], window=4096, hint=4096 + q_len - 1)


def test_long_prefill(lib):
    c = Case(4, 2, 64, [9000, 2048], [600, 2048], 83, gain=2.0)
    for r in (dict(softcap=50.0), dict(window=1000, softcap=20.0), dict(slopes=_slopes(4)),
              dict(prefix_lens=torch.tensor([8999, 700], dtype=torch.int32, device="cuda"))):
        c.check(lib, "paged_prefill_varlen_scored", 1, **r)


def test_without_rules_the_plain_results(lib):
    """All rules off: the plain calls' log-sum-exp and outputs."""
    for T, name in ((1, "paged_decode"), (4, "paged_decode"), (100, "paged_prefill")):
        c = Case(16, 8, 16, [300, 129, T], T, 84, dirty=False)
        for S in (1, 3):
            out, lse = c.check(lib, name + "_scored", S)
            p = c.p
            o2, l2 = torch.empty_like(out), torch.empty_like(lse)
            size = lib.prefill_workspace_bytes(p.B, T, p.Hq, 128, S)
            ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
            getattr(lib, name)(c.q, c.kc, c.vc, p.block_tables, p.seq_lens, o2, q_len=T,
                               num_splits=S, max_seq_len_hint=300, lse_out=l2, workspace=ws)
            torch.cuda.synchronize()
            n = c.rows
            assert torch.allclose(lse[:n], l2[:n], rtol=1e-6, atol=1e-6)
            assert torch.allclose(out[:n].float(), o2[:n].float(), rtol=2.0 ** -7, atol=2e-3)


def test_empty_batch_and_sequences(lib):
    c = Case(16, 8, 16, [33, 0, 5], [33, 0, 5], 85)
    c.check(lib, "paged_prefill_varlen_scored", 1, window=9, softcap=2.0)
    e = torch.empty(0, 16, 128, dtype=torch.bfloat16, device="cuda")
    i = dict(dtype=torch.int32, device="cuda")
    lib.paged_decode_scored(e, c.kc, c.vc, torch.empty(0, 4, **i), torch.empty(0, **i), e, window=3)


def test_strided_q_and_cache_views(lib):
    c = Case(16, 8, 16, [300, 45, 129], 2, 86)
    both = torch.stack((c.kc, c.vc), 1).contiguous()
    c.kc, c.vc = both[:, 0], both[:, 1]
    wide = torch.zeros(c.rows, 20, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:19] = c.q
    c.q = wide[:, 3:19]
    for which in ("paged_decode_scored", "paged_prefill_scored"):
        c.check(lib, which, 2, softcap=4.0, window=60)


def test_graph_on_a_side_stream(lib):
    c = Case(16, 8, 16, [700, 345, 129, 1000], 1, 87)
    rules = dict(softcap=9.0, window=300, slopes=_slopes(16))
    for S in (3, 0):
        out, lse = c.check(lib, "paged_decode_scored", S, **rules)
        p = c.p
        ws = torch.empty(max(lib.decode_workspace_bytes(4, 1, 16, 128, S), 256), dtype=torch.uint8,
                         device="cuda")
        o2, l2 = torch.zeros_like(out[:4]), torch.zeros_like(lse[:4])
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            lib.paged_decode_scored(c.q, c.kc, c.vc, p.block_tables, p.seq_lens, o2, num_splits=S,
                                    max_seq_len_hint=1000, lse_out=l2, workspace=ws, **rules)
        torch.cuda.current_stream().wait_stream(s)
        for _ in range(2):
            o2.zero_()
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o2, out[:4]) and torch.equal(l2, lse[:4])


def test_nan_rows_stay_alone(lib):
    """A NaN in one q row makes NaN of that row only, and a NaN in a visible key of the rows
    that see it."""
    for which, T, S in (("paged_decode_scored", 1, 1), ("paged_decode_scored", 4, 3),
                        ("paged_prefill_scored", 40, 1)):
        c = Case(16, 8, 16, [300, 45, 129], T, 88, dirty=False)
        p = c.p

        def run(q, k):
            out = torch.zeros(c.rows, 16, 128, dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros(c.rows, 16, device="cuda")
            ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
            getattr(lib, which)(q, k, c.vc, p.block_tables, p.seq_lens, out, q_len=T,
                                num_splits=S, lse_out=lse, workspace=ws, softcap=3.0, window=64,
                                slopes=_slopes(16))
            torch.cuda.synchronize()
            return out, lse

        clean = run(c.q, c.kc)
        q = c.q.clone()
        q[T - 1, 5, 9] = NAN
        k = c.kc.clone()
        k[int(p.block_tables_host[2, 100 // 16]), 100 % 16, 3, 11] = NAN   # seen by 100 .. 163
        rows = torch.zeros(c.rows, 16, dtype=torch.bool, device="cuda")
        rows[T - 1, 5] = True
        for t in range(T):
            if 129 - T + t >= 100:
                rows[2 * T + t, 6:8] = True
        out, lse = run(q, k)
        assert torch.isnan(out.float())[rows].all() and torch.isnan(lse)[rows].all()
        assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])


@pytest.mark.parametrize("rules", ["none", "cap", "slopes", "window", "documents", "all"])
def test_more_places_than_sms(lib, rules):
    """Grids that each SM works through several places of: even and packed batches (listed
    and, past 256 sequences, not), with and without boxes of q, whole and split."""
    rng = np.random.default_rng(5)
    lens = [int(rng.integers(1, 400)) for _ in range(40)]
    new = [int(rng.integers(0, n + 1)) for n in lens]
    for Hq, Hkv in ((16, 8), (12, 4)):
        c = Case(Hq, Hkv, 16, lens, new, 90, gain=2.0)
        for S in (1, 3):
            c.check(lib, "paged_prefill_scored", S, seqs=[0, 7, 19, 39], **_rules(rules, c, S))
    lens = [int(rng.integers(1, 40)) for _ in range(300)]
    c = Case(4, 2, 16, lens, [int(rng.integers(0, n + 1)) for n in lens], 91, gain=2.0)
    c.check(lib, "paged_prefill_scored", 1, seqs=list(range(0, 300, 29)), **_rules(rules, c, 1))
    c = Case(16, 8, 16, [300 + 5 * i for i in range(30)], 260, 92, gain=2.0)
    c.check(lib, "paged_prefill_scored", 1, seqs=[0, 17, 29], **_rules(rules, c, 1))


def test_places_in_order_give_the_same_bits(lib):
    """Which SM takes which place is decided as they come free: the results do not show it."""
    rng = np.random.default_rng(6)
    lens = [int(rng.integers(100, 900)) for _ in range(24)]
    c = Case(16, 8, 16, lens, lens, 93, gain=2.0)
    r = _rules("all", c)
    outs = [c.check(lib, "paged_prefill_scored", 1, seqs=[3], **r) for _ in range(4)]
    assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)
