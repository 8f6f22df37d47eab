"""The longest chunk under score rules, rows of it against a float64 softmax.

V is made of unit vectors, one per key tile or one per slot of a tile, so that an output
element is the weight of one tile's keys (or of every tile's key in one slot): a tile or a
slot that is left out, counted twice or taken from elsewhere is off by its whole value.

Tolerance: elements are sums of non-negative terms, and so is their bound.  P is rounded to
bf16 (2^-8 of a weight at most) and the output again (2^-8 of the value): 2^-7 of the value.
A score off by d moves a weight and the sum by d relative each: 2 d.  d is what fp32 sums of
128 exact products are off (128 * 2^-24 of sum |q k| scale), with a cap that every |score| is
below half of the polynomial's error, 6e-7 of the score and so of that sum, and with a bias
2^-23 of its size.  fp32 sums of T terms in any order are off by T 2^-24 = 2^-10 at most, in
the numerator and in the sum of weights.  lse is off by d, by its own rounding and by its sum,
which a thread forms in under 256 steps: 2^-16.
"""

import pytest
import torch

from oracle.scored import visible
from paged_kv_cache_qk_gb300 import workloads

pytestmark = pytest.mark.gpu

T, BS = 16384, 64
# the ends of the chunk and of row tiles and key tiles, early and late
ROWS = [0, 1, 127, 128, 129, 2047, 8191, 8192, 12345, 16127, 16128, 16255, 16256, 16382, 16383]


def _dense(cache, table):
    """[T, 128] float64 of the one sequence's one kv head."""
    return cache[table.long()].reshape(-1, 128)[:T].double()


def _rules(name):
    if name == "none hidden":
        return dict(window=T, softcap=2.0 ** 20)
    if name == "first keys of 0":
        return dict(first_keys=torch.zeros(T, dtype=torch.int32, device="cuda"))
    if name == "cap":
        return dict(softcap=64.0)
    if name == "cap, one reference":
        return dict(softcap=30.0)
    if name == "window, documents":
        cuts = torch.tensor([0, 3000, 3001, 9000, 16200], dtype=torch.int32, device="cuda")
        rows = torch.arange(T, dtype=torch.int32, device="cuda")
        return dict(window=7000, first_keys=cuts[torch.searchsorted(cuts, rows, right=True) - 1])
    return dict(slopes=torch.tensor([2.0 ** -10, 2.0 ** -6, 2.0 ** -13, 0.0], device="cuda"))


@pytest.mark.parametrize("Hq", [2, 4])
@pytest.mark.parametrize("by", ["tile", "slot"])
@pytest.mark.parametrize("name", ["none hidden", "first keys of 0", "cap", "cap, one reference",
                                  "window, documents", "slopes"])
def test_longest_chunk(lib, name, by, Hq):
    p = workloads.make_problem("long", Hq, 1, 128, BS, [T], T, T // BS, 45, "cuda")
    table = p.block_tables[0]
    keys = torch.arange(T, device="cuda")
    v = torch.zeros(T, 128, dtype=torch.bfloat16, device="cuda")
    v[keys, keys // 128 if by == "tile" else keys % 128] = 1.0
    p.v_cache[table.long()] = v.view(T // BS, BS, 1, 128)
    rules = _rules(name)
    if "slopes" in rules:
        rules["slopes"] = rules["slopes"][:Hq].contiguous()
    out = torch.empty(T, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, Hq, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_prefill_scored(p.q, p.k_cache, p.v_cache, p.block_tables, p.seq_lens, out, q_len=T,
                             lse_out=lse, status_flags=flags, **rules)
    torch.cuda.synchronize()
    assert flags.item() == 0

    cap = rules.get("softcap", 0.0)
    K, V = _dense(p.k_cache, table), v.double()
    first = rules.get("first_keys")
    for r in ROWS:
        lo, hi = visible(r, T, rules.get("window", 0), 0 if first is None else int(first[r]))
        for h in range(Hq):
            q = p.q[r, h].double()
            s = K[lo:hi] @ q / 128 ** 0.5
            dot = float((K[lo:hi].abs() @ q.abs()).max()) / 128 ** 0.5
            d = 128 * 2.0 ** -24 * dot
            if cap > 0:
                assert float(s.abs().max()) < cap / 2
                s = cap * torch.tanh(s / cap)
                d += 6e-7 * dot
            if "slopes" in rules:
                slope = float(rules["slopes"][h])
                s = s - slope * (r - keys[lo:hi]).double()
                d += 2.0 ** -23 * slope * r
            ref_lse = torch.logsumexp(s, 0)
            ref = torch.exp(s - ref_lse) @ V[lo:hi]
            off = (out[r, h].double() - ref).abs()
            assert bool((off <= (2.0 ** -7 + 2.0 ** -9 + 2 * d) * ref + 1e-30).all()), (r, h)
            off = abs(float(lse[r, h]) - float(ref_lse))
            assert off <= d + 2.0 ** -16 + 2.0 ** -22 * (1 + abs(float(ref_lse))), (r, h)
