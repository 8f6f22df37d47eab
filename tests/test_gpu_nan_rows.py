"""A NaN in a query row, or in a key that the row sees, makes that row's output and
log-sum-exp NaN on every attention path and schedule, and changes no other row: the rows
of a call are computed independently, so the others keep their bits."""

import numpy as np
import pytest
import torch

from paged_kv_cache_qk_gb300 import workloads
from tests._q8 import Q8

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _problem(Hq, Hkv, q_len, lens, seed):
    nb = sum(-(-n // 16) for n in lens) + 2
    return workloads.make_problem("nan", Hq, Hkv, 128, 16, lens, q_len, nb, seed, "cuda")


def _run(lib, which, p, cache, q, S):
    out = torch.zeros(p.B, p.q_len, p.Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(p.B, p.q_len, p.Hq, device="cuda")
    size = (lib.prefill_workspace_bytes if "prefill" in which else lib.decode_workspace_bytes)(
        p.B, p.q_len, p.Hq, 128, S)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    getattr(lib, which)(q, *cache, p.block_tables, p.seq_lens, out, q_len=p.q_len, num_splits=S,
                        max_seq_len_hint=p.max_seq_len, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    return out, lse


def _same_but(a, b, rows):
    """a's `rows` [B, T, H] are NaN, everything else has b's bits."""
    (out, lse), (out0, lse0) = a, b
    assert torch.isnan(out.float())[rows].all() and torch.isnan(lse)[rows].all()
    assert not torch.isnan(out0.float()).any() and not torch.isnan(lse0).any()
    assert torch.equal(out[~rows].view(torch.int16), out0[~rows].view(torch.int16))
    assert torch.equal(lse[~rows], lse0[~rows])


# (entry point, Hq, Hkv, q_len, schedules): bf16 CUDA-core dots and mma tiles, 8-bit with
# one and two warps a head and one and two n-tiles, the multi-query kernel, and decode
# calls that run on it
PATHS = [
    ("paged_decode", 16, 8, 1, (1, 3, 0)), ("paged_decode", 16, 8, 4, (1, 3, 0)),
    ("paged_decode", 32, 4, 5, (1, 2, 0)), ("paged_prefill", 16, 8, 40, (1, 3)),
    ("paged_decode_q8", 16, 8, 1, (1, 3, 0)), ("paged_decode_q8", 16, 8, 5, (1, 3, 0)),
    ("paged_decode_q8", 32, 4, 2, (1, 3, 0)), ("paged_decode_q8", 14, 2, 1, (1, 3, 0)),
    ("paged_decode_q8", 32, 4, 5, (1, 2, 0)), ("paged_prefill_q8", 16, 8, 40, (1, 3)),
]
LENS = [300, 45, 700]


def _cache(p, which):
    if which.endswith("q8"):
        return Q8(p, "e4m3", 5, unused=None).args()
    return p.k_cache, p.v_cache


@pytest.mark.parametrize("path", PATHS, ids=lambda x: f"{x[0]}-{x[1]}q{x[2]}kv-T{x[3]}")
def test_nan_in_a_query_row(lib, path):
    which, Hq, Hkv, q_len, schedules = path
    p = _problem(Hq, Hkv, q_len, LENS, 61)
    cache = _cache(p, which)
    q = p.q.clone()
    rows = torch.zeros(p.B, q_len, Hq, dtype=torch.bool, device="cuda")
    for b, t, h in ((0, 0, 1), (2, q_len - 1, Hq - 1), (2, q_len // 2, 0)):
        q[b * q_len + t, h, 5 + h] = NAN
        rows[b, t, h] = True
    for S in schedules:
        _same_but(_run(lib, which, p, cache, q, S), _run(lib, which, p, cache, p.q, S), rows)


@pytest.mark.parametrize("path", PATHS, ids=lambda x: f"{x[0]}-{x[1]}q{x[2]}kv-T{x[3]}")
def test_nan_in_a_key(lib, path):
    """One key of the prior context (seen by every token) and one among the new tokens
    (seen from its own token on)."""
    which, Hq, Hkv, q_len, schedules = path
    p = _problem(Hq, Hkv, q_len, LENS, 62)
    clean = _cache(p, which)
    k = clean[0].clone()
    rows = torch.zeros(p.B, q_len, Hq, dtype=torch.bool, device="cuda")
    group = Hq // Hkv
    for b, n, kvh in ((0, 130, 1), (2, LENS[2] - q_len + q_len // 2, 0)):
        at = int(p.block_tables_host[b, n // 16]), n % 16, kvh, 9
        if k.dtype == torch.bfloat16:
            k[at] = NAN
        else:
            k.view(torch.uint8)[at] = 0x7F
        first = max(0, n - (LENS[b] - q_len))
        rows[b, first:, kvh * group:(kvh + 1) * group] = True
    for S in schedules:
        _same_but(_run(lib, which, p, (k, *clean[1:]), p.q, S),
                  _run(lib, which, p, clean, p.q, S), rows)


def test_combine_of_partials_with_a_nan(lib):
    """The merge by itself: NaN among the splits, beside empty ones, in any lane."""
    rng = np.random.default_rng(3)
    rows, S = 40, 70
    o = torch.from_numpy(rng.normal(size=(rows, S, 128)).astype(np.float32)).cuda()
    lse = torch.from_numpy(rng.normal(size=(rows, S)).astype(np.float32)).cuda()
    lse[3:20, :60] = float("-inf")
    lse[30] = float("-inf")
    dirty = lse.clone()
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for r, j in ((0, 0), (4, 65), (5, 3), (21, 33), (39, 69)):
        dirty[r, j] = NAN
        hit[r] = True
    res = []
    for x in (lse, dirty):
        out = torch.zeros(rows, 128, dtype=torch.bfloat16, device="cuda")
        merged = torch.zeros(rows, device="cuda")
        lib.lse_combine(o, x, rows, S, out, merged)
        torch.cuda.synchronize()
        res.append((out, merged))
    (out0, lse0), (out, merged) = res
    assert torch.isnan(out.float())[hit].all() and torch.isnan(merged)[hit].all()
    assert torch.equal(out[~hit].view(torch.int16), out0[~hit].view(torch.int16))
    assert torch.equal(merged[~hit], lse0[~hit])
    assert torch.all(out[30] == 0) and torch.isneginf(merged[30])
