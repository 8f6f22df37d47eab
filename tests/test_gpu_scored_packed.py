"""Packed prompts under score rules: the row tiles that there are, whatever the prompts'
lengths (none, one token, a tile and one token), their number (up to and past what a warp
counts at once) and the heads of a group.  Tolerances as in test_gpu_scored_attention."""

import numpy as np
import pytest
import torch

from tests.test_gpu_scored_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_qk_gb300 import binding
    return binding


def _lengths(rng, batch, tile):
    """New tokens of each sequence: a third of them none, some at the borders of a tile."""
    some = [0, 0, 0, 1, 2, tile - 1, tile, tile + 1, 17, 33]
    q = [int(rng.choice(some)) for _ in range(batch)]
    q[int(rng.integers(batch))] = tile + 5       # one is the longest
    return q


@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 127, 128, 129])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (7, 1)])
def test_row_tiles(lib, batch, Hq, Hkv):
    rng = np.random.default_rng(batch * 10 + Hq)
    tile = 256 // (Hq // Hkv) if batch < 64 else 20
    q = _lengths(rng, batch, tile)
    lens = [max(1, n + int(rng.integers(0, 20))) for n in q]
    c = Case(Hq, Hkv, 16, lens, q, batch)
    c.check(lib, "paged_prefill_scored", 1, window=9)
    c.check(lib, "paged_prefill_scored", 1, softcap=5.0)
    c.check(lib, "paged_prefill_scored", 2, window=30)


def _bits_of(lib, c, longest, splits=1, **rules):
    p = c.p
    out = torch.full((c.rows, p.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.rows, p.Hq), 7.0, device="cuda")
    ws = torch.empty(max(256, lib.prefill_workspace_bytes(1, c.rows, p.Hq, 128, splits)),
                     dtype=torch.uint8, device="cuda")
    lib.paged_prefill_varlen_scored(c.q, p.cu_seqlens, longest, c.kc, c.vc, p.block_tables,
                                    p.seq_lens, out, num_splits=splits, workspace=ws,
                                    max_seq_len_hint=p.max_seq_len, lse_out=lse, **rules)
    torch.cuda.synchronize()
    return out.view(torch.int16), lse


@pytest.mark.parametrize("splits", [1, 3])
def test_a_longer_bound_changes_nothing(lib, splits):
    """max_q_len is a bound: the longest prompt's length and four times it."""
    rng = np.random.default_rng(5)
    q = _lengths(rng, 20, 128)
    c = Case(16, 8, 16, [max(1, n + 40) for n in q], q, 5)
    want = _bits_of(lib, c, max(q), splits, softcap=8.0)
    got = _bits_of(lib, c, 4 * max(q), splits, softcap=8.0)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_batch_and_its_parts(lib):
    """130 prompts at once (more than a warp counts), and 65 at a time: the same bits."""
    rng = np.random.default_rng(6)
    q = _lengths(rng, 130, 24)
    c = Case(8, 4, 16, [max(1, n + int(rng.integers(0, 30))) for n in q], q, 6)
    p = c.p
    want = _bits_of(lib, c, max(q), window=21)
    cu = p.cu_seqlens.cpu().tolist()
    for b0 in (0, 65):
        r0, r1 = cu[b0], cu[b0 + 65]
        out = torch.full((r1 - r0, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((r1 - r0, 8), 7.0, device="cuda")
        part = (p.cu_seqlens[b0:b0 + 66] - r0).contiguous()
        lib.paged_prefill_varlen_scored(c.q[r0:r1], part, max(q), c.kc, c.vc,
                                        p.block_tables[b0:b0 + 65], p.seq_lens[b0:b0 + 65], out,
                                        max_seq_len_hint=p.max_seq_len, lse_out=lse, window=21)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0][r0:r1])
        assert torch.equal(lse, want[1][r0:r1])
