"""GPU parity of pkvqk_paged_decode_q8 below 8 kv heads a CTA, where two warps share a
head, over segments long enough to go round the ring of tiles several times, with up to
16 rows a kv head; tolerances in tests/_q8.py."""

import pytest

import numpy as np
import torch

from paged_kv_cache_qk_gb300 import workloads
from tests._q8 import CLASSES, Q8, check_attention

pytestmark = pytest.mark.gpu


def _decode(lib, p, c, S):
    out = torch.full((p.B, p.q_len, p.Hq, p.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.B, p.q_len, p.Hq), float("nan"), device="cuda")
    n = lib.decode_workspace_bytes(p.B, p.q_len, p.Hq, p.D, S)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_decode_q8(p.q, *c.args(), p.block_tables, p.seq_lens, out, q_len=p.q_len,
                        num_splits=S, max_seq_len_hint=p.max_seq_len, lse_out=lse, workspace=ws,
                        status_flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 0
    return out, lse


def _problem(Hq, Hkv, q_len, bs, lens, seed):
    nb = sum(-(-n // bs) for n in lens) + 2
    return workloads.make_problem("q8", Hq, Hkv, 128, bs, lens, q_len, nb, seed, "cuda")


# (Hq, Hkv, q_len): 9 to 16 rows a kv head at 4, 2 and 1 heads a CTA, and up to 8
HEADS = [(32, 4, 2), (12, 4, 3), (12, 4, 4), (12, 4, 5), (14, 2, 2), (8, 1, 2), (4, 4, 13),
         (32, 4, 1), (28, 4, 1), (14, 2, 1), (8, 1, 1)]


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"Hq{h[0]}-Hkv{h[1]}-T{h[2]}")
@pytest.mark.parametrize("S", [1, 2, 0])
def test_long_segments(lib, fmt, heads, S):
    """Tile counts of every remainder by 4, from 32 tiles (twice round a ring) to 150."""
    p = _problem(*heads, 16, [512, 530, 545, 561, 1203, 2391, 40], 90)
    c = Q8(p, fmt, 91)
    out, lse = _decode(lib, p, c, S)
    check_attention(p, c, out, lse, f"{fmt} {heads} S={S}")


@pytest.mark.parametrize("fmt", CLASSES)
@pytest.mark.parametrize("heads", [(32, 4, 2), (12, 4, 5), (32, 4, 1), (14, 2, 2), (8, 1, 1)],
                         ids=lambda h: f"Hq{h[0]}-Hkv{h[1]}-T{h[2]}")
def test_segments_one_after_another(lib, fmt, heads):
    """Balanced schedule over sequences whose padded tile counts are 2 modulo 4 and
    others, several to a CTA and cut across CTAs."""
    lens = ([96, 160, 29, 224, 500, 16, 80, 97] * 48)[:380] + [2000, 4100]
    p = _problem(*heads, 16, lens, 92)
    c = Q8(p, fmt, 93, unused=None)
    out, lse = _decode(lib, p, c, 0)
    seqs = list(range(0, 382, 19)) + [380, 381]
    check_attention(p, c, out, lse, f"{fmt} {heads}", seqs=seqs)
    again, lse2 = _decode(lib, p, c, 0)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    assert np.isfinite(lse.cpu().numpy()).all()
