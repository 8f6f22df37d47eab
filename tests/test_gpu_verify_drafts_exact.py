"""pkvqk_verify_drafts where a rounding, or a value that is no probability, would show:
every output equals the oracle's whole-number verdict.
"""

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_verify_drafts import TYPES, _check, _run
from tests.test_oracle_verify_values import JUDGED

pytestmark = pytest.mark.gpu


def _draw(lib, p, u):
    """Tokens drawn from rows p [B, V] at uniforms u [B], checked against the oracle."""
    B = p.shape[0]
    drafts = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    tokens, _ = _check(lib, p[:, None].cuda(), None, drafts,
                       torch.as_tensor(u, dtype=torch.float32)[:, None].cuda())
    return tokens[:, 0]


def test_a_draw_beside_a_border(lib):
    """u times the sum is 2^44 - 2^20 + 1 - 2^-24, 68 bits: a float64 product rounds it to the
    border itself, and the token behind it would be drawn."""
    p = torch.tensor([[1 - 2.0 ** -24, 2.0 ** -44, 2.0 ** -24]])
    assert _draw(lib, p, [1 - 2.0 ** -24]).tolist() == [1]


def test_draws_beside_every_border(lib):
    """Rows whose total is 1 + 2^-20 to 2^19 units, uniforms next to where a border lies."""
    rng = np.random.default_rng(1)
    V = 64
    rows, uniforms = [], []
    for _ in range(40):
        w = rng.integers(1, 1 << 30, size=V).astype(np.float64)
        units = np.rint(w * (2.0 ** 44 / w.sum()))
        p = np.float32(np.ldexp(units, -44))
        total = int(np.rint(np.ldexp(p.astype(np.float64), 44)).sum())
        cum = np.cumsum(np.rint(np.ldexp(p.astype(np.float64), 44)).astype(np.int64))
        at = np.float32(int(cum[rng.integers(0, V)]) / total)
        for u in (np.nextafter(at, np.float32(0)), at, np.nextafter(at, np.float32(2))):
            rows.append(p)
            uniforms.append(u)
    _draw(lib, torch.from_numpy(np.stack(rows)), np.array(uniforms, np.float32))


@pytest.mark.parametrize("V", [5, 70000])
def test_uniforms_of_every_size(lib, V):
    """Uniforms of every exponent over totals from one unit to V whole probabilities."""
    rows = [torch.ones(V), torch.full((V,), 2.0 ** -44), torch.full((V,), 1 - 2.0 ** -24)]
    rows[1][1:] = 0.0
    u = [float(np.ldexp(np.float32(m), -e)) for e in (1, 2, 11, 23, 24, 25, 43, 44, 45, 63, 64,
                                                      65, 126, 127, 140)
         for m in (1.0, 2 - 2.0 ** -23) if np.ldexp(m, -e) < 1]
    u += [2.0 ** -149, 3 * 2.0 ** -149, 1 - 2.0 ** -24, 0.0]
    p = torch.stack([r for r in rows for _ in u])
    tokens = _draw(lib, p, u * len(rows))
    assert (tokens[len(u):2 * len(u)] == 0).all()


def _accept(lib, dtype, cases):
    """cases: (u, q of the draft, p of it); every sequence drafts token 2 of 9."""
    B, V = len(cases), 9
    p = torch.full((B, 2, V), 0.0625)
    q = torch.full((B, 1, V), 0.0625)
    u = torch.full((B, 2), 0.5)
    for b, (ub, qb, pb) in enumerate(cases):
        p[b, 0, 2], q[b, 0, 2], u[b, 0] = pb, qb, ub
    drafts = torch.full((B, 1), 2, dtype=torch.int32, device="cuda")
    args = (p.to(TYPES[dtype]).cuda(), q.to(TYPES[dtype]).cuda(), drafts, u.cuda())
    tokens, n, _, _ = _run(lib, *args)
    ref, ref_n = oracle.verify_drafts(args[0].double().cpu().numpy(),
                                      args[1].double().cpu().numpy(), drafts.cpu().numpy(),
                                      args[3].cpu().numpy())
    assert np.array_equal(tokens, ref) and np.array_equal(n, ref_n)
    return n.tolist()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_values_that_are_no_probabilities_decide_as_what_they_count_as(lib, dtype):
    """Above 1 counts as 1, NaN and negative values as 0, also where a draft is judged."""
    cases = [c[:3] for c in JUDGED]
    assert _accept(lib, dtype, cases) == [kept for *_, kept in JUDGED]
