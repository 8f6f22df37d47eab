"""What pkvqk_norm_rope_append_q8 reports: non-finite values of tokens that it appends,
and nothing else."""

import pytest
import torch

from paged_kv_cache_qk_gb300 import workloads
from tests._q8 import Q8
from tests.test_gpu_q8_append import _before, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [[1], [5, 3], [16, 17], [700, 900, 460]],
                         ids=lambda n: f"{sum(n)} tokens")
def test_finite_values_without_eps_are_not_reported(lib, new):
    """eps 0: half-warps without a token normalise zeros."""
    lens = [n + c for n, c in zip(new, (13, 0, 200))]
    nb = sum(-(-n // 16) for n in lens) + 1
    p = workloads.make_problem("q8", 4, 2, 128, 16, lens, new, nb, 80, "cuda", eps=0.0)
    c = Q8(p, "e4m3", 81, unused=None)
    slots = p.slot_mapping.clone()
    if p.T > 8:
        slots[-3:] = -1                      # padding
    before = _before(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(p.q)
    _run(lib, p, c, slots=slots, q_out=q_out, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 0
    _check(p, c, before, q_out, slots=slots)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("tokens", [3, 2100])
def test_non_finite_values_are_reported_where_they_are_appended(lib, tokens, eps):
    p = workloads.make_problem("q8", 4, 2, 128, 16, [tokens], tokens, -(-tokens // 16), 82, "cuda",
                               eps=eps)
    p.v[tokens - 1, 1, 77] = float("nan")
    for skip in (False, True):
        c = Q8(p, "int8", 83, unused=None)
        slots = p.slot_mapping.clone()
        if skip:
            slots[tokens - 1] = -1
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        _run(lib, p, c, slots=slots, q_out=torch.empty_like(p.q), flags=flags)
        torch.cuda.synchronize()
        assert flags.item() == (0 if skip else lib.FLAG_BAD_VALUE)
