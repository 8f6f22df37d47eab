"""The append of many tokens with more head vectors than four half-warp passes of a narrow CTA
hold (more than 24): its own launch, for one position and for several axes, with and without
a rotary table, against the fp64 oracle (1 bf16 ulp, v and untouched slots exact) and bit for
bit against the launch that few tokens take.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_append_axes import _check, _positions, _problem, _table
from tests.test_gpu_norm_rope_append import _run_and_check, bits_t

pytestmark = pytest.mark.gpu

# 36, 48 and 72 vectors a token: whole and partial passes, and the loop past the first loads;
# 25, the least, and 14 q and 12 kv heads, whose k vectors start inside a warp
HEADS = [(32, 4), (40, 8), (64, 8), (24, 1), (24, 12)]


@pytest.mark.parametrize("T", [1024, 1500])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_one_position(lib, Hq, Hkv, T):
    p = _problem(Hq, Hkv, 16, [T], T, 60 + Hq)
    p.positions = _positions(np.random.default_rng(T), 1, T, 65536)[0]
    f, _, _ = _run_and_check(lib, p)
    assert f == 0


def _append(lib, p, lo, hi, q, kc, vc, table, table_positions):
    tail = (p.positions[lo:hi], p.slot_mapping[lo:hi], p.gamma_q, p.gamma_k, p.theta, p.eps)
    if table is None:
        lib.norm_rope_append(q[lo:hi], p.k[lo:hi], p.v[lo:hi], *tail, kc, vc)
    else:
        lib.norm_rope_append_cached(q[lo:hi], p.k[lo:hi], p.v[lo:hi], *tail, kc, vc, table,
                                    table_positions)


@pytest.mark.parametrize("table_positions", [0, 30000, 65536], ids=["computed", "some", "table"])
@pytest.mark.parametrize("Hq,Hkv", HEADS + [(128, 8)])
def test_the_bits_of_few_tokens(lib, Hq, Hkv, table_positions):
    T = 1500
    p = _problem(Hq, Hkv, 16, [T], T, 61 + Hq)
    p.positions = _positions(np.random.default_rng(Hq), 1, T, 65536)[0]
    table = _table(lib, table_positions, p.theta) if table_positions else None
    got = []
    for step in (T, 500):
        q, kc, vc = p.q.clone(), p.k_cache.clone(), p.v_cache.clone()
        for lo in range(0, T, step):
            _append(lib, p, lo, lo + step, q, kc, vc, table, table_positions)
        torch.cuda.synchronize()
        got.append((q, kc, vc))
    assert all(torch.equal(bits_t(a), bits_t(b)) for a, b in zip(*got))
    assert not torch.equal(got[0][0], p.q)


@pytest.mark.parametrize("table_positions", [0, 700, 2000], ids=["computed", "some", "table"])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("sections,interleaved", [((16, 24, 24), False), ((24, 20, 20), True)])
def test_several_axes(lib, sections, interleaved, Hq, Hkv, table_positions):
    T = 1500 if interleaved else 1024
    p = _problem(Hq, Hkv, 16, [T], T, 62 + Hq)
    pos = _positions(np.random.default_rng(Hkv), 3, T, 2000)
    if table_positions == 700:
        pos[:, ::2] %= 700                     # every other token lies in the table whole
    _check(lib, p, pos, lib.rope_axes(sections, interleaved=interleaved), table_positions)


def test_padding_and_bad_slots(lib):
    T = 1100
    p = _problem(40, 8, 16, [T], T, 63)
    slots = p.slot_mapping.clone()
    slots[5:400:7] = -1
    slots[1099] = p.num_blocks * 16
    f, _, _ = _run_and_check(lib, p, slots=slots)
    assert f == lib.FLAG_BAD_SLOT
    f, _, _ = _check(lib, p, _positions(np.random.default_rng(4), 3, T, 900),
                     lib.rope_axes((24, 20, 20), interleaved=True), 2000, slots=slots)
    assert f == lib.FLAG_BAD_SLOT
