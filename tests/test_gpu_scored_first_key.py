"""Attention under score rules: what lies before the first key that any row sees may hold
anything, also where rows that see nothing, or first keys that fall from row to row, stand
between a row's own bound and that key.

Bounds: those of test_gpu_scored_attention, whose Case is used.
"""

import numpy as np
import pytest
import torch

from oracle.scored import visible
from tests.test_gpu_scored_attention import NAN, Case

pytestmark = pytest.mark.gpu

# rows per kv head: CUDA-core dots (2), mma tiles (8, 12), the tcgen05 kernel from the decode
# call (20) and from its own, one row tile and several
CALLS = [("paged_decode_scored", 8, 8, 2), ("paged_decode_scored", 16, 8, 4),
         ("paged_decode_scored", 12, 4, 4), ("paged_decode_scored", 32, 8, 5),
         ("paged_prefill_scored", 16, 8, 4), ("paged_prefill_scored", 16, 8, 40),
         ("paged_prefill_scored", 8, 2, 200)]
BS = 16


def _bury(c, first_keys, window=0, prefix_lens=None):
    """NaN in every slot before the first visible key of each sequence, no block where a
    whole page lies before it; returns those keys (the length where no row sees any)."""
    T, firsts = c.q_lens[0], []
    for b, n in enumerate(int(x) for x in c.p.seq_lens_host):
        first = n
        for t in range(T):
            lo, hi = visible(n - T + t, n, window, int(first_keys[b * T + t]),
                             0 if prefix_lens is None else int(prefix_lens[b]))
            if lo < hi:
                first = min(first, lo)
        for key in range(first):
            blk = int(c.p.block_tables_host[b, key // BS])
            c.kc[blk, key % BS] = NAN
            c.vc[blk, key % BS] = NAN
        c.p.block_tables[b, :(n + BS - 1) // BS if first == n else first // BS] = -7
        firsts.append(first)
    return firsts


def _check(lib, c, which, first_keys, prefix_lens=None, **rules):
    rules["first_keys"] = torch.tensor(first_keys, dtype=torch.int32, device="cuda")
    if prefix_lens is not None:
        rules["prefix_lens"] = torch.tensor(prefix_lens, dtype=torch.int32, device="cuda")
    decode = which == "paged_decode_scored"
    for S in (1, 3) + ((0,) if decode else ()):
        c.check(lib, which, S, **rules)


@pytest.mark.parametrize("which,Hq,Hkv,T", CALLS)
def test_first_keys_that_fall_under_a_window(lib, which, Hq, Hkv, T):
    """The earliest window start and the least first key belong to different rows."""
    lens, window = [T + 114, T + 306, T + 517], 100   # the first two at the border of a page
    c = Case(Hq, Hkv, BS, lens, T, 95)
    first = []
    for n in lens:
        first += [n - T - 30] + [0] * (T - 1)  # the first row's own bound lies above its window
    want = _bury(c, first, window)
    assert all(f == n - T + 2 - window for f, n in zip(want, lens))
    _check(lib, c, which, first, window=window)
    _check(lib, c, which, first, window=window, softcap=6.0)


@pytest.mark.parametrize("which,Hq,Hkv,T", CALLS)
def test_rows_that_see_nothing_under_a_window(lib, which, Hq, Hkv, T):
    """Padding in front of the chunk: a first key far behind the row."""
    lens, window = [T + 104, T + 312, T + 517], 10
    c = Case(Hq, Hkv, BS, lens, T, 96)
    first = []
    for n in lens:
        first += [n + 100] + [0] * (T - 1)
    want = _bury(c, first, window)
    assert all(f == n - T + 2 - window for f, n in zip(want, lens))
    _check(lib, c, which, first, window=window)


@pytest.mark.parametrize("which,Hq,Hkv,T", CALLS)
def test_rows_that_see_nothing_without_a_window(lib, which, Hq, Hkv, T):
    """The first rows' bounds lie behind them and before every visible key."""
    lens = [T + 100, T + 300, T + 517]
    c = Case(Hq, Hkv, BS, lens, T, 97)
    first = []
    for n in lens:
        # row t stands at n - T + t: the last row alone sees a key, its own
        first += [n - T + t + 1 for t in range(T - 1)] + [n - 1]
    want = _bury(c, first)
    assert want == [n - 1 for n in lens]
    _check(lib, c, which, first)


@pytest.mark.parametrize("which,Hq,Hkv,T", CALLS)
def test_sequences_of_rows_that_see_nothing(lib, which, Hq, Hkv, T):
    """One sequence without a visible key between two that have them."""
    lens = [T + 100, T + 300, T + 17]
    c = Case(Hq, Hkv, BS, lens, T, 98)
    first = [5] * T + list(range(301, T + 301)) + [0] * T
    want = _bury(c, first)
    assert want == [5, T + 300, 0]
    _check(lib, c, which, first)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("which,Hq,Hkv,T", CALLS)
def test_any_first_keys(lib, which, Hq, Hkv, T, seed):
    """Windows, first keys before, on and past their rows, and prefixes, at random."""
    rng = np.random.default_rng(100 * seed + T)
    lens = [int(rng.integers(T, T + 400)) for _ in range(4)]
    c = Case(Hq, Hkv, BS, lens, T, 99)
    window = int(rng.integers(1, 200)) if seed % 2 else 0
    prefix = [int(rng.integers(-3, n + 9)) for n in lens] if seed % 3 == 0 else None
    first = []
    for n in lens:
        low = int(rng.integers(0, n))          # no row of the sequence sees a key before it
        first += [int(rng.integers(low, n + 3)) for _ in range(T)]
    _bury(c, first, window, prefix)
    _check(lib, c, which, first, prefix, window=window)
