"""Pins of the oracle's steps beyond plain causal attention."""

import numpy as np
import pytest

import oracle
from oracle.scored import visible


def _bits(rng, *shape):
    return oracle.f64_to_bf16_bits(rng.normal(size=shape))


def _axes_case(rng, T=5, Hq=4, Hkv=2, nb=3, bs=16):
    return dict(q=_bits(rng, T, Hq, 128), k=_bits(rng, T, Hkv, 128), v=_bits(rng, T, Hkv, 128),
                gamma_q=_bits(rng, 128), gamma_k=_bits(rng, 128), theta=1e6, eps=1e-6,
                k_cache=_bits(rng, nb, bs, Hkv, 128), v_cache=_bits(rng, nb, bs, Hkv, 128),
                slot_mapping=np.array([3, 17, -1, 40, 99])[:T], block_size=bs)


def test_equal_positions_on_every_axis_are_the_plain_append():
    rng = np.random.default_rng(1)
    c = _axes_case(rng)
    pos = np.array([0, 7, 8191, 31, 100000])
    got = oracle.norm_rope_append_axes(positions=[pos] * 3, freq_axes=[0] * 16 + [1] * 24 + [2] * 24,
                                       **c)
    want = oracle.norm_rope_append(positions=pos, **c)[:3]
    assert all(np.array_equal(g, w) for g, w in zip(got, want))


def test_each_frequency_turns_by_its_own_axis():
    """Two axes in turn: the even frequencies are those of one append, the odd of another."""
    rng = np.random.default_rng(2)
    c = _axes_case(rng)
    pos = rng.integers(0, 5000, size=(2, 5))
    got = oracle.norm_rope_append_axes(positions=pos, freq_axes=[0, 1] * 32, **c)[0]
    for a in range(2):
        want = oracle.norm_rope_append(positions=pos[a], **c)[0]
        at = np.r_[a:64:2, 64 + a:128:2]
        assert np.array_equal(got[..., at], want[..., at])


@pytest.mark.parametrize("p,L,window,first,prefix,want", [
    (9, 20, 0, 0, 0, (0, 10)), (9, 20, 4, 0, 0, (6, 10)), (9, 20, 1, 0, 0, (9, 10)),
    (9, 20, 0, 5, 0, (5, 10)), (9, 20, 4, 8, 0, (8, 10)), (9, 20, 0, 0, 15, (0, 15)),
    (9, 20, 0, 0, 50, (0, 20)), (9, 20, 4, 0, 15, (6, 15)), (9, 20, 0, 10, 0, (10, 10)),
    (9, 20, 0, 30, 15, (30, 30)), (-2, 3, 0, 0, 0, (0, 0)), (0, 1, 9, 0, 1, (0, 1)),
])
def test_visible_interval(p, L, window, first, prefix, want):
    assert visible(p, L, window, first, prefix) == want


def _attention_case(rng, L=40, n=3, Hq=4, Hkv=2, bs=16):
    P = -(-L // bs)
    return dict(q=_bits(rng, n, Hq, 128), k_cache=_bits(rng, P + 2, bs, Hkv, 128),
                v_cache=_bits(rng, P + 2, bs, Hkv, 128),
                block_tables=rng.permutation(P + 2)[:P][None], seq_lens=[L], block_size=bs,
                q_lens=[n])


def test_no_rule_is_plain_attention():
    rng = np.random.default_rng(3)
    c = _attention_case(rng)
    out, lse = oracle.scored_attention(**c)
    ref, ref_lse = oracle.paged_attention(c["q"][None], c["k_cache"], c["v_cache"],
                                          c["block_tables"], [40], 16, q_len=3)
    assert np.allclose(out, ref[0], rtol=1e-12) and np.allclose(lse, ref_lse[0], rtol=1e-12)


def test_rules_by_brute_force():
    """One head at a time, key by key in Python floats."""
    rng = np.random.default_rng(4)
    c = _attention_case(rng)
    slopes = [0.5, 0.25, 0.1, 0.01]
    first = [0, 30, 39]
    out, lse = oracle.scored_attention(**c, softcap=3.0, window=25, slopes=slopes,
                                       first_keys=first, prefix_lens=[39])
    q = oracle.bf16_bits_to_f64(c["q"])
    kc, vc = (oracle.bf16_bits_to_f64(c[x]) for x in ("k_cache", "v_cache"))
    for t in range(3):
        p = 37 + t
        for h in range(4):
            num, den = np.zeros(128), 0.0
            for n in range(40):
                seen = n >= first[t] and p - n < 25 and (n <= p or n < 39)
                if not seen:
                    continue
                at = c["block_tables"][0][n // 16], n % 16, h // 2
                s = float(q[t, h] @ kc[at]) / 128 ** 0.5
                s = 3.0 * np.tanh(s / 3.0) - slopes[h] * abs(p - n)
                num += np.exp(s) * vc[at]
                den += np.exp(s)
            assert np.allclose(out[t, h], num / den, rtol=1e-10)
            assert np.isclose(lse[t, h], np.log(den), rtol=1e-10)


def test_a_row_without_keys_is_zero():
    rng = np.random.default_rng(5)
    c = _attention_case(rng)
    out, lse = oracle.scored_attention(**c, first_keys=[0, 39, 40])
    assert not out[1:].any(axis=(1, 2))[0] and np.isneginf(lse[1]).all()
    assert np.isfinite(lse[0]).all() and np.isneginf(lse[2]).all()


def test_verdict_by_hand():
    t = np.array([[[0.5, 0.5, 0.0, 0.0], [0.0, 0.25, 0.25, 0.5]]])
    d = np.array([[[0.25, 0.75, 0.0, 0.0]]])
    # u q(1) = 0.75 u < 0.5: kept below u = 2/3, then the second row decides
    out, n = oracle.verify_drafts(t, d, np.array([[1]]), np.array([[0.5, 0.25]]))
    assert out.tolist() == [[1, 2]] and n.tolist() == [1]
    # refused: only token 0 has more of p than of q
    out, n = oracle.verify_drafts(t, d, np.array([[1]]), np.array([[0.7, 0.99]]))
    assert out.tolist() == [[0, -1]] and n.tolist() == [0]
    # certain draft: what is left is p without it
    out, n = oracle.verify_drafts(t, None, np.array([[1]]), np.array([[0.5, 0.0]]))
    assert out.tolist() == [[0, -1]] and n.tolist() == [0]
    # p == q: nothing is left, p itself
    out, n = oracle.verify_drafts(t, t[:, :1], np.array([[2]]), np.array([[0.0, 0.5]]))
    assert out.tolist() == [[1, -1]] and n.tolist() == [0]


def test_verdicts_follow_the_target():
    """Over uniforms on a grid the first token has the target's own frequencies."""
    t = np.array([0.1, 0.2, 0.3, 0.4])
    d = np.array([0.4, 0.3, 0.2, 0.1])
    m = 40
    count = np.zeros(4)
    for x in range(4):
        grid = (np.arange(m) + 0.5) / m
        u = np.stack(np.meshgrid(grid, grid), -1).reshape(-1, 2)
        B = len(u)
        out, _ = oracle.verify_drafts(np.broadcast_to(t, (B, 2, 4)), np.broadcast_to(d, (B, 1, 4)),
                                      np.full((B, 1), x), u)
        count += d[x] * np.bincount(out[:, 0], minlength=4) / B
    # a grid of m cells places each border within half a cell: 0.5 / m for the acceptance
    # and 0.5 / m for the draw, over the four drafts' masses
    assert np.abs(count - t).max() <= 1.0 / m
