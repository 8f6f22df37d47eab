"""Helpers of the 8-bit cache tests: seeded caches, their values as the oracle
reads them, and the tolerances.

Tolerances, from the roundings that the kernels make (half a step each):
  * append: the scale is the rule's exactly, unless the largest value lies within
    2^-20 of a power-of-two step (fp32 norm and rotation); a code is the exact
    value's rounding within half a code step and 2^-18 of the value;
  * attention: K, V and q enter the products exactly, P is rounded to f16
    (half a step, 2^-11 relative, of every term p |v|), exp2 and fp32 sums stay
    below 2^-14 of sum p |v|, the output is rounded to bf16 (2^-8 of it):
        |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-14) sum p |v|
    f16 has no smaller step than 2^-24, so a term's P' = p sv / W * P'max (W the
    row's largest p sv) is off by up to 2^-25 absolutely where it is small; the
    kernels keep P'max >= 2^9, so that is p sv off by 2^-34 W, and W <= max sv:
        + 2^-34 max sv sum |code|
    which matters only where V scales of one sequence are 2^20 and more apart;
  * lse: fp32 scores, 128 products of sum |q k| scale up to about 32 with
    2^-24 each at most, and fp32 log2: 2^-11 absolute.
"""

from __future__ import annotations

import numpy as np
import torch

import oracle
from tests._parity import bits, oracle_attention

DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
CLASSES = ("e4m3", "int8")


def code_bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def from_bytes(b, fmt, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(b)).to(device).view(DTYPES[fmt])


class Q8:
    """An 8-bit cache of a workloads.Problem's shape with seeded contents: codes of
    about N(0, 1) values, scales 2^e with e spread over `spread` steps."""

    def __init__(self, p, fmt, seed, device="cuda", spread=3, unused="nan"):
        self.p, self.fmt = p, fmt
        rng = np.random.default_rng(seed)
        nb, bs, H, D = p.k_cache.shape
        self.k, self.ks = self._draw(rng, nb, bs, H, D, fmt, spread, device)
        self.v, self.vs = self._draw(rng, nb, bs, H, D, fmt, spread, device)
        if unused == "nan":
            self.poison_unused()

    @staticmethod
    def _draw(rng, nb, bs, H, D, fmt, spread, device):
        e = rng.integers(-(8 if fmt == "e4m3" else 6), -(8 if fmt == "e4m3" else 6) + spread,
                         (nb, bs // 16, H))
        s = 2.0 ** e
        x = rng.normal(size=(nb, bs // 16, 16, H, D)) / s[:, :, None, :, None]
        c = oracle.q8_bytes(oracle.q8_round(x, fmt), fmt).reshape(nb, bs, H, D)
        return (from_bytes(c, fmt, device),
                torch.from_numpy(s.astype(np.float32)).to(device))

    def poison_unused(self):
        """What no sequence's keys occupy: codes of all ones (an e4m3 NaN), and in
        groups without any key NaN scales."""
        p = self.p
        nb, bs = p.k_cache.shape[:2]
        used = np.zeros((nb, bs), bool)
        for b in range(p.B):
            for n in range(int(p.seq_lens_host[b])):
                used[p.block_tables_host[b, n // bs], n % bs] = True
        dead = torch.from_numpy(~used).to(self.k.device)
        dead_groups = torch.from_numpy(~used.reshape(nb, bs // 16, 16).any(-1)).to(self.k.device)
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            c.view(torch.uint8)[dead] = 0xFF
            s[dead_groups] = float("nan")

    def args(self):
        return self.k, self.v, self.ks, self.vs

    def values(self, which):
        """The cache as bf16 (code * power of two: exact); unused slots as 0."""
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        v = oracle.q8_values(code_bytes(c), self.fmt)
        v = v * np.repeat(s.double().cpu().numpy(), 16, axis=1)[..., None]
        v = np.nan_to_num(v, nan=0.0)
        t = torch.from_numpy(v)
        assert torch.equal(t, t.bfloat16().double())
        return t.bfloat16()


def underflow_term(p, cache, b):
    """2^-34 max sv sum |code| of sequence b, [Hkv, D] (see above)."""
    n = np.arange(int(p.seq_lens_host[b]))
    if n.size == 0:
        return np.zeros((p.Hkv, p.D))
    blk, off = np.asarray(p.block_tables_host)[b, n // p.block_size], n % p.block_size
    ok = (blk >= 0) & (blk < p.num_blocks)
    blk, off = blk[ok], off[ok]
    codes = np.abs(oracle.q8_values(code_bytes(cache.v)[blk, off], cache.fmt)).sum(0)
    return 2.0 ** -34 * cache.vs.double().cpu().numpy()[blk, off // 16].max(0)[:, None] * codes


def check_attention(p, cache, out, lse, what="", scale=None, q=None, seqs=None):
    """out/lse [B, T, Hq(, D)] against the oracle over the cache's values."""
    k, v = cache.values("k"), cache.values("v")
    qb = bits(p.q if q is None else q)
    ref, ref_lse = oracle_attention(p, qb, seqs=seqs, k_cache=k, v_cache=v, scale=scale)
    mag, _ = oracle_attention(p, qb, seqs=seqs, k_cache=k, v_cache=v.abs(), scale=scale)
    got = out.double().cpu().numpy().reshape((p.B,) + ref.shape[1:])
    glse = lse.double().cpu().numpy().reshape((p.B,) + ref_lse.shape[1:])
    if seqs is not None:
        got, glse = got[list(seqs)], glse[list(seqs)]
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    under = np.stack([underflow_term(p, cache, b) for b in (range(p.B) if seqs is None else seqs)])
    under = np.repeat(under, p.Hq // p.Hkv, axis=1)[:, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14) * mag + under
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{(np.abs(got - ref) / np.maximum(tol, 1e-300)).max():.2f} tolerances")
    assert np.array_equal(np.isneginf(glse), np.isneginf(ref_lse)), f"{what}: -inf pattern"
    fin = ~np.isneginf(ref_lse)
    assert (np.abs(glse[fin] - ref_lse[fin]) <= 2.0 ** -11).all(), \
        f"{what}: lse off by {np.abs(glse[fin] - ref_lse[fin]).max():.2e}"


def check_appended(exact, slots, codes0, scales0, codes1, scales1, fmt, what=""):
    """A cache after an append of the float64 values `exact` [T, H, D] at `slots`
    against the rule: codes0/scales0 before, codes1/scales1 after (numpy)."""
    want_c, want_s = oracle.q8_append(exact, slots, codes0, scales0, fmt)
    # the rule's scales for values 2^-20 lower and higher: where they agree, the
    # scale is settled
    lo_s = oracle.q8_append(exact * (1 - 2.0 ** -20), slots, codes0, scales0, fmt)[1]
    hi_s = oracle.q8_append(exact * (1 + 2.0 ** -20), slots, codes0, scales0, fmt)[1]
    s1 = scales1.astype(np.float64)
    nb, bs, H, D = codes0.shape
    touched = np.zeros(nb * bs // 16, bool)
    for slot in np.asarray(slots).tolist():
        if 0 <= slot < nb * bs:
            touched[slot // 16] = True
    touched = touched.reshape(nb, bs // 16)
    assert np.array_equal(scales1[~touched], scales0[~touched], equal_nan=True), \
        f"{what}: a scale outside"
    assert ((s1 == lo_s) | (s1 == hi_s))[touched].all(), f"{what}: scales"
    same = np.repeat((s1 == want_s), 16, axis=1)[..., None] & np.ones(codes0.shape, bool)
    c1 = oracle.q8_values(codes1, fmt)
    written = np.zeros((nb * bs, H, D), bool)
    value = np.zeros((nb * bs, H, D))
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if 0 <= slot < nb * bs:
            written[slot] = True
            value[slot] = exact[t]
    written, value = written.reshape(codes0.shape), value.reshape(codes0.shape)
    # everything not written: the rule's codes, bit for bit where no scale is unsettled
    rest = ~written & same
    assert np.array_equal(c1[rest], want_c[rest], equal_nan=True), f"{what}: another code changed"
    # written: the nearest code
    x = value / np.repeat(s1, 16, axis=1)[..., None]
    with np.errstate(invalid="ignore"):
        step = (np.ldexp(1.0, np.maximum(np.frexp(np.where(x == 0, 1.0, np.abs(x)))[1] - 1, -6) - 3)
                if fmt == "e4m3" else np.ones_like(x))
        err = np.abs(c1 - np.clip(x, -oracle.quantised.TOP[fmt], oracle.quantised.TOP[fmt]))
        ok = err <= step / 2 + 2.0 ** -18 * np.abs(x)
    assert ok[written].all(), f"{what}: {(~ok[written]).sum()} codes are not the nearest"
