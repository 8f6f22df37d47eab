"""The operators of one model together, as a server runs them: prompts with images appended
and prefilled, then speculative steps -- append, verify attention, the target's
probabilities, the verdict -- in which a step's rejected tokens are written over by the next.

Each call is compared with the oracle on what the calls before it left in the cache, by the
tolerances of its own tests; the verdicts are equal.
"""

import numpy as np
import pytest
import torch

import oracle
from tests._parity import ULP_TOL, assert_attention_close, bf16_ulp_distance, bits

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, K, V = 8, 2, 128, 16, 3, 700
THETA, EPS = 1e6, 1e-6


class Model:
    """Queries, keys and values of tokens, and a head from attention outputs to tokens."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        self.gq, self.gk = ((1 + 0.1 * torch.randn(D, device="cuda", generator=g)).bfloat16()
                            for _ in range(2))
        self.head = torch.randn(HQ * D, V, device="cuda", generator=g) * 0.1
        self.vocab = torch.randn(V, HQ + 2 * HKV, D, device="cuda", generator=g)
        self.slopes = torch.exp2(-torch.arange(1, HQ + 1, device="cuda").float())

    def qkv(self, tokens):
        x = self.vocab[tokens].bfloat16()
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def probs(self, out):
        return torch.softmax(out.reshape(out.shape[0], -1).float() @ self.head, -1)


def _step(lib, m, cache, tokens, pos, axes, slots, rope):
    """Appends the tokens; returns their rotated queries."""
    kc, vc = cache
    q, k, v = m.qkv(tokens)
    before = bits(kc), bits(vc)
    q_out = torch.empty(len(tokens), HQ, D, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.norm_rope_append_axes(q, k, v, pos, axes, slots, m.gq, m.gk, THETA, EPS, kc, vc,
                              q_out=q_out, rope_table=rope, table_positions=512,
                              status_flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 0
    qh, kco, vco = oracle.norm_rope_append_axes(
        bits(q), bits(k), bits(v), pos.cpu().numpy(), axes, slots.cpu().numpy(), bits(m.gq),
        bits(m.gk), THETA, EPS, *before, BS)
    assert bf16_ulp_distance(bits(q_out), qh).max() <= ULP_TOL
    assert bf16_ulp_distance(bits(kc), kco).max() <= ULP_TOL
    assert np.array_equal(bits(vc), vco)
    return q_out


def _slots(table, seq, first, n):
    at = np.arange(first, first + n)
    return [int(table[seq, p // BS]) * BS + p % BS for p in at]


@pytest.mark.parametrize("interleaved", [False, True])
def test_prompts_with_images_then_speculative_steps(lib, interleaved):
    rng = np.random.default_rng(4)
    m = Model(11)
    prompts = [37, 150, 64, 5]
    B = len(prompts)
    pages = 14
    table = rng.permutation(B * pages).reshape(B, pages).astype(np.int32)
    dev_table = torch.from_numpy(table).cuda()
    cache = tuple(torch.full((B * pages, BS, HKV, D), float("nan"), dtype=torch.bfloat16,
                             device="cuda") for _ in range(2))
    rope = torch.empty(lib.rope_table_bytes(512), dtype=torch.uint8, device="cuda")
    lib.rope_table_build(rope, 512, THETA)
    axes = lib.rope_axes((24, 20, 20) if interleaved else (16, 24, 24), interleaved=interleaved)
    rules = dict(softcap=20.0, window=120, slopes=m.slopes,
                 prefix_lens=torch.tensor([20, 100, 0, 5], dtype=torch.int32, device="cuda"))
    host_rules = {k: v.cpu().numpy() if torch.is_tensor(v) else v for k, v in rules.items()}

    # the prompts: 8 x 8 images of rows and columns after each 8 tokens of text
    total = sum(prompts)
    tokens = torch.from_numpy(rng.integers(0, V, total)).cuda()
    pos = np.zeros((3, total), np.int64)
    at = 0
    for n in prompts:
        for i in range(n):
            block, o = divmod(i, 72)
            base = 16 * block
            text = o < 8
            pos[:, at + i] = base + o if text else (base + 8, base + 8 + (o - 8) // 8,
                                                    base + 8 + (o - 8) % 8)
        at += n
    slots = torch.tensor(sum((_slots(table, b, 0, n) for b, n in enumerate(prompts)), []),
                         device="cuda")
    q = _step(lib, m, cache, tokens, torch.from_numpy(pos).cuda(), axes, slots, rope)
    cu = torch.tensor(np.r_[0, np.cumsum(prompts)], dtype=torch.int32, device="cuda")
    seq_lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    out = torch.empty(total, HQ, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(total, HQ, device="cuda")
    lib.paged_prefill_varlen_scored(q, cu, max(prompts), *cache, dev_table, seq_lens, out,
                                    lse_out=lse, **rules)
    torch.cuda.synchronize()
    ref, ref_lse = oracle.scored_attention(bits(q), bits(cache[0]), bits(cache[1]), table, prompts,
                                           BS, prompts, **host_rules)
    assert_attention_close(bits(out), ref, lse.cpu().numpy(), ref_lse, "prefill")
    last = torch.multinomial(m.probs(out[cu[1:].long() - 1]), 1, generator=m.g)[:, 0]

    # speculative steps: the last token and K drafts of a draft model a sequence
    S = 3
    ws = torch.empty(lib.decode_workspace_bytes(B, K + 1, HQ, D, S), dtype=torch.uint8,
                     device="cuda")
    kept_any = rejected_any = 0
    have = np.array(prompts)
    for step in range(5):
        draft_probs = torch.softmax(torch.randn(B, K, V, device="cuda", generator=m.g), -1)
        lookup = step == 3
        drafts = draft_probs.argmax(-1) if lookup else torch.multinomial(
            draft_probs.view(B * K, V), 1, generator=m.g).view(B, K)
        tokens = torch.cat((last[:, None], drafts), 1).reshape(-1)
        pos = np.concatenate([np.tile(np.arange(n, n + K + 1), (3, 1)) for n in have], 1)
        slots = torch.tensor(sum((_slots(table, b, n, K + 1) for b, n in enumerate(have)), []),
                             device="cuda")
        q = _step(lib, m, cache, tokens, torch.from_numpy(pos).cuda(), axes, slots, rope)
        seq_lens = torch.from_numpy((have + K + 1).astype(np.int32)).cuda()
        out = torch.empty(B, K + 1, HQ, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, K + 1, HQ, device="cuda")
        lib.paged_decode_scored(q, *cache, dev_table, seq_lens, out, q_len=K + 1, num_splits=S,
                                max_seq_len_hint=int(have.max()) + K + 1, lse_out=lse,
                                workspace=ws, **rules)
        torch.cuda.synchronize()
        ref, ref_lse = oracle.scored_attention(
            bits(q), bits(cache[0]), bits(cache[1]), table, have + K + 1, BS, [K + 1] * B,
            **host_rules)
        assert_attention_close(bits(out).reshape(-1, HQ, D), ref,
                               lse.reshape(-1, HQ).cpu().numpy(), ref_lse, f"step {step}")

        target = m.probs(out.view(B * (K + 1), HQ, D)).view(B, K + 1, V)
        u = torch.rand(B, K + 1, device="cuda", generator=m.g)
        got = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
        n = torch.empty(B, dtype=torch.int32, device="cuda")
        lib.verify_drafts(target, None if lookup else draft_probs, drafts.int().contiguous(), u,
                          got, n, seq_lens=seq_lens, kept_lens=seq_lens)
        torch.cuda.synchronize()
        want, want_n = oracle.verify_drafts(
            target.double().cpu().numpy(), None if lookup else draft_probs.double().cpu().numpy(),
            drafts.cpu().numpy(), u.cpu().numpy())
        assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), want_n)
        # what stays in the cache: the last token and the accepted drafts
        have = have + 1 + want_n
        assert np.array_equal(seq_lens.cpu().numpy(), have)
        last = got.gather(1, n.long()[:, None])[:, 0].long()
        assert (last >= 0).all()
        kept_any += int(want_n.sum())
        rejected_any += int((K - want_n).sum())
    assert kept_any and rejected_any
