"""Refusals of the append with positions of several axes, of attention under score rules
and of the verdict on drafts (no GPU needed): every case fails before a pointer is looked
at."""

import ctypes

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_qk_gb300 import build
    build.build()
    from paged_kv_cache_qk_gb300 import binding
    return binding


def _layout(lib, nb=64, bs=16, hkv=8, d=128):
    return lib.CacheLayout(nb, bs, hkv, d, 0, bs * hkv * d, hkv * d, d)


def _refused(lib, status, code, words):
    assert status == getattr(lib, "PKVQK_ERR_" + code), lib.pkvqk_last_error()
    assert words in lib.pkvqk_last_error().decode()


def _append(lib, T=4, Hq=16, theta=1e6, eps=1e-6, qs=2048, ost=2048, axes=3, table=0, stride=4,
            freq=bytes([0] * 16 + [1] * 24 + [2] * 24), d=128):
    lay = _layout(lib, d=d)
    return lib.pkvqk_norm_rope_append_axes(
        FAKE, qs, 128, FAKE, ost, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, stride, axes, freq,
        FAKE, FAKE, FAKE, theta, eps, T, Hq, FAKE, FAKE, ctypes.byref(lay), FAKE, table, None,
        None)


@pytest.mark.parametrize("more,code,words", [
    (dict(axes=0), "INVALID_ARG", "num_axes"), (dict(axes=5), "INVALID_ARG", "num_axes"),
    (dict(axes=2), "INVALID_ARG", "freq_axes[40]"), (dict(freq=None), "INVALID_ARG", "freq_axes"),
    (dict(stride=-1), "INVALID_ARG", "axis stride"), (dict(ost=2044), "INVALID_ARG", "q_out"),
    (dict(qs=2044), "INVALID_ARG", "strides"), (dict(theta=0.0), "INVALID_ARG", "theta"),
    (dict(eps=-1.0), "INVALID_ARG", "eps"), (dict(T=-1), "INVALID_ARG", "num_tokens"),
    (dict(Hq=0), "INVALID_ARG", "num_q_heads"), (dict(table=-1), "INVALID_ARG", "table_positions"),
    (dict(table=(1 << 21) + 1), "INVALID_ARG", "table_positions"),
    (dict(d=64), "UNSUPPORTED", "head_dim"),
])
def test_append_refusals(lib, more, code, words):
    _refused(lib, _append(lib, **more), code, words)


def test_append_of_nothing(lib):
    assert _append(lib, T=0) == lib.PKVQK_OK


def _drafts(lib, kind=0, B=4, K=4, V=1000, ts=(5000, 1000), ds=(4000, 1000), seq=None, kept=None):
    return lib.pkvqk_verify_drafts(FAKE, *ts, FAKE, *ds, kind, FAKE, None, FAKE, B, K, V, FAKE,
                                   FAKE, seq, kept, None, None)


@pytest.mark.parametrize("more,code,words", [
    (dict(kind=3), "UNSUPPORTED", "type"), (dict(kind=-1), "UNSUPPORTED", "type"),
    (dict(B=-1), "INVALID_ARG", "batch"), (dict(B=65536), "INVALID_ARG", "batch"),
    (dict(K=-1), "INVALID_ARG", "max_drafts"), (dict(K=256), "INVALID_ARG", "max_drafts"),
    (dict(V=0), "INVALID_ARG", "vocab_size"), (dict(V=1 << 20), "INVALID_ARG", "vocab_size"),
    (dict(ts=(-5000, 1000)), "INVALID_ARG", "strides"),
    (dict(ds=(4000, -1)), "INVALID_ARG", "strides"),
    (dict(seq=FAKE), "INVALID_ARG", "go together"), (dict(kept=FAKE), "INVALID_ARG", "go together"),
])
def test_draft_refusals(lib, more, code, words):
    _refused(lib, _drafts(lib, **more), code, words)


def test_drafts_of_nothing(lib):
    assert _drafts(lib, B=0) == lib.PKVQK_OK


@pytest.mark.parametrize("sections", [(16, 24), (16, 24, 25), (), (-1, 65), (13,) * 5])
def test_bad_sections(lib, sections):
    with pytest.raises(ValueError, match="sections"):
        lib.rope_axes(sections)


def test_sections(lib):
    assert lib.rope_axes((16, 24, 24)) == bytes([0] * 16 + [1] * 24 + [2] * 24)
    assert lib.rope_axes((24, 20, 20), interleaved=True) == bytes([0, 1, 2] * 20 + [0] * 4)


def _append_tensors():
    h = dict(dtype=torch.bfloat16)
    return dict(q=torch.zeros(5, 4, 128, **h), k=torch.zeros(5, 2, 128, **h),
                v=torch.zeros(5, 2, 128, **h), positions=torch.zeros(3, 5, dtype=torch.int64),
                freq_axes=bytes(64), slot_mapping=torch.zeros(5, dtype=torch.int64),
                gamma_q=torch.zeros(128, **h), gamma_k=torch.zeros(128, **h),
                theta=1e6, eps=1e-6, k_cache=torch.zeros(3, 16, 2, 128, **h),
                v_cache=torch.zeros(3, 16, 2, 128, **h))


@pytest.mark.parametrize("name,value,words", [
    ("q", torch.zeros(5, 4, 128), "q must be bfloat16"),
    ("k", torch.zeros(4, 2, 128, dtype=torch.bfloat16), "agree"),
    ("v", torch.zeros(5, 4, 128, dtype=torch.bfloat16), "agree"),
    ("positions", torch.zeros(3, 4, dtype=torch.int64), "positions"),
    ("positions", torch.zeros(3, 5, dtype=torch.int32), "positions"),
    ("positions", torch.zeros(5, 3, dtype=torch.int64).T, "positions"),
    ("freq_axes", bytes(63), "freq_axes"),
    ("slot_mapping", torch.zeros(5, dtype=torch.int32), "slot_mapping"),
    ("gamma_k", torch.zeros(64, dtype=torch.bfloat16), "gamma_k"),
    ("k_cache", torch.zeros(3, 16, 2, 128, dtype=torch.float16), "bfloat16"),
    ("v_cache", torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16), "share one layout"),
])
def test_append_tensors_refused(lib, name, value, words):
    args = _append_tensors() | {name: value}
    with pytest.raises(ValueError, match=words):
        lib.norm_rope_append_axes(**args)


def test_host_tensors_refused(lib):
    with pytest.raises(lib.PkvqkError):
        lib.norm_rope_append_axes(**_append_tensors())
    with pytest.raises(lib.PkvqkError):
        lib.verify_drafts(**_draft_tensors())


def _draft_tensors():
    i = dict(dtype=torch.int32)
    return dict(target_probs=torch.zeros(2, 4, 9), draft_probs=torch.zeros(2, 3, 9),
                draft_tokens=torch.zeros(2, 3, **i), uniforms=torch.zeros(2, 4),
                tokens=torch.zeros(2, 4, **i), num_accepted=torch.zeros(2, **i))


@pytest.mark.parametrize("name,value,words", [
    ("target_probs", torch.zeros(2, 4, 9, dtype=torch.float64), "float32"),
    ("target_probs", torch.zeros(2, 3, 9), "target_probs"),
    ("target_probs", torch.zeros(2, 9, 4).transpose(1, 2), "target_probs"),
    ("draft_probs", torch.zeros(2, 3, 9, dtype=torch.bfloat16), "type"),
    ("draft_probs", torch.zeros(2, 2, 9), "draft_probs"),
    ("draft_probs", torch.zeros(2, 3, 8), "draft_probs"),
    ("draft_tokens", torch.zeros(2, 3, dtype=torch.int64), "draft_tokens"),
    ("uniforms", torch.zeros(2, 3), "uniforms"),
    ("uniforms", torch.zeros(2, 4, dtype=torch.float64), "uniforms"),
    ("tokens", torch.zeros(2, 3, dtype=torch.int32), "tokens"),
    ("num_accepted", torch.zeros(3, dtype=torch.int32), "num_accepted"),
    ("draft_lens", torch.zeros(3, dtype=torch.int32), "draft_lens"),
    ("seq_lens", torch.zeros(2, dtype=torch.int64), "seq_lens"),
])
def test_draft_tensors_refused(lib, name, value, words):
    with pytest.raises(ValueError, match=words):
        lib.verify_drafts(**(_draft_tensors() | {name: value}))


def _scored(lib, name, softcap=0.0, window=0, rules=True, B=4, T=1, Hq=16, S=1, ws=0, scale=0.0,
            d=128):
    lay = _layout(lib, d=d)
    r = lib.ScoreRules(softcap, window, None, None, None)
    rules = ctypes.byref(r) if rules else None
    if name == "pkvqk_paged_prefill_varlen_scored":
        return getattr(lib, name)(FAKE, 2048, 128, FAKE, T, B * T, FAKE, FAKE, ctypes.byref(lay),
                                  FAKE, 16, FAKE, B, Hq, S, 256, scale, rules, FAKE, None, FAKE,
                                  ws, None, None)
    return getattr(lib, name)(FAKE, 2048, 128, FAKE, FAKE, ctypes.byref(lay), FAKE, 16, FAKE, B, T,
                              Hq, S, 256, scale, rules, FAKE, None, FAKE, ws, None, None)


SCORED = ["pkvqk_paged_decode_scored", "pkvqk_paged_prefill_scored",
          "pkvqk_paged_prefill_varlen_scored"]


@pytest.mark.parametrize("name", SCORED)
@pytest.mark.parametrize("more,code,words", [
    (dict(rules=False), "INVALID_ARG", "rules is NULL"),
    (dict(softcap=-1.0), "INVALID_ARG", "softcap"),
    (dict(softcap=float("nan")), "INVALID_ARG", "softcap"),
    (dict(softcap=float("inf")), "INVALID_ARG", "softcap"),
    (dict(softcap=2.0 ** -21), "INVALID_ARG", "softcap"),
    (dict(softcap=2.0 ** 21), "INVALID_ARG", "softcap"),
    (dict(window=-1), "INVALID_ARG", "window"),
    (dict(Hq=12), "INVALID_ARG", "num_q_heads"), (dict(T=0), "INVALID_ARG", "q_len"),
    (dict(S=257), "INVALID_ARG", "num_splits"), (dict(S=2), "WORKSPACE_TOO_SMALL", "workspace"),
    (dict(scale=float("nan")), "INVALID_ARG", "scale"), (dict(d=64), "UNSUPPORTED", "head_dim"),
])
def test_scored_refusals(lib, name, more, code, words):
    _refused(lib, _scored(lib, name, **more), code, words)


@pytest.mark.parametrize("name", SCORED)
def test_scored_attention_of_nothing(lib, name):
    assert _scored(lib, name, softcap=5.0, window=3, B=0) == lib.PKVQK_OK


@pytest.mark.parametrize("name,value,words", [
    ("slopes", torch.zeros(3), "slopes"), ("slopes", torch.zeros(4, dtype=torch.float64), "slopes"),
    ("first_keys", torch.zeros(2, dtype=torch.int32), "first_keys"),
    ("first_keys", torch.zeros(6, dtype=torch.int64), "first_keys"),
    ("prefix_lens", torch.zeros(6, dtype=torch.int32), "prefix_lens"),
    ("out", torch.zeros(6, 4, 128), "out"), ("lse_out", torch.zeros(5, 4), "lse_out"),
    ("k_cache", torch.zeros(3, 16, 2, 128), "bfloat16"),
    ("seq_lens", torch.zeros(2, dtype=torch.int64), "seq_lens"),
    ("block_tables", torch.zeros(3, 2, dtype=torch.int32), "block_tables"),
    ("q_len", 2, "q_len"),
])
def test_scored_tensors_refused(lib, name, value, words):
    h = dict(dtype=torch.bfloat16)
    args = dict(q=torch.zeros(6, 4, 128, **h), k_cache=torch.zeros(3, 16, 2, 128, **h),
                v_cache=torch.zeros(3, 16, 2, 128, **h),
                block_tables=torch.zeros(2, 2, dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32), out=torch.zeros(6, 4, 128, **h),
                q_len=3) | {name: value}
    for f in (lib.paged_decode_scored, lib.paged_prefill_scored):
        with pytest.raises(ValueError, match=words):
            f(**args)
    if name != "q_len":
        del args["q_len"]
        cu = torch.tensor([0, 3, 6], dtype=torch.int32)
        with pytest.raises(ValueError, match=words):
            lib.paged_prefill_varlen_scored(args.pop("q"), cu, 3, **args)
