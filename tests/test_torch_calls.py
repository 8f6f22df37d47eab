"""The native part of the binding (no GPU needed): what it refuses before the C entry is
called, and that nothing of a refused call is kept."""

import sys

import pytest
import torch

BF = dict(dtype=torch.bfloat16)
I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_qk_gb300 import build
    build.build()
    from paged_kv_cache_qk_gb300 import binding
    return binding


def _decode():
    return dict(q=torch.zeros(4, 4, 128, **BF), k_cache=torch.zeros(6, 16, 2, 128, **BF),
                v_cache=torch.zeros(6, 16, 2, 128, **BF), block_tables=torch.zeros(2, 3, **I32),
                seq_lens=torch.zeros(2, **I32), out=torch.zeros(2, 2, 4, 128, **BF), q_len=2)


def _varlen():
    a = _decode()
    del a["q_len"]
    return a | dict(cu_seqlens_q=torch.zeros(3, **I32), max_q_len=3)


CACHE = torch.zeros(6, 16, 2, 128, **BF)
WRONG = [
    ("q", torch.zeros(4, 4, 128), "q must be bfloat16"),
    ("q", torch.zeros(4, 512, **BF), "q must be bfloat16"),
    ("q", torch.zeros(4, 4, 256, **BF)[..., ::2], "q must be bfloat16"),
    ("k_cache", CACHE.half(), "bfloat16"), ("k_cache", CACHE[:5], "share one layout"),
    ("v_cache", CACHE.transpose(1, 2).contiguous().transpose(1, 2), "share one layout"),
    ("block_tables", torch.zeros(2, 3), "block_tables"),
    ("block_tables", torch.zeros(3, 3, **I32), "block_tables"),
    ("block_tables", torch.zeros(3, 2, **I32).T, "block_tables"),
    ("seq_lens", torch.zeros(2, dtype=torch.int64), "seq_lens"),
    ("seq_lens", torch.zeros((), **I32), "seq_lens"),
    ("out", torch.zeros(2, 2, 4, 128), "out"), ("out", torch.zeros(2, 2, 4, 64, **BF), "out"),
    ("lse_out", torch.zeros(15), "lse_out"), ("lse_out", torch.zeros(16, **BF), "lse_out"),
    ("slopes", torch.zeros(3), "slopes"), ("first_keys", torch.zeros(3, **I32), "first_keys"),
    ("prefix_lens", torch.zeros(4, **I32), "prefix_lens"),
    ("workspace", torch.zeros(4, 4, dtype=torch.uint8).T[:, :2], "workspace"),
    ("status_flags", torch.zeros(1), "status_flags"),
    ("window", 1 << 31, "window"), ("num_splits", -(1 << 31) - 1, "num_splits"),
]


@pytest.mark.parametrize("name,value,words", WRONG, ids=[f"{n}{i}" for i, (n, _, _)
                                                         in enumerate(WRONG)])
def test_attention_refuses(lib, name, value, words):
    for f, args in ((lib.paged_decode_scored, _decode()), (lib.paged_prefill_scored, _decode()),
                    (lib.paged_prefill_varlen_scored, _varlen())):
        with pytest.raises(ValueError, match=words):
            f(**(args | {name: value}))


def test_rows_and_lengths_agree(lib):
    with pytest.raises(ValueError, match="q_len rows"):
        lib.paged_decode_scored(**(_decode() | dict(q_len=3)))
    with pytest.raises(ValueError, match="q_len"):
        lib.paged_decode_scored(**(_decode() | dict(q_len=-2)))
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        lib.paged_prefill_varlen_scored(**(_varlen() | dict(cu_seqlens_q=torch.zeros(2, **I32))))


@pytest.mark.parametrize("name,value", [("q", None), ("k_cache", [1]), ("seq_lens", (4, 4)),
                                        ("q_len", 2.0), ("window", "4"), ("softcap", "no"),
                                        ("lse_out", 1)])
def test_other_types_refused(lib, name, value):
    with pytest.raises(TypeError):
        lib.paged_decode_scored(**(_decode() | {name: value}))


def test_stream_objects(lib):
    class Stream:
        cuda_stream = 0

    with pytest.raises(AttributeError):
        lib.paged_decode_scored(**(_decode() | dict(stream=7)))
    with pytest.raises(lib.PkvqkError, match="device memory|cudaPointerGetAttributes"):
        lib.paged_decode_scored(**(_decode() | dict(stream=Stream())))


def test_a_call_keeps_nothing(lib):
    args = _decode() | dict(softcap=30.0, lse_out=torch.zeros(16), stream=None)
    before = {k: sys.getrefcount(v) for k, v in args.items()}
    for _ in range(50):
        with pytest.raises(lib.PkvqkError):     # host tensors
            lib.paged_decode_scored(**args)
        with pytest.raises(ValueError):
            lib.paged_decode_scored(**(args | dict(q_len=7)))
    after = {k: sys.getrefcount(v) for k, v in args.items()}
    tensors = [k for k, v in args.items() if isinstance(v, torch.Tensor)]
    assert {k: before[k] for k in tensors} == {k: after[k] for k in tensors}


def test_number_of_arguments(lib):
    calls = lib._native_calls()
    for name in ("append_axes", "decode_scored", "prefill_scored", "prefill_varlen_scored",
                 "verify_drafts"):
        with pytest.raises(TypeError, match="arguments"):
            getattr(calls, name)(1, 2, 3)


def test_frequencies_as_a_list(lib):
    h = torch.zeros(5, 2, 128, **BF)
    args = dict(q=h, k=h, v=h, positions=torch.zeros(3, 5, dtype=torch.int64),
                slot_mapping=torch.zeros(5, dtype=torch.int64), gamma_q=torch.zeros(128, **BF),
                gamma_k=torch.zeros(128, **BF), theta=1e6, eps=1e-6, k_cache=CACHE,
                v_cache=CACHE.clone())
    with pytest.raises(ValueError, match="freq_axes"):
        lib.norm_rope_append_axes(**args, freq_axes=[0] * 63)
    with pytest.raises(lib.PkvqkError):         # host tensors: the list itself is fine
        lib.norm_rope_append_axes(**args, freq_axes=[0] * 64)
