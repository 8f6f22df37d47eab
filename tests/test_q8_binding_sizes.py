"""Refusals of the 8-bit calls' Python layer (no GPU needed): tensors of the right type
that are too small, or laid out otherwise, for what the kernels read and write."""

import pytest
import torch

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64
T, HQ, HKV, D = 4, 4, 2, 128


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_qk_gb300 import build
    build.build()
    from paged_kv_cache_qk_gb300 import binding
    return binding


def _caches():
    kc = torch.zeros(4, 16, HKV, D, dtype=torch.int8)
    s = torch.zeros(4, 1, HKV)
    return kc, kc.clone(), s, s.clone()


def _append(lib, **change):
    a = dict(q=torch.zeros(T, HQ, D, dtype=BF), k=torch.zeros(T, HKV, D, dtype=BF),
             v=torch.zeros(T, HKV, D, dtype=BF), pos=torch.zeros(T, dtype=I64),
             slots=torch.zeros(T, dtype=I64), gq=torch.ones(D, dtype=BF),
             gk=torch.ones(D, dtype=BF), q_out=None, rope_table=None, table_positions=0,
             status_flags=None)
    a.update(change)
    lib.norm_rope_append_q8(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["gq"], a["gk"], 1e6,
                            1e-6, *_caches(), q_out=a["q_out"], rope_table=a["rope_table"],
                            table_positions=a["table_positions"], status_flags=a["status_flags"])


def _attend(lib, which, **change):
    a = dict(q=torch.zeros(T, HQ, D, dtype=BF), out=torch.zeros(T, HQ, D, dtype=BF),
             workspace=None, status_flags=None)
    a.update(change)
    table, lens = torch.zeros(T, 4, dtype=I32), torch.zeros(T, dtype=I32)
    kw = dict(workspace=a["workspace"], status_flags=a["status_flags"])
    if which == "varlen":
        cu = torch.arange(T + 1, dtype=I32)
        lib.paged_prefill_varlen_q8(a["q"], cu, 1, *_caches(), table, lens, a["out"], **kw)
    else:
        f = lib.paged_decode_q8 if which == "decode" else lib.paged_prefill_q8
        f(a["q"], *_caches(), table, lens, a["out"], q_len=1, **kw)


@pytest.mark.parametrize("change", [
    # a head size other than the cache's
    dict(q=torch.zeros(T, HQ, 64, dtype=BF)), dict(q=torch.zeros(T, HQ, 256, dtype=BF)),
    dict(k=torch.zeros(T, HKV, 64, dtype=BF)), dict(v=torch.zeros(T, HKV, 64, dtype=BF)),
    dict(q_out=torch.zeros(T, HQ, 64, dtype=BF)),
    # gains
    dict(gq=torch.ones(64, dtype=BF)), dict(gk=torch.ones(127, dtype=BF)),
    dict(gk=torch.ones(256, dtype=BF)[::2]), dict(gq=torch.ones(D)),
    # a rotary table shorter than the positions it is said to hold, or with gaps
    dict(rope_table=torch.zeros(1024 * 8 - 1, dtype=torch.uint8), table_positions=8),
    dict(rope_table=torch.zeros(8, 512, dtype=torch.uint8), table_positions=8),
    dict(rope_table=torch.zeros(16, 1024, dtype=torch.uint8)[::2], table_positions=8),
    dict(status_flags=torch.zeros(1, dtype=torch.uint8)),
    dict(status_flags=torch.zeros(0, dtype=I32))], ids=lambda c: next(iter(c)))
def test_append_refuses(lib, change):
    with pytest.raises(ValueError):
        _append(lib, **change)


@pytest.mark.parametrize("which", ["decode", "prefill", "varlen"])
@pytest.mark.parametrize("change", [
    # q's head size, with a result that would hold 128 a head
    dict(q=torch.zeros(T, HQ, 64, dtype=BF)), dict(q=torch.zeros(T, HQ, 256, dtype=BF)),
    dict(status_flags=torch.zeros(4, dtype=torch.uint8)),
    dict(workspace=torch.zeros(64, 64, dtype=torch.uint8)[:, ::2])], ids=lambda c: next(iter(c)))
def test_attention_refuses(lib, which, change):
    with pytest.raises(ValueError):
        _attend(lib, which, **change)


def test_well_formed_calls_reach_the_library(lib):
    """With tables, flags and workspaces that fit; host tensors are refused there."""
    flags = torch.zeros(1, dtype=I32)
    with pytest.raises(lib.PkvqkError):
        _append(lib, rope_table=torch.zeros(8 * 1024, dtype=torch.uint8), table_positions=8,
                status_flags=flags)
    for which in ("decode", "prefill", "varlen"):
        with pytest.raises(lib.PkvqkError):
            _attend(lib, which, workspace=torch.zeros(256, dtype=torch.uint8), status_flags=flags)
