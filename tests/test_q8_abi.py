"""Refusals of the 8-bit cache entry points (no GPU needed): every case fails
before a pointer is looked at."""

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


def _cache(lib, nb=64, bs=16, hkv=8, d=128, fmt=1, strides=None, scale_strides=None):
    strides = strides or (bs * hkv * d, hkv * d, d)
    scale_strides = scale_strides or (bs // 16 * hkv, hkv, 1)
    return lib.Q8Cache(FAKE, FAKE, FAKE, FAKE, lib.CacheLayout(nb, bs, hkv, d, 0, *strides),
                       fmt, 0, *scale_strides)


BAD_CACHES = [
    (dict(d=64), "UNSUPPORTED", "head_dim"),
    (dict(bs=24), "UNSUPPORTED", "block_size"),
    (dict(bs=512), "UNSUPPORTED", "block_size"),
    (dict(nb=0), "INVALID_ARG", "num_blocks"),
    (dict(hkv=0), "INVALID_ARG", "num_kv_heads"),
    (dict(fmt=0), "UNSUPPORTED", "format"),
    (dict(fmt=3), "UNSUPPORTED", "format"),
    (dict(strides=(16384, 1024, 136)), "INVALID_ARG", "multiples of 16"),
    (dict(strides=(16384, -1024, 128)), "INVALID_ARG", "slot_stride"),
    (dict(scale_strides=(8, 8, 0)), "INVALID_ARG", "scale strides"),
    (dict(scale_strides=(-8, 8, 1)), "INVALID_ARG", "scale strides"),
]


def _append(lib, cache, T=4, Hq=16, theta=1e6, eps=1e-6, qst=2048, ost=2048, table=0):
    return lib.pkvqk_norm_rope_append_q8(
        FAKE, qst, 128, FAKE, ost, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, FAKE, FAKE, FAKE,
        theta, eps, T, Hq, None if cache is None else ctypes.byref(cache), FAKE, table, None, None)


def _decode(lib, cache, B=4, q_len=1, Hq=16, S=1, ws=0, maxp=16, qs=(2048, 128), scale=0.0):
    return lib.pkvqk_paged_decode_q8(
        FAKE, *qs, None if cache is None else ctypes.byref(cache), FAKE, maxp, FAKE, B, q_len, Hq,
        S, 256, scale, FAKE, None, FAKE, ws, None, None)


def _prefill(lib, cache, B=4, q_len=32, Hq=16, S=1, ws=0, maxp=16, qs=(2048, 128), scale=0.0):
    return lib.pkvqk_paged_prefill_q8(
        FAKE, *qs, None if cache is None else ctypes.byref(cache), FAKE, maxp, FAKE, B, q_len, Hq,
        S, 256, scale, FAKE, None, FAKE, ws, None, None)


def _varlen(lib, cache, B=4, q_len=32, Hq=16, S=1, ws=0, maxp=16, qs=(2048, 128), scale=0.0,
            cu=FAKE, total=64):
    return lib.pkvqk_paged_prefill_varlen_q8(
        FAKE, *qs, cu, q_len, total, None if cache is None else ctypes.byref(cache), FAKE, maxp,
        FAKE, B, Hq, S, 256, scale, FAKE, None, FAKE, ws, None, None)


@pytest.mark.parametrize("bad,status,word", BAD_CACHES, ids=lambda x: str(x))
def test_caches_are_refused(lib, bad, status, word):
    for call in (_append, _decode, _prefill, _varlen):
        assert call(lib, _cache(lib, **bad)) == getattr(lib, "PKVQK_ERR_" + status)
        assert word in lib.pkvqk_last_error().decode()


def test_null_cache(lib):
    for call in (_append, _decode, _prefill, _varlen):
        assert call(lib, None) == lib.PKVQK_ERR_INVALID_ARG


def test_append_arguments(lib):
    c = _cache(lib)
    for kw in (dict(T=-1), dict(Hq=0), dict(theta=0.0), dict(theta=float("inf")), dict(eps=-1.0),
               dict(qst=2047), dict(ost=2044), dict(table=-1), dict(table=(1 << 21) + 1)):
        assert _append(lib, c, **kw) == lib.PKVQK_ERR_INVALID_ARG, kw
    assert _append(lib, c, T=0) == lib.PKVQK_OK
    assert lib.pkvqk_last_error() == b""


def test_decode_arguments(lib):
    c = _cache(lib)
    for kw in (dict(B=-1), dict(q_len=0), dict(q_len=17), dict(Hq=12), dict(S=257), dict(S=-1),
               dict(maxp=0), dict(qs=(2048, 100)), dict(scale=float("nan"))):
        assert _decode(lib, c, **kw) == lib.PKVQK_ERR_INVALID_ARG, kw
    assert _decode(lib, c, S=4, ws=100) == lib.PKVQK_ERR_WORKSPACE_TOO_SMALL
    assert _decode(lib, c, S=0, ws=100) == lib.PKVQK_ERR_WORKSPACE_TOO_SMALL
    assert _decode(lib, c, B=0) == lib.PKVQK_OK


@pytest.mark.parametrize("call", [_prefill, _varlen])
def test_prefill_arguments(lib, call):
    c = _cache(lib)
    for kw in (dict(B=-1), dict(q_len=0), dict(q_len=16385), dict(Hq=12), dict(S=257), dict(S=0),
               dict(maxp=0), dict(qs=(2048, 100)), dict(scale=float("inf"))):
        assert call(lib, c, **kw) == lib.PKVQK_ERR_INVALID_ARG, kw
    assert call(lib, c, S=4, ws=100) == lib.PKVQK_ERR_WORKSPACE_TOO_SMALL
    assert call(lib, c, B=0) == lib.PKVQK_OK


def test_varlen_arguments(lib):
    c = _cache(lib)
    assert _varlen(lib, c, cu=None) == lib.PKVQK_ERR_INVALID_ARG
    assert _varlen(lib, c, total=-1) == lib.PKVQK_ERR_INVALID_ARG
    assert _varlen(lib, c, total=0) == lib.PKVQK_OK


def test_binding_refuses_mismatched_tensors(lib):
    k = torch.zeros(4, 32, 2, 128, dtype=torch.int8)
    s = torch.zeros(4, 2, 2)
    assert lib.q8_cache(k, k.clone(), s, s.clone()).format == lib.Q8_INT8
    e = k.view(torch.float8_e4m3fn)
    assert lib.q8_cache(e, e.clone(), s, s.clone()).format == lib.Q8_E4M3
    for args in ((k, e, s, s), (k.bfloat16(), k.bfloat16(), s, s), (k, k[:2], s, s),
                 (k, k, s.double(), s.double()), (k, k, s[:, :1], s[:, :1]), (k, k, s, s[:2]),
                 (k.transpose(2, 3), k.transpose(2, 3), s, s)):
        with pytest.raises(ValueError):
            lib.q8_cache(*args)


def _cpu_call(**change):
    """Arguments of an append and a decode on host tensors, some of them replaced."""
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    a = dict(q=torch.zeros(4, 4, 128, dtype=bf), k=torch.zeros(4, 2, 128, dtype=bf),
             v=torch.zeros(4, 2, 128, dtype=bf), pos=torch.zeros(4, dtype=i64),
             slots=torch.zeros(4, dtype=i64), g=torch.zeros(128, dtype=bf),
             kc=torch.zeros(4, 16, 2, 128, dtype=torch.int8), s=torch.zeros(4, 1, 2),
             table=torch.zeros(4, 4, dtype=i32), lens=torch.zeros(4, dtype=i32),
             out=torch.zeros(4, 4, 128, dtype=bf), lse=torch.zeros(4, 4), q_out=None)
    a.update(change)
    return a


def _cpu_append(lib, **change):
    a = _cpu_call(**change)
    lib.norm_rope_append_q8(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["g"], a["g"], 1e6,
                            1e-6, a["kc"], a["kc"].clone(), a["s"], a["s"].clone(),
                            q_out=a["q_out"])


def _cpu_decode(lib, **change):
    a = _cpu_call(**change)
    for f, kw in ((lib.paged_decode_q8, {}), (lib.paged_prefill_q8, dict(q_len=1))):
        f(a["q"], a["kc"], a["kc"].clone(), a["s"], a["s"].clone(), a["table"], a["lens"],
          a["out"], lse_out=a["lse"], **kw)


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(4, 4, 128)), dict(k=torch.zeros(4, 3, 128, dtype=torch.bfloat16)),
    dict(k=torch.zeros(4, 2, 256, dtype=torch.bfloat16)[..., ::2]),
    dict(v=torch.zeros(3, 2, 128, dtype=torch.bfloat16)),
    dict(pos=torch.zeros(4, dtype=torch.int32)), dict(slots=torch.zeros(3, dtype=torch.int64)),
    dict(slots=torch.zeros(8, dtype=torch.int64)[::2]), dict(g=torch.zeros(128)),
    dict(q_out=torch.zeros(4, 5, 128, dtype=torch.bfloat16))], ids=lambda c: next(iter(c)))
def test_append_binding_refuses(lib, change):
    with pytest.raises(ValueError):
        _cpu_append(lib, **change)


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(4, 4, 128)), dict(q=torch.zeros(5, 4, 128, dtype=torch.bfloat16)),
    dict(table=torch.zeros(4, 4, dtype=torch.int64)),
    dict(table=torch.zeros(3, 4, dtype=torch.int32)), dict(lens=torch.zeros(4)),
    dict(out=torch.zeros(4, 4, 128)), dict(out=torch.zeros(4, 3, 128, dtype=torch.bfloat16)),
    dict(lse=torch.zeros(4, 3)), dict(lse=torch.zeros(4, 4, dtype=torch.float64))],
    ids=lambda c: next(iter(c)))
def test_attention_binding_refuses(lib, change):
    with pytest.raises(ValueError):
        _cpu_decode(lib, **change)


def test_host_tensors_are_refused(lib):
    """Well-formed, but on the host: the library's residency check."""
    for call in (_cpu_append, _cpu_decode):
        with pytest.raises(lib.PkvqkError):
            call(lib)
