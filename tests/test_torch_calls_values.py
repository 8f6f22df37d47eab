"""Numbers that the native part of the binding refuses (no GPU needed): 0 leaves the cap out and
asks for the default scale, so a value that fp32 only has as 0 must not become it.
"""

import pytest

from tests.test_torch_calls import _decode, _varlen, lib  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("name", ["softcap", "scale"])
@pytest.mark.parametrize("value", [1e-46, -1e-60, 5e-324])
def test_values_below_fp32(lib, name, value):  # noqa: F811
    for f, args in ((lib.paged_decode_scored, _decode()), (lib.paged_prefill_scored, _decode()),
                    (lib.paged_prefill_varlen_scored, _varlen())):
        with pytest.raises(ValueError, match=name):
            f(**(args | {name: value}))


@pytest.mark.parametrize("name,value", [("softcap", 0), ("softcap", -0.0), ("scale", 0.0),
                                        ("scale", 1e-40), ("softcap", 30)])
def test_values_that_are_taken(lib, name, value):  # noqa: F811
    with pytest.raises(lib.PkvqkError, match="device memory|cudaPointerGetAttributes"):
        lib.paged_decode_scored(**(_decode() | {name: value}))


@pytest.mark.parametrize("value", [1e-9, 2.0 ** 21, float("nan"), float("inf"), -1.0, 1e300])
def test_caps_that_the_entry_refuses(lib, value):  # noqa: F811
    with pytest.raises(lib.PkvqkError, match="softcap"):
        lib.paged_decode_scored(**(_decode() | dict(softcap=value)))
