"""Strides at the end of their range, without a GPU: every call here carries a
null pointer, which is refused right after the strides."""
import ctypes

import pytest

import block_quantized_int8_q8_amd as mmq

p = ctypes.c_void_p


def rope(T, H, D, odt, odh):
    return mmq.lib().mmq_rope(0, None, H * D, D, 0, None, odt, odh, p(1 << 20), p(1 << 20), 8, 0, 1.0, 0, T, H, D, None)


@pytest.mark.parametrize("T,H,odt,odh,why", [
    (1 << 24, 2, 1 << 40, 0, "overlap"), (1 << 24, 2, 1 << 40, 7, "overlap"), ((1 << 23) + 1, 1024, 1 << 40, 4, "overlap"),
    (1 << 24, 1024, 1 << 40, 8, "null"), (1 << 24, 1024, 1 << 40, 1 << 30, "null"), (1 << 24, 1024, 8, 1 << 27, "null"),
    (1 << 24, 1024, 8, (1 << 27) - 1, "overlap"), (1 << 24, 1024, 9, 1 << 40, "null"), (1 << 24, 1, 1 << 40, 0, "null"),
    (1, 1024, 0, 1 << 40, "null")])
def test_largest_strides_of_an_output(T, H, odt, odh, why):
    assert rope(T, H, 8, odt, odh) == 0
    assert why in mmq.last_error(), mmq.last_error()


def test_no_tokens_have_no_places():
    for odt, odh in ((16, 8), (8, 0), (0, 0)):
        assert rope(0, 2, 8, odt, odh) == 1
