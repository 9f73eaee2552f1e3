"""The binding of the rotary, cache and attention calls, without a GPU."""
import torch

import block_quantized_int8_q8_amd as mmq


def test_frequencies_are_on_the_host_whatever_the_default_device():
    want, m = mmq.rope_frequencies(64, base=1e6, scaling="yarn", factor=4.0, original=8192)
    with torch.device("meta"):
        got, again = mmq.rope_frequencies(64, base=1e6, scaling="yarn", factor=4.0, original=8192)
    assert got.device.type == "cpu" and torch.equal(got, want) and again == m
