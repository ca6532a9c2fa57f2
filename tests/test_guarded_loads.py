"""Loads of 16-bit elements that stand under a condition.  CUDA's __ldg of
__half and __nv_bfloat16 is an assembly statement without `volatile`, which the
compiler may execute ahead of the condition; a row's bound then guards nothing.
So the types through which kernels read 16-bit elements load them plainly."""
import os
import re

import pytest

from fft_long_convolution_flashconv_b200 import build


@pytest.mark.parametrize("name", ["__half", "__nv_bfloat16"])
@pytest.mark.parametrize("head,file", [("struct IO<%s>", "common.cuh"), ("struct UPair<%s>", "fftconv_impl.cuh")])
def test_16_bit_elements_are_loaded_plainly(name, head, file):
    with open(os.path.join(build.CSRC, file)) as fh:
        txt = re.sub(r"//[^\n]*", "", fh.read())
    body = txt[txt.index(head % name):]
    body = body[:body.index("\n};")]
    assert " ld(" in body or " load(" in body
    assert "__ldg" not in body
