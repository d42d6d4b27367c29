"""The decoder example: training with 8-bit checkpoints lowers the loss, streaming gives what the whole sequence gives."""
import os
import sys

import pytest

from _block import need_gpu

pytestmark = pytest.mark.gpu


def test_decoder_trains_and_streams():
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import upsampling_decoder
    finally:
        sys.path.pop(0)
    losses, off = upsampling_decoder.main(steps=12)
    assert all(b < a for a, b in zip(losses[:-1:4], losses[4::4])) and losses[-1] < 0.9 * losses[0]
    # bf16 features of norm about 1, a few roundings of 2^-8 on each way
    assert off < 4 * 2.0 ** -8
