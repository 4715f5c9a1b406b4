"""The FP8 operand of the binding: its descriptor and its fields cannot part."""
import pytest
import torch

import microscaling_fp4_quantized_block_amd as mx


def test_fields_that_the_descriptor_holds_cannot_be_reassigned():
    """The library reads the descriptor's addresses and sizes: a field that was set to another tensor
    or size would be ignored, and the memory it replaced read after it is freed."""
    q = mx.empty_fp8(5, 300, "cpu", pair=2)
    assert (q.rows, q.k, q.pair, q.device.type) == (5, 300, 2, "cpu")
    assert q.codes.shape == (5, 384) and q.scales.shape == (3, 16)
    assert q._struct.codes == q.codes.data_ptr() and q._struct.scales == q.scales.data_ptr()
    for name, value in (("codes", torch.zeros_like(q.codes)), ("scales", torch.zeros_like(q.scales)), ("rows", 4),
                        ("k", 128), ("device", torch.device("cpu"))):
        with pytest.raises(AttributeError):
            setattr(q, name, value)
    q.codes.fill_(7)   # (their contents may)
    assert int(q.codes[4, 383]) == 7 and q._struct.codes == q.codes.data_ptr()
    q.pair = None      # (which the descriptor does not hold)
    assert q.pair is None
