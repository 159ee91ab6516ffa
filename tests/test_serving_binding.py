"""The Python side of the serving calls, as far as it needs no GPU."""

import types

import pytest
import torch

import block_sparse_attention_48_b200 as fa


@pytest.mark.parametrize("name", ["rope_apply", "paged_append", "flex_decode_paged", "flex_decode_shared"])
def test_stream_of_another_device(name):
    """stream= looks at the first tensor, whether it is given by place or by name."""
    fn, first = getattr(fa, name), "k" if name == "paged_append" else "q"
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(x, stream=stream)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(**{first: x}, stream=stream)
    for bad in ({}, {first: None}, {first: [1.0]}):
        with pytest.raises(TypeError, match=first):
            fn(**bad, stream=stream)
