"""What the calls of the rotated append and the 8-bit cache refuse or derive on the host, without a GPU."""
import pytest
import torch

from paged_kv_decode_block_gb300 import pkv


# ------------------------------------------------------------------ token tensors

def tokens_arg(t, shape):
    pkv._bf16_types()
    return pkv._tokens_arg(t, "k_new", shape, -1)   # (a CPU tensor's device index; the checks are the same)


@pytest.mark.parametrize("T, heads, D", [(4, 2, 64), (2, 1, 64), (300, 8, 128)])
def test_broadcast_tokens_are_refused(T, heads, D):
    """A tensor expanded over its tokens has a distance of 0 between them, which the C call reads as "dense": T tokens
    would be read, or written, where one lies."""
    one = torch.zeros(1, heads, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tokens_arg(one.expand(T, heads, D), (T, heads, D))
    with pytest.raises(ValueError):
        tokens_arg(torch.zeros(heads, D, dtype=torch.bfloat16).expand(T, heads, D), (T, heads, D))
    if heads > 1:   # nor over the heads
        with pytest.raises(ValueError):
            tokens_arg(torch.zeros(T, 1, D, dtype=torch.bfloat16).expand(T, heads, D), (T, heads, D))


def test_token_strides():
    """Dense tensors, slices of a projection, every other token, and single tokens however they lie."""
    x = torch.zeros(6, 10, 64, dtype=torch.bfloat16)
    for t, stride in ((x, 640), (x[:, 2:4], 640), (x[::2], 1280), (x[:, 3:4], 640), (x[:1], 0), (x[4:5, 7:9], 0),
                      (x[:1].expand(1, 10, 64), 0)):
        assert tokens_arg(t, tuple(t.shape)) == (t.data_ptr(), stride)
    assert tokens_arg(x[:0], (0, 10, 64)) == (0, 0)
