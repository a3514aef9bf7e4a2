"""pkv_extend and pkv_extend_q8 on the GPU where test_gpu_extend.py does not look.  Its tolerances, unless a test says
otherwise."""
import math

import pytest
import torch

from paged_kv_decode_block_gb300 import pkv
from test_gpu_extend import BOTH, FP8, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load()


def slots(p, b, n):
    """Where the pools hold the first n tokens of row b."""
    t = torch.arange(n, device="cuda")
    return p.table[b].long()[t // p.ps] * p.ps + t % p.ps


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -120, -2.0 ** -120, 2.0 ** -149, 2.0 ** -22])
def test_queries_and_keys_of_next_to_nothing(scale, D):
    """8-bit: the product of a query's factor and a scale of K may be too small for fp32; places that a row does not see
    stay out all the same, so that a query of zeros answers the mean of V and the logarithm of the tokens it sees."""
    p = Problem([200, 0, 37, 3], [70, 13, 1, 300], q8=True, Hq=4, Hkv=2, D=D)
    p.ks.fill_(scale)
    for size in (0.0, 2.0 ** -110, 2.0 ** -60):
        p.q.copy_((torch.randn(p.q.shape, generator=p.gen, device="cuda") * size).bfloat16())
        p.run().check()
        if size == 0.0:
            seen = torch.cat([torch.arange(n + 1, n + a + 1, device="cuda") for n, a in zip(p.lens, p.new)])
            assert (p.lse - seen.log()[:, None]).abs().max().item() <= 1e-4
    p.k.view(torch.uint8).zero_()   # an append's scale of a block of zeros is 2^-120
    p.q.zero_()
    p.run().check()
