"""What the calls of the rotated append and the 8-bit cache refuse or derive on the host, without a GPU."""
import ctypes
from fractions import Fraction

import numpy as np
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


# ------------------------------------------------------------------ angles

def turns_of(freq):
    """freq / 2 pi modulo 1 as a fraction, 1 / 2 pi to 400 bits by Machin's formula in integers."""
    bits = 420
    one = 1 << bits

    def arctan_inverse(x):
        term = total = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return Fraction(freq) * Fraction(one, 2 * pi) % 1


@pytest.mark.parametrize("base, dim", [(10000.0, 128), (500000.0, 64), (1e6, 16)])
def test_rotary_steps_to_a_unit_of_the_last_place(base, dim):
    """The angle of a step off by one unit, 2^-64 turns, is off by 2^-33 turns at position 2^31."""
    got = pkv.Rotary(dim, base=base).params
    for m, f in enumerate(base ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)):
        off = (got.step[m] - turns_of(float(f)) * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, m


def test_rotary_steps_of_any_frequency():
    rng = np.random.default_rng(1)
    freq = np.concatenate([rng.uniform(-10, 10, 100), 2.0 ** rng.uniform(-70, 40, 100), -2.0 ** rng.uniform(-70, 40, 100),
                           [0.0, -0.0, 2.0 ** -1074, -2.0 ** -64, 2 * np.pi, 2.0 ** 40, 1e300, -1e300, 1.7e308, 2.0 ** 62]])
    for i in range(0, len(freq) - 8, 8):
        got = pkv.Rotary(16, inv_freq=freq[i:i + 8]).params
        for m in range(8):
            if abs(freq[i + m]) > 2.0 ** 40:   # finite: taken, its angle says nothing
                continue
            off = (got.step[m] - turns_of(float(freq[i + m])) * 2 ** 64) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= 1, freq[i + m]
    for f in freq[-10:]:
        up, down = (pkv.Rotary(16, inv_freq=np.full(8, x)).params.step[0] for x in (f, -f))
        assert (up + down) % 2 ** 64 == 0   # the other way round


# ------------------------------------------------------------------ devices

def test_a_plan_names_its_own_device(monkeypatch):
    """The device that tensors are checked against is the one the library bound the plan to, whatever torch, which may
    not even be imported when the plan is made, holds for current."""
    class Library:
        def pkv_plan(self, lens, table, page_size, geom, opts, handle):
            handle._obj.value = 1
            return pkv.OK

        def pkv_plan_device(self, handle, device):
            device._obj.value = 3
            return pkv.OK

        def pkv_plan_destroy(self, handle):
            pass
    monkeypatch.setattr(pkv, "_lib", Library())
    plan = pkv.Plan([1], None, 16, B=1, Hq=4, Hkv=1, D=64, max_pages=1, num_pages=1)
    device = plan.device
    plan.close()
    assert device == 3


def test_plan_device_refuses_null():
    device = ctypes.c_int32(7)
    assert pkv.load().pkv_plan_device(None, ctypes.byref(device)) == pkv.EINVAL and device.value == 7
