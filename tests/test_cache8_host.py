"""The 8-bit cache and the rotated append without a GPU: the oracle's definitions
against torch's float8 and float64 arithmetic, pkv_rotary_init, and every
refusal that needs no device."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cache8
from paged_kv_decode_block_gb300 import pkv


def test_e4m3_table_is_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.E4M3, want, equal_nan=True)


def test_e4m3_encode_is_torchs_rounding():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000), cache8.E4M3[:0x7F],
                        (cache8.E4M3[:0x7E] + cache8.E4M3[1:0x7F]) / 2, [0.0, -0.0]])   # ties too
    x = x.astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(cache8.e4m3_encode(x), want)
    assert cache8.e4m3_encode([np.nan, np.inf])[0] & 0x7F == 0x7F
    assert cache8.e4m3_encode([np.inf])[0] & 0x7F == 0x7F


def test_block_scale_by_hand():
    got = cache8.block_scale(np.array([448.0, 448.1, 896.0, 1.0, 0.875, 0.0, 3e38]))
    # 1 / 448 = 2^-8.8: 2^-8; 0.875 = 448 * 2^-9 exactly
    assert got.tolist() == [1.0, 2.0, 2.0, 2.0 ** -8, 2.0 ** -9, 2.0 ** -120, 2.0 ** 120]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64))
    pos = np.array([0, 1, 7, 1000, 123456])
    freq = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    y = cache8.rotate(x, pos, freq, interleaved, 1.5)
    f, s = (np.s_[..., 0:32:2], np.s_[..., 1:32:2]) if interleaved else (np.s_[..., :16], np.s_[..., 16:32])
    z = (x[f] + 1j * x[s]) * 1.5 * np.exp(1j * pos[:, None] * freq)[:, None]
    assert np.allclose(y[f], z.real, atol=1e-12) and np.allclose(y[s], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_decode_oracle_is_torchs_attention_in_float64():
    rng = np.random.default_rng(3)
    H, G, D, ps, n = 2, 4, 64, 32, 75
    codes = [rng.integers(0, 256, (8, ps, H, D)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0
    scales = [(rng.random((8, ps // 16, H)) * 0.01).astype(np.float32) for _ in range(2)]
    table = np.array([[5, 0, 3, -1]], np.int32)
    q = rng.standard_normal((1, H * G, D))
    out, lse = cache8.decode_q8(q, *codes, *scales, table, [n])
    dense = [torch.from_numpy((cache8.E4M3[c] * np.repeat(s, 16, 1)[..., None])[table[0, :3]].reshape(-1, H, D)[:n])
             for c, s in zip(codes, scales)]
    k, v = (x.permute(1, 0, 2).repeat_interleave(G, 0) for x in dense)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[0])[:, None], k, v)[:, 0]
    assert np.allclose(out[0], want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse[0], torch.logsumexp((torch.from_numpy(q[0])[:, None] @ k.mT)[:, 0] / 8, -1).numpy())


def test_append_oracle_by_hand():
    """Two tokens into a block that holds one: the old code 1.0 at scale 2^-2 moves to scale 1 as 0.25."""
    codes = np.zeros((1, 16, 1, 1), np.uint8)
    codes[0, 0] = cache8.e4m3_encode(1.0)
    scales = np.full((1, 1, 1), 0.25)
    x = np.array([300.0, -448.0]).reshape(2, 1, 1)
    c, s, _ = cache8.append_q8(x, codes, scales, np.array([[0]]), [1], [2], 16)
    assert s.item() == 1.0
    assert cache8.E4M3[c[0, :3, 0, 0]].tolist() == [0.25, 288.0, -448.0]   # 300: between 288 and 320
    # and from the block's start the old content has no say
    c, s, _ = cache8.append_q8(x / 1024, codes, scales, np.array([[0]]), [0], [2], 16)
    assert s.item() == 2.0 ** -10


def test_rotary_steps():
    freq = np.array([1.0, 0.5, 2 * np.pi, -1.0, 0.0, 1e-6, 7.0, 100.0])
    r = pkv.Rotary(16, inv_freq=freq, interleaved=True, scale=0.5).params
    assert (r.dim, r.interleaved, r.scale) == (16, 1, 0.5)
    turns = np.array([r.step[m] for m in range(8)], np.float64) / 2.0 ** 64
    want = np.mod(freq / (2 * np.pi), 1.0)
    assert np.all(np.abs((turns - want + 0.5) % 1.0 - 0.5) < 2.0 ** -48)
    # the default frequencies
    r = pkv.Rotary(64, base=500000.0).params
    assert np.isclose(r.step[31] / 2.0 ** 64 * 2 * np.pi, 500000.0 ** (-62 / 64), rtol=1e-14)


@pytest.mark.parametrize("dim, interleaved, scale, freq", [
    (0, 0, 1.0, 1.0), (8, 0, 1.0, 1.0), (24, 0, 1.0, 1.0), (144, 0, 1.0, 1.0), (-16, 0, 1.0, 1.0), (16, 2, 1.0, 1.0),
    (16, -1, 1.0, 1.0), (16, 0, float("nan"), 1.0), (16, 0, 1.0, float("inf")), (16, 0, 1.0, float("nan"))])
def test_rotary_refusals(dim, interleaved, scale, freq):
    f = (ctypes.c_double * 128)(*[freq] * 128)
    r = pkv.RotaryParams()
    r.dim = 77
    assert pkv.load().pkv_rotary_init(f, dim, interleaved, scale, ctypes.byref(r)) == pkv.EINVAL
    assert r.dim == 77   # left as it was
    assert pkv.load().pkv_rotary_init(None, 16, 0, 1.0, ctypes.byref(r)) == pkv.EINVAL
    assert pkv.load().pkv_rotary_init(f, 16, 0, 1.0, None) == pkv.EINVAL


def test_rotary_shape_check():
    with pytest.raises(ValueError):
        pkv.Rotary(32, inv_freq=np.ones(8))
    with pytest.raises(pkv.PkvError):
        pkv.Rotary(24)


def test_struct_layouts_match_the_header(tmp_path):
    """pkv_rotary and pkv_tokens as the C compiler lays them out, against the binding's."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = []
    for name, cls in (("pkv_rotary", pkv.RotaryParams), ("pkv_tokens", pkv.Tokens)):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in (pkv.RotaryParams, pkv.Tokens):
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want
    assert pkv.ROTARY_MAX_DIM == 128 and pkv.Q8_BLOCK == cache8.BLOCK


def test_calls_without_a_plan_are_refused():
    lib = pkv.load()
    t = pkv.Tokens()
    assert lib.pkv_append_rotary(ctypes.byref(t), None, None, None, None, None, None, None, None) == pkv.EINVAL
    assert lib.pkv_append_q8(ctypes.byref(t), None, None, None, None, None, None, None, None, None, None) == pkv.EINVAL
    assert lib.pkv_decode_q8(None, None, None, None, None, None, None, None, None, None, None) == pkv.EINVAL


def test_cpu_tensors_are_refused():
    class FakePlan:   # the checks come before the plan is used
        geom = pkv.Geom(1, 4, 1, 64, 4, 8)
        page_size, D, Hq, Hkv, handle, device = 16, 64, 4, 1, None, 0
        pool_shape, scales_shape, table_shape, rows_shape = (8, 16, 1, 64), (8, 1, 1), (1, 4), (1,)
        out_shape, lse_shape = (1, 4, 64), (1, 4)
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    pages = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.append_rotary(k, k, pages, pages, torch.zeros(1, 4, dtype=torch.int32), i, i.clone(), FakePlan, None)
    with pytest.raises(TypeError):
        pkv.append_q8(None, k, pages, pages, None, None, torch.zeros(1, 4, dtype=torch.int32), i, i.clone(), FakePlan)
    with pytest.raises(TypeError):
        pkv.decode_q8(torch.zeros(1, 4, 64, dtype=torch.bfloat16), pages, pages, i, i, torch.zeros(1, 4, dtype=torch.int32),
                      i, FakePlan, k, k)
