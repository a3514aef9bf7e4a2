"""pkv_append_q8 and pkv_decode_q8 on the GPU where test_gpu_cache8.py does not look: calls that follow one another with
nothing between them.

Tolerances: as in test_gpu_cache8.py.
"""
import numpy as np
import pytest
import torch

from oracle import cache8
from paged_kv_decode_block_gb300 import pkv
from test_gpu_cache8 import Cache, New, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load()


# ------------------------------------------------------------------ calls back to back

@pytest.mark.parametrize("route", ["direct", "split_padded"])
@pytest.mark.parametrize("B, H, G, D", [(1, 8, 4, 128), (3, 4, 8, 64), (16, 8, 1, 128)])
def test_append_and_decode_back_to_back(B, H, G, D, route):
    """Forty steps enqueued behind a busy GPU, so that each decode's CTAs are there before the append has written: every
    step turns the queries, raises the scales of blocks that are being filled, and is compared with the oracle over the
    cache as it was after that step.  Grids of at most one CTA an SM: the append lets the decode in early."""
    rng = np.random.default_rng(B)
    steps = 40
    lens = rng.integers(1, 200, B)
    c = Cache(lens, Hq=G * H, H=H, D=D, seed=90 + B, room=steps)
    r = pkv.Rotary(64)
    news = [New(c, [1] * B, offsets=False, seed=100 + i, size=1.02 ** i * (1 + i % 7)) for i in range(steps)]
    outs = [torch.full((B, G * H, D), 7.0, device="cuda") for _ in range(steps)]
    lses = [torch.full((B, G * H), 7.0, device="cuda") for _ in range(steps)]

    def start():
        d = c.upload()
        plan = pkv.Plan(lens + steps, None, 16, B=B, Hq=G * H, Hkv=H, D=D, max_pages=c.table.shape[1],
                        num_pages=c.pages, force_mode=route, num_splits=0 if route == "direct" else 3)
        buf = [d["lens"], torch.empty_like(d["lens"])]
        # the plan goes to the device now, not between the calls
        pkv.decode_q8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["lens"], plan, d["out"], d["lse"])
        torch.cuda.synchronize()
        return d, plan, buf

    def append(i, d, plan, buf):
        x = news[i]
        pkv.append_q8(x.kd, x.vd, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], buf[i % 2], buf[1 - i % 2], plan, r,
                      q=x.qd, q_out=x.q_out)

    d, plan, buf = start()
    torch.cuda._sleep(20_000_000)   # some 10 ms, in which all calls are enqueued
    for i in range(steps):
        append(i, d, plan, buf)
        pkv.decode_q8(news[i].q_out, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], buf[1 - i % 2], plan, outs[i], lses[i])
    torch.cuda.synchronize()
    assert plan.status() == 0
    turned = [bits(x.q_out) for x in news]

    d, plan, buf = start()   # once more, step by step, for the cache that each decode has read
    for i in range(steps):
        append(i, d, plan, buf)
        torch.cuda.synchronize()
        assert np.array_equal(bits(news[i].q_out), turned[i])
        c.kc, c.vc = (d[x].view(torch.uint8).cpu().numpy() for x in ("kp", "vp"))
        c.ks, c.vs = (d[x].cpu().numpy() for x in ("ks", "vs"))
        c.lens, c.q = (lens + i + 1).astype(np.int32), turned[i]
        d["out"], d["lse"] = outs[i], lses[i]
        c.check(what=f"step {i}")
