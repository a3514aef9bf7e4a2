"""pkv_append_q8 and pkv_decode_q8 on the GPU where test_gpu_cache8.py does not look: calls that follow one another with
nothing between them, weights and V scales far apart,
values next to the middles between two codes.

Tolerances are derived at the tests; two come from test_gpu_cache8.py:
* Rotation: the angle is cut to 2^-32 turns (2^-29 rad) and rounded to fp32 twice, by 2^-25 of at most pi / 4 each; the
  first terms that the series of sin and cos leave out are below 2^-28 and their evaluation rounds a few times by 2^-25;
  factor, products and sum add three roundings of 2^-24: |error| <= 2^-20 (|x| + |y|) scale covers it.
* Attention: exact inputs, fp32 dot products and sums.  A score is off by at most
  d = (D + 16) 2^-23 max_t sum_d |q_d k_td| / sqrt(D); a weight by a factor of 2 d and about 2^-20 (exp2, the f16 split,
  the reference's product), the sum of n weights by n 2^-23.
"""
import numpy as np
import pytest
import torch

from oracle import cache8
from paged_kv_decode_block_gb300 import pkv
from test_gpu_cache8 import Cache, New, bf16, bits, on_gpu, rotary_of

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


@pytest.mark.parametrize("route", ["direct", "split_padded"])
@pytest.mark.parametrize("copy", ["tma", "lsu"])
@pytest.mark.parametrize("B, H, G, D", [(1, 8, 4, 128), (16, 4, 8, 64)])
def test_rotated_append_and_bf16_decode_back_to_back(B, H, G, D, copy, route):
    """The same into bf16 pages, read by pkv_decode with either copy engine: the bits of a run that waits after each
    call, and the oracle's values at the last step."""
    rng = np.random.default_rng(B)
    steps = 40
    lens = rng.integers(1, 200, B)
    c = Cache(lens, Hq=G * H, H=H, D=D, seed=140 + B, room=steps)
    d = c.upload()
    kv = [bf16(rng.standard_normal((c.pages, 16, H, D))) for _ in range(2)]
    r = pkv.Rotary(64)
    news = [New(c, [1] * B, offsets=False, seed=150 + i) for i in range(steps)]

    def run(wait):
        kp, vp = (on_gpu(x) for x in kv)
        buf = [torch.from_numpy(c.lens.copy()).cuda(), torch.empty(B, dtype=torch.int32, device="cuda")]
        plan = pkv.Plan(lens + steps, None, 16, B=B, Hq=G * H, Hkv=H, D=D, max_pages=c.table.shape[1], copy=copy,
                        num_pages=c.pages, force_mode=route, num_splits=0 if route == "direct" else 3)
        outs = torch.full((steps, B, G * H, D), 7.0, device="cuda")
        lses = torch.full((steps, B, G * H), 7.0, device="cuda")
        pkv.decode(d["q"], kp, vp, d["table"], buf[0], plan, outs[0], lses[0])   # the plan goes to the device now
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for i, x in enumerate(news):
            pkv.append_rotary(x.kd, x.vd, kp, vp, d["table"], buf[i % 2], buf[1 - i % 2], plan, r, q=x.qd, q_out=x.q_out)
            if wait:
                torch.cuda.synchronize()
            pkv.decode(x.q_out, kp, vp, d["table"], buf[1 - i % 2], plan, outs[i], lses[i])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert plan.status() == 0
        return outs, lses, kp, vp

    apart, at_once = run(True), run(False)
    for a, b in zip(apart, at_once):
        assert torch.equal(a, b)
    import oracle
    outs, lses, kp, vp = at_once
    ref = oracle.decode(bits(news[-1].q_out), bits(kp), bits(vp), c.table, (lens + steps).astype(np.int32))
    assert np.max(np.abs(outs[-1].cpu().numpy() - ref[0])) <= 2e-3   # pkv_decode's own tolerances
    assert np.max(np.abs(lses[-1].cpu().numpy() - ref[1])) <= 1e-4


# ------------------------------------------------------------------ weights and V scales far apart

def check_by_terms(c, what=""):
    """out against the oracle, each element by the sum of its own terms: |error| <= F sum_t p_t |v_t| with the factor F
    of Cache.bounds (scores of the tokens that weigh anything, weights, sums; once for the numerator and once for the
    denominator), and for each token at most half a step of the least weight kept, 2^-42 of the row's largest weight times V scale, times a code of 448."""
    torch.cuda.synchronize()
    q = cache8.bf16_to_f64(c.q)
    out, lse = c.d["out"].cpu().numpy().astype(np.float64), c.d["lse"].cpu().numpy()
    G = c.Hq // c.H
    for b in range(c.B):
        n = int(c.lens[b])
        rows = cache8.places(c.table, b, 0, n, c.ps)
        for h in range(c.H):
            ks, vs = (s.reshape(-1, c.H).astype(np.float64)[rows // 16, h][:, None] for s in (c.ks, c.vs))
            k, v = (cache8.E4M3[x.reshape(-1, c.H, c.D)[rows, h]] * s for x, s in ((c.kc, ks), (c.vc, vs)))
            s = q[b, h * G:(h + 1) * G] @ k.T / np.sqrt(c.D)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            dot = (np.abs(q[b, h * G:(h + 1) * G]) @ np.abs(k).T)[p >= 2.0 ** -126].max() / np.sqrt(c.D)
            f = 2 * (c.D + 16) * 2.0 ** -23 * dot + (n + 64) * 2.0 ** -23 + 2.0 ** -20
            want, size = p @ v / total, p @ np.abs(v) / total
            least = n * 448 * 2.0 ** -42 * (p * np.abs(vs).T).max(1, keepdims=True) / total
            off = np.abs(out[b, h * G:(h + 1) * G] - want)
            limit = 2 * f * size + least
            assert np.all(off <= limit), (what, b, h, np.max(off / np.maximum(limit, 1e-300)))
            ref = (m + np.log(total))[:, 0]
            assert np.all(np.abs(lse[b, h * G:(h + 1) * G] - ref) <= f * np.maximum(1, np.abs(ref))), (what, b, h)


@pytest.mark.parametrize("D, G", [(64, 1), (64, 8), (128, 2), (128, 4), (128, 8)])
@pytest.mark.parametrize("k", [12, 20, 30, 36, 44, 80, 120])
@pytest.mark.parametrize("first", [True, False])
def test_decode_heavy_token_in_a_block_of_small_scale(D, G, k, first):
    """One key far above the others, in a block whose V scale is 2^-k of the others', before or behind them in the same
    warp's blocks (0 and 8): the others weigh nothing (e^-1000), and out is that token's V: its weight times scale split
    to 22 bits, one rounding where the parts meet, the division by its weight and its rounding, 2^-21 in all."""
    c = Cache([144], Hq=G, H=1, D=D, seed=200 + k)
    rows = cache8.places(c.table, 0, 0, 144, 16)
    c.kc[:] = 0
    q = cache8.bf16_to_f64(c.q)[0]
    c.q = bf16(np.broadcast_to(q[:1], (1, G, D)))
    heavy = rows[3] if first else rows[8 * 16 + 3]
    c.kc.reshape(-1, 1, D)[heavy, 0] = cache8.e4m3_encode(np.sign(q[0]) * 448)
    c.ks[:] = 1.0   # the heavy token's score: 448 sum |q| / sqrt(D), over 1000
    c.vs[:] = 1.0
    c.vs.reshape(-1)[heavy // 16] = 2.0 ** -k
    c.upload()
    for route in ("direct", "persistent"):
        c.d["out"].fill_(7.0)
        c.decode(c.plan(force_mode=route))
        torch.cuda.synchronize()
        want = cache8.E4M3[c.vc.reshape(-1, D)[heavy]] * 2.0 ** -k
        got = c.d["out"].cpu().numpy().astype(np.float64)[0]
        assert np.all(np.abs(got - want) <= 2.0 ** -20 * np.abs(want)), (route, np.max(np.abs(got - want)) * 2.0 ** k)


@pytest.mark.parametrize("D, G, n", [(64, 4, 700), (128, 4, 700), (128, 8, 300), (64, 1, 3000), (128, 2, 6000)])
@pytest.mark.parametrize("seed", [1, 2])
def test_decode_scales_against_weights(D, G, n, seed):
    """Blocks whose V scales, from 2^-55 to 2^55, undo their tokens' weights up to a factor of 2^12, in a random order:
    every block adds to the output, the heavy ones to the sum, and both references move again and again.  6000 tokens
    of D = 128 and 3000 of D = 64 (one tile) take the loop that reduces two blocks a turn."""
    rng = np.random.default_rng(300 + seed)
    c = Cache([n], Hq=G, H=1, D=D, seed=310 + seed)
    rows = cache8.places(c.table, 0, 0, n, 16)
    blk = rows[::16] // 16
    c.q = bf16(np.full((1, G, D), 0.5))
    power = rng.uniform(-55, 55, len(blk))
    c.kc[:] = 0
    c.kc.reshape(-1, 1, D)[rows, 0, 0] = cache8.e4m3_encode(rng.uniform(240, 272, n))
    # a score of -power ln 2 at a code of 256 (and up to 1/16 of it more or less)
    c.ks.reshape(-1)[blk] = -power * np.log(2.0) * np.sqrt(D) / 128
    c.vs.reshape(-1)[blk] = 2.0 ** np.round(power + rng.uniform(-6, 6, len(blk)))
    c.upload()
    for route, splits in (("direct", 0), ("split_queue", 3)):
        c.d["out"].fill_(7.0)
        c.decode(c.plan(force_mode=route, num_splits=splits))
        check_by_terms(c, route)


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -149, 2.0 ** 110, -2.0 ** 100])
def test_decode_blocks_of_extreme_scale_that_weigh_nothing(scale):
    """Blocks of extreme V scale before (every warp's first), between and behind ordinary ones, with scores so low that
    their weights are zero: the output is the ordinary ones'."""
    c = Cache([800], Hq=8, H=2, D=128, seed=320)
    rows = cache8.places(c.table, 0, 0, 800, 16)
    q = cache8.bf16_to_f64(c.q)[0]
    c.q = bf16(np.broadcast_to(q[:1], (1, 8, 128)))
    for i in np.r_[0:9, 20:24, 45:50]:
        at = rows[16 * i:16 * i + 16]
        c.kc.reshape(-1, 2, 128)[at] = cache8.e4m3_encode(np.sign(q[0]) * -448)
        c.ks.reshape(-1, 2)[at[0] // 16] = 1.0
        c.vs.reshape(-1, 2)[at[0] // 16] = scale
    c.upload()
    c.decode(c.plan(force_mode="direct"))
    check_by_terms(c)


@pytest.mark.parametrize("route, splits", [("direct", 0), ("split_queue", 3), ("persistent", 0)])
def test_decode_values_near_the_largest_float(route, splits):
    """V values up to 448 * 2^118, which is 2^126.8: sums of weights times values pass the largest float where the
    output does not."""
    c = Cache([500, 3, 33], Hq=8, H=2, D=64, seed=330)
    c.vs[:] = 2.0 ** 118
    c.upload()
    c.decode(c.plan(force_mode=route, num_splits=splits))
    check_by_terms(c)


@pytest.mark.parametrize("route, splits", [("direct", 0), ("split_queue", 3), ("persistent", 0)])
def test_decode_scores_of_minus_infinity(route, splits):
    """Scores past the least float, in every warp's first blocks: those tokens weigh nothing; a row of nothing else has
    no weight at all, as an empty row."""
    c = Cache([500, 500, 40, 40], Hq=4, H=1, D=64, seed=331)
    q = cache8.bf16_to_f64(c.q)
    c.q = bf16(np.broadcast_to(np.sign(q[:, :1]) * 2.0 ** 60, q.shape))
    kc, ks = c.kc.reshape(-1, 1, 64), c.ks.reshape(-1)
    c.ks *= np.float32(2.0 ** -60)
    for b, blocks in ((0, range(8)), (1, range(3, 32)), (2, range(1)), (3, range(3))):
        for i in blocks:
            at = cache8.places(c.table, b, 16 * i, 16 * i + 16, 16)
            kc[at] = cache8.e4m3_encode(np.sign(q[b, 0]) * -448)
            ks[at[0] // 16] = 2.0 ** 100   # scores of -2^60 448 64 2^100 / 8
    c.upload()
    c.decode(c.plan(force_mode=route, num_splits=splits))
    torch.cuda.synchronize()
    assert (c.d["out"][3] == 0).all() and torch.isneginf(c.d["lse"][3]).all()
    c.lens[3] = 0   # (in 64 bits its scores are finite)
    live = c.d["out"].clone(), c.d["lse"].clone()
    c.B, c.d["out"], c.d["lse"] = 3, live[0][:3], live[1][:3]
    check_by_terms(c)


# ------------------------------------------------------------------ codes at scales that are no powers of two

def nearest_codes(c, n, turn, before):
    """Every code of the written slots is a nearest one: of exact values (V, and K without rotation) the oracle's own,
    ties included; of a rotated key at most the rotation's error (see test_gpu_cache8.py) further off than it."""
    d = c.d
    for x, codes, scales, pages, sc, exact in (
            (turn(cache8.bf16_to_f64(n.k), n.pos), before[0], before[1], "kp", "ks", turn is not_turned),
            (cache8.bf16_to_f64(n.v), before[2], before[3], "vp", "vs", True)):
        wc, ws, want = cache8.append_q8(x, codes, scales, c.table, c.lens, n.counts, c.ps)
        assert np.array_equal(d[sc].cpu().numpy().astype(np.float64), ws)
        got, wc = d[pages].view(torch.uint8).cpu().numpy().reshape(want.shape), wc.reshape(want.shape)
        written = ~np.isnan(want)
        assert np.array_equal(got[~written], codes.reshape(want.shape)[~written])
        if exact:
            assert np.array_equal(got[written], wc[written]), np.mean(got[written] != wc[written])
        else:
            slop = 2.0 ** -20 * 2 * np.abs(cache8.bf16_to_f64(n.k)).max() / np.repeat(ws.reshape(-1, c.H), 16, 0)[..., None]
            off, least = np.abs(cache8.E4M3[got] - want), np.abs(cache8.E4M3[wc] - want)
            assert np.all(off[written] <= (least + 2 * slop)[written])


def not_turned(x, pos):
    return cache8.rotate(x, pos, [])


@pytest.mark.parametrize("scale", [7.0, 0.3, 1 / 448, 100 / 3])
def test_append_rounds_ties_at_any_held_scale(scale):
    """Values at and next to the middles between two codes, in units of a scale that the block's tokens hold (e4m3's
    middles have five significant bits; times 7 they are bf16 values)."""
    c = Cache([3, 20, 9], Hq=2, H=1, D=64, seed=400, room=16)
    c.ks[:] = c.vs[:] = np.float32(scale)
    c.upload()
    n = New(c, [12, 5, 7], seed=401)
    rng = np.random.default_rng(402)
    middles = np.arange(17, 32, 2) * 2.0 ** rng.integers(-8, 4, (24, 1, 8))   # 17/256 .. 31 * 8 of the scale
    near = (middles[..., None] * scale * 2.0 ** (np.arange(8) / 512 - 4 / 512)).reshape(24, 1, 64)
    near[..., ::8] = (middles * np.float64(np.float32(scale)))   # as near to the middle as bf16 comes
    n.k = n.v = bf16(near * np.where(rng.random((24, 1, 64)) < 0.5, -1, 1))
    n.kd = n.vd = on_gpu(n.k)
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, None,
                  cu_tokens=n.cu)
    torch.cuda.synchronize()
    assert plan.status() == 0
    nearest_codes(c, n, not_turned, (c.kc, c.ks, c.vc, c.vs))


@pytest.mark.parametrize("dim, interleaved", [(0, False), (64, False), (128, True)])
@pytest.mark.parametrize("size", [0.01, 1.0, 300.0])
def test_append_into_blocks_of_any_scale(dim, interleaved, size):
    """Rows that go on inside blocks quantised by somebody else: the held scale stays (small values), or rises to a
    power of two and the held codes move to it (large ones)."""
    c = Cache([5, 16, 31, 100, 7, 48], Hq=8, H=4, D=128, ps=48, seed=410, room=40, scales="amax")
    c.upload()
    n = New(c, [1, 11, 16, 33, 0, 3], fused=True, seed=411, size=size)
    r, turn = (None, not_turned) if not dim else rotary_of(dim=dim, interleaved=interleaved)
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r,
                  q=n.qd, q_out=n.q_out, cu_tokens=n.cu)
    torch.cuda.synchronize()
    assert plan.status() == 0
    nearest_codes(c, n, turn, (c.kc, c.ks, c.vc, c.vs))


def test_append_into_blocks_of_negative_scale():
    """A code stands for code * scale whatever the scale's sign: the held tokens keep their values at the new scale."""
    c = Cache([5, 9], Hq=2, H=1, D=64, seed=420, room=16)
    n = New(c, [3, 4], seed=421, size=4.0)
    c.ks[:], c.vs[:] = -np.float32(2.0) ** -3, -np.float32(2.0) ** 4   # lower and higher than the new values ask for
    c.upload()
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, None,
                  cu_tokens=n.cu)
    torch.cuda.synchronize()
    # the same cache with positive scales
    c.kc, c.vc, c.ks, c.vs = c.kc ^ 0x80, c.vc ^ 0x80, -c.ks, -c.vs
    for b in range(2):   # (blocks without new tokens are left as they are)
        rows = cache8.places(c.table, b, c.lens[b], c.lens[b] + n.counts[b], 16)
        blk = np.unique(rows // 16)
        for x, codes, scales, pages, sc in ((n.k, c.kc, c.ks, "kp", "ks"), (n.v, c.vc, c.vs, "vp", "vs")):
            wc, ws, want = cache8.append_q8(cache8.bf16_to_f64(x), codes, scales, c.table, c.lens, n.counts, 16)
            got = c.d[pages].view(torch.uint8).cpu().numpy().reshape(want.shape)
            assert np.array_equal(c.d[sc].cpu().numpy().reshape(-1)[blk], ws.reshape(-1)[blk])
            here = np.arange(blk[0] * 16, blk[-1] * 16 + 16)
            here = here[~np.isnan(want[here, 0, 0])]
            assert np.array_equal(cache8.E4M3[got[here]], cache8.E4M3[wc.reshape(want.shape)[here]])
