"""pkv_append_rotary, pkv_append_q8 and pkv_decode_q8 on the GPU against the fp64
oracle (oracle/cache8.py), alone and run together.

Tolerances.
* Rotation: an fp32 rotation of a bf16 pair (x, y).  The angle is reduced exactly and enters
  sincospif rounded by 2^-25 of at most a quarter half-turn, sincospif is off by a few ulps, and three
  fp32 roundings follow: |error| <= 2^-20 (|x| + |y|) scale covers it.  Rounding the result adds half a
  step: 2^-8 of the value in bf16, 2^-4 in e4m3, or 2^-10 of the scale in e4m3's subnormal range.
* Attention: exact inputs, fp32 dot products and sums.  A score is off by at most
  d = (D + 16) 2^-23 max_t sum_d |q_d k_td| / sqrt(D); a weight by a factor of 2 d and about 2^-20 (exp2,
  the f16 split, the reference's product), the sum of n weights by n 2^-23.  So |out error| <=
  (2 d + (n + 64) 2^-23 + 2^-20) * 2 max|v| (numerator and denominator), |lse error| <= half of that factor.
"""
import numpy as np
import pytest
import torch

from oracle import cache8
from paged_kv_decode_block_gb300 import pkv

pytestmark = pytest.mark.gpu

ROUTES = ["direct", "split_queue", "split_padded", "persistent"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load()


def bf16(x):
    """float array to bf16 bit patterns (nearest even)."""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def on_gpu(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def make_table(rng, lens, ps, extra=3, max_pages=None):
    used = [-(-int(n) // ps) for n in lens]
    pages = sum(used) + extra
    table = np.full((len(lens), max_pages or max(max(used), 1) + 1), -1, np.int32)
    order = rng.permutation(pages).astype(np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def make_codes(rng, pages, ps, H, D, scales="pow2"):
    codes = rng.integers(0, 256, (pages, ps, H, D)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x55
    s = rng.random((pages, ps // 16, H)) * 0.02 + 0.001
    s = 2.0 ** np.round(np.log2(s)) if scales == "pow2" else s
    return codes, s.astype(np.float32)


def make_plan(lens, ps, Hq, H, D, table, pages, **opts):
    return pkv.Plan(lens, None, ps, B=len(lens), Hq=Hq, Hkv=H, D=D, max_pages=table.shape[1], num_pages=pages, **opts)


class Cache:
    """A random 8-bit cache on the host and the device."""

    def __init__(self, lens, *, Hq, H, D, ps=16, seed=0, scales="pow2", extra=3, max_pages=None, room=0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.ps, self.Hq, self.H, self.D = rng, np.array(lens, np.int32), ps, Hq, H, D
        self.B = len(lens)
        self.table, self.pages = make_table(rng, self.lens + room, ps, extra, max_pages)
        self.kc, self.ks = make_codes(rng, self.pages, ps, H, D, scales)
        self.vc, self.vs = make_codes(rng, self.pages, ps, H, D, scales)
        self.q = bf16(rng.standard_normal((self.B, Hq, D)))

    def upload(self):
        f8 = lambda c: torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn)  # noqa: E731
        self.d = dict(q=on_gpu(self.q), kp=f8(self.kc), vp=f8(self.vc), ks=torch.from_numpy(self.ks.copy()).cuda(),
                      vs=torch.from_numpy(self.vs.copy()).cuda(), table=torch.from_numpy(self.table).cuda(),
                      lens=torch.from_numpy(self.lens.copy()).cuda(),
                      out=torch.full((self.B, self.Hq, self.D), 7.0, device="cuda"),
                      lse=torch.full((self.B, self.Hq), 7.0, device="cuda"))
        return self.d

    def plan(self, **opts):
        return make_plan(self.lens, self.ps, self.Hq, self.H, self.D, self.table, self.pages, **opts)

    def decode(self, plan, stream=None):
        d = self.d
        pkv.decode_q8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["lens"], plan, d["out"], d["lse"],
                      stream=stream)

    def check(self, rows=None, what=""):
        torch.cuda.synchronize()
        q = cache8.bf16_to_f64(self.q)
        ref_out, ref_lse = cache8.decode_q8(q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens)
        out, lse = self.d["out"].cpu().numpy(), self.d["lse"].cpu().numpy()
        for b in range(self.B) if rows is None else rows:
            check_row(out[b], lse[b], ref_out[b], ref_lse[b], *self.bounds(b, q), what=f"{what} row {b}")

    def bounds(self, b, q):
        n, G = int(self.lens[b]), self.Hq // self.H
        if n == 0:
            return 0.0, 0.0
        rows = cache8.places(self.table, b, 0, n, self.ps)
        kf = np.abs(cache8.E4M3[self.kc.reshape(-1, self.H, self.D)[rows]])
        kf *= self.ks.reshape(-1, self.H).astype(np.float64)[rows // 16][..., None]
        dot = max(float((np.abs(q[b, h * G:(h + 1) * G]) @ kf[:, h].T).max()) for h in range(self.H))
        vf = np.abs(cache8.E4M3[self.vc.reshape(-1, self.H, self.D)[rows]])
        vmax = float((vf * self.vs.reshape(-1, self.H).astype(np.float64)[rows // 16][..., None]).max())
        f = 2 * (self.D + 16) * 2.0 ** -23 * dot / np.sqrt(self.D) + (n + 64) * 2.0 ** -23 + 2.0 ** -20
        return 2 * f * vmax, f


def check_row(out, lse, ref_out, ref_lse, out_tol, lse_tol, what=""):
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse)), what
    fine = ~np.isneginf(ref_lse)
    assert np.max(np.abs(out - ref_out), initial=0) <= out_tol, (what, np.max(np.abs(out - ref_out)), out_tol)
    assert np.max(np.abs(lse[fine] - ref_lse[fine]), initial=0) <= lse_tol * max(1.0, np.max(np.abs(ref_lse[fine]), initial=1.0)), what


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("ps", [16, 48])
def test_decode_shapes_and_edge_lengths(D, G, ps):
    c = Cache([1, 15, 16, 17, 0, 47, 48, 49, 300], Hq=2 * G, H=2, D=D, ps=ps, seed=D + G + ps)
    c.upload()
    plan = c.plan()
    c.decode(plan)
    c.check()
    assert plan.status() == 0


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("merge", ["last", "all", "separate"])
@pytest.mark.parametrize("splits", [1, 3, 70])
def test_decode_every_route_and_merge(route, merge, splits):
    if merge == "all" and route not in ("split_queue", "split_padded"):
        pytest.skip("the ALL merge belongs to the queue and padded routes")
    c = Cache([1200, 1, 0, 333], Hq=8, H=2, D=128, seed=splits, scales="amax")
    c.upload()
    opts = dict(separate_merge=True) if merge == "separate" else dict(merge=merge)
    plan = c.plan(force_mode=route, num_splits=splits, **opts)
    for _ in range(3):   # the counters are back at zero after each launch
        c.d["out"].fill_(7.0)
        c.decode(plan)
        c.check(what=f"{route} {merge} {splits}")
    first = c.d["out"].clone()
    c.decode(plan)
    torch.cuda.synchronize()
    assert torch.equal(first, c.d["out"])   # the same bits each time
    assert plan.status() == 0


def test_decode_more_than_one_batch_of_blocks():
    """A warp's blocks pass 32 (one fetch of table entries and scales) twice: 8 * 16 * 70 tokens in one tile."""
    c = Cache([9000, 4095, 4097], Hq=4, H=1, D=64, ps=16, seed=5, scales="amax")
    c.upload()
    c.decode(c.plan(force_mode="direct"))
    c.check()


@pytest.mark.parametrize("B", [200, 256, 257])
def test_decode_many_unequal_rows(B):
    """More tiles than the GPU holds at once, rows of all lengths (equal ones, empty ones): up to 256 rows are taken
    longest first, more in row order; the device's lengths decide, also after the plan was made."""
    rng = np.random.default_rng(B)
    lens = rng.choice([0, 1, 16, 33, 100, 100, 250, 600], B)
    c = Cache(lens, Hq=8, H=2, D=64, seed=B, room=16)
    c.upload()
    plan = c.plan(force_mode="direct")
    assert plan.info()["grid_ctas"] == 2 * B
    c.decode(plan)
    c.check()
    c.lens = (lens + rng.integers(0, 17, B)).astype(np.int32)   # the direct route follows the device's lengths
    c.d["lens"].copy_(torch.from_numpy(c.lens))
    c.d["out"].fill_(7.0)
    c.decode(plan)
    c.check()
    c.lens = c.lens.copy()
    c.d["lens"][3] = -5   # and flags one that cannot be
    c.decode(plan)
    torch.cuda.synchronize()
    assert plan.status() == pkv.DEV_PLAN_MISMATCH and torch.isnan(c.d["out"][3]).all()
    c.check(rows=[b for b in range(B) if b != 3])


def test_decode_reads_nothing_behind_the_last_token():
    c = Cache([5, 16, 31, 100], Hq=16, H=2, D=128, ps=32, seed=6)
    for b, n in enumerate(c.lens):
        rest = cache8.places(c.table, b, n, -(-n // 32) * 32, 32)
        c.kc.reshape(-1, 2, 128)[rest] = 0x7F   # NaN codes
        c.vc.reshape(-1, 2, 128)[rest] = 0xFF
        for s in (c.ks, c.vs):
            tail = rest[rest % 16 == 0] // 16   # blocks wholly behind the last token
            s.reshape(-1, 2)[tail] = np.nan
    c.upload()
    for route in ROUTES:
        c.d["out"].fill_(7.0)
        c.decode(c.plan(force_mode=route, num_splits=2))
        c.check(what=route)


def test_decode_scales_far_apart():
    """V scales from 2^-30 to 2^10 and K scales that make a row's scores rise and fall: the references of the
    weights and of the sums move, and a token of a small block that holds the whole weight keeps its value."""
    c = Cache([800, 800, 64, 800], Hq=8, H=2, D=128, seed=7)
    nblk = 50
    for b, order in ((0, np.linspace(-30, 10, nblk)), (1, np.linspace(10, -30, nblk))):
        blk = cache8.places(c.table, b, 0, 800, 16)[::16] // 16
        c.vs.reshape(-1, 2)[blk] = (2.0 ** np.round(order))[:, None]
    blk = cache8.places(c.table, 3, 0, 800, 16)[::16] // 16
    c.ks.reshape(-1, 2)[blk] = np.linspace(0.0, 0.05, nblk)[:, None]
    c.vs.reshape(-1, 2)[blk[:3]] = 0.0
    c.upload()
    c.decode(c.plan(num_splits=2, force_mode="split_queue"))
    c.check()


def test_decode_one_token_holds_the_weight_in_a_small_block():
    """One key far above the others, in a block whose V scale is 2^-12 of the others': out is that token's V, whose
    error is relative to itself plus 2^-31 of the others'."""
    c = Cache([160], Hq=4, H=1, D=64, seed=8)
    c.kc[:] = 0
    rows = cache8.places(c.table, 0, 0, 160, 16)
    q = cache8.bf16_to_f64(c.q)[0]
    c.q = bf16(np.broadcast_to(q[:1], (1, 4, 64)))
    c.kc.reshape(-1, 1, 64)[rows[37], 0] = cache8.e4m3_encode(np.sign(q[0]) * 448)
    c.ks[:] = 2.0 ** -2
    c.vs[:] = 1.0
    c.vs.reshape(-1)[rows[37] // 16] = 2.0 ** -12
    c.upload()
    c.decode(c.plan(force_mode="direct"))
    torch.cuda.synchronize()
    v = cache8.E4M3[c.vc.reshape(-1, 1, 64)[rows[37], 0]] * 2.0 ** -12
    got = c.d["out"].cpu().numpy()[0]
    assert np.max(np.abs(got - v)) <= 2.0 ** -20 * np.abs(v).max() + 448 * 2.0 ** -31


@pytest.mark.parametrize("D, G", [(64, 1), (64, 8), (128, 2), (128, 4)])
def test_decode_many_light_tokens_beside_a_heavy_one(D, G):
    """One key 2^31 times heavier than each of 200 thousand others: together the light ones carry 2^-13 of the sum, and
    their values, 2^10 times larger, an eighth of the output."""
    n = 200_000
    c = Cache([n], Hq=G, H=1, D=D, ps=256, seed=17)
    c.q = bf16(np.full((1, G, D), 0.5))
    c.kc[:], c.ks[:] = 0, 1.0
    first = int(c.table[0, 0]) * 256
    score = 31 * np.log(2.0) * np.sqrt(D)
    c.kc.reshape(-1, 1, D)[first] = cache8.e4m3_encode(1.0)
    c.ks.reshape(-1)[first // 16] = score / (0.5 * D)
    c.vs[:] = 2.0 ** -9 * 1024
    c.vs.reshape(-1)[first // 16] = 2.0 ** -9
    c.vc &= 0x7F   # no signs: the light tokens' values do not cancel
    c.upload()
    for route in ("direct", "split_queue"):
        c.decode(c.plan(force_mode=route))
        torch.cuda.synchronize()
        ref, _ = cache8.decode_q8(cache8.bf16_to_f64(c.q), c.kc, c.vc, c.ks, c.vs, c.table, c.lens)
        got = c.d["out"].cpu().numpy()
        # every term is positive: sums, weights and values are each off by a few 2^-20 relative at most
        # (200000 tokens over 8 warps and 8 lanes: 2^12 additions of 2^-24 each in a lane)
        assert np.max(np.abs(got / ref - 1)) <= 2.0 ** -11, (route, np.max(np.abs(got / ref - 1)))


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 1.0, 2.0 ** 40])
def test_decode_queries_of_any_size(size):
    """q times a power of two with K scales divided by it: the same scores."""
    c = Cache([200, 33], Hq=8, H=2, D=128, seed=9)
    c.q = bf16(cache8.bf16_to_f64(c.q) * size)
    c.ks = (c.ks / size).astype(np.float32)
    c.upload()
    c.decode(c.plan())
    c.check()


def test_decode_zero_queries_and_a_zero_cache():
    c = Cache([40, 16], Hq=4, H=2, D=64, seed=10)
    c.q[:] = 0
    c.upload()
    c.decode(c.plan())
    c.check()
    c.kc[:], c.vc[:], c.ks[:], c.vs[:] = 0x80, 0, 0.0, 0.0
    c.q = bf16(np.ones((2, 4, 64)))
    c.upload()
    c.decode(c.plan())
    c.check()


def test_decode_flags_a_bad_page_and_a_stale_plan():
    for bad in (-1, 10 ** 6):
        c = Cache([100, 100, 50], Hq=8, H=2, D=128, seed=11)
        good = c.table.copy()
        c.table[1, 3] = bad
        c.upload()
        for route in ROUTES:
            plan = c.plan(force_mode=route, num_splits=3)
            c.decode(plan)
            torch.cuda.synchronize()
            assert plan.status() == pkv.DEV_PAGE_OOB
            assert torch.isnan(c.d["out"][1]).all() and torch.isnan(c.d["lse"][1]).all(), route
            c.table = good
            c.check(rows=[0, 2], what=route)
            c.table = good.copy()
            c.table[1, 3] = bad
    c = Cache([100, 100, 50], Hq=8, H=2, D=128, seed=12)
    c.upload()
    plan = c.plan(force_mode="split_queue", num_splits=2)
    c.d["lens"][0] = 17   # not what was planned
    c.decode(plan)
    torch.cuda.synchronize()
    assert plan.status() & pkv.DEV_PLAN_MISMATCH
    assert torch.isnan(c.d["out"][0]).all()
    c.check(rows=[1, 2])


def test_decode_offsets_past_32_bits():
    """A pool of more than 2^31 bytes a tensor; the rows' pages lie at its two ends."""
    H, D, ps = 8, 128, 256
    pages = (1 << 31) // (ps * H * D) + 200
    c = Cache([600, 300], Hq=32, H=H, D=D, ps=ps, seed=13)
    small_k, small_v, small_ks, small_vs, small_table = c.kc, c.vc, c.ks, c.vs, c.table
    move = {int(p): pages - 1 - i if i % 2 else i for i, p in enumerate(np.unique(small_table[small_table >= 0]))}
    assert any(p * ps * H * D > 1 << 31 for p in move.values())
    table = np.vectorize(lambda p: move.get(int(p), -1))(small_table).astype(np.int32)
    c.upload()
    d = c.d
    for key, src in (("kp", small_k), ("vp", small_v)):
        big = torch.zeros((pages, ps, H, D), dtype=torch.uint8, device="cuda")
        for a, b in move.items():
            big[b] = torch.from_numpy(src[a]).cuda()
        d[key] = big.view(torch.float8_e4m3fn)
    for key, src in (("ks", small_ks), ("vs", small_vs)):
        big = torch.zeros((pages, ps // 16, H), device="cuda")
        for a, b in move.items():
            big[b] = torch.from_numpy(src[a]).cuda()
        d[key] = big
    d["table"] = torch.from_numpy(table).cuda()
    plan = make_plan(c.lens, ps, 32, H, D, table, pages)
    c.decode(plan)
    c.check()
    # and the append at the far end: row 0's next tokens
    rot = pkv.Rotary(64)
    new = bf16(c.rng.standard_normal((2, H, D)))
    after = torch.zeros(2, dtype=torch.int32, device="cuda")
    pkv.append_q8(on_gpu(new), on_gpu(new), d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["lens"], after, plan, rot)
    torch.cuda.synchronize()
    assert after.tolist() == [601, 301] and plan.status() == 0
    x = cache8.bf16_to_f64(new)
    for b in range(2):
        at = int(cache8.places(table, b, c.lens[b], c.lens[b] + 1, ps)[0])
        got = cache8.E4M3[d["vp"].view(-1, H, D)[at].view(torch.uint8).cpu().numpy()]
        s = d["vs"].view(-1, H)[at // 16].cpu().numpy().astype(np.float64)[:, None]
        assert np.all(np.abs(got * s - x[b]) <= 2.0 ** -4 * np.abs(x[b]) + s * 2.0 ** -10)


def test_decode_on_another_stream_and_in_a_graph():
    c = Cache([700, 20, 0, 1500], Hq=16, H=4, D=128, seed=14)
    c.upload()
    plan = c.plan(force_mode="split_queue", num_splits=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.decode(plan, stream=side)
    side.synchronize()
    c.check(what="side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.decode(plan)
    for seed in (1, 2):   # other inputs in the same buffers
        rng = np.random.default_rng(seed)
        c.q = bf16(rng.standard_normal(c.q.shape))
        c.kc, c.ks = make_codes(rng, c.pages, 16, 4, 128)
        c.d["q"].copy_(on_gpu(c.q))
        c.d["kp"].view(torch.uint8).copy_(torch.from_numpy(c.kc))
        c.d["ks"].copy_(torch.from_numpy(c.ks))
        graph.replay()
        c.check(what=f"replay {seed}")
    assert plan.status() == 0


def test_decode_refusals():
    c = Cache([40, 16], Hq=4, H=2, D=64, seed=15)
    d = c.upload()
    plan = c.plan()
    call = lambda **kw: pkv.decode_q8(*[kw.get(n, d[n]) for n in ("q", "kp", "vp", "ks", "vs", "table", "lens")],  # noqa: E731
                                      kw.get("plan", plan), kw.get("out", d["out"]), d["lse"])
    with pytest.raises(pkv.PkvError) as e:
        call(plan=c.plan(math="fma"))
    assert e.value.code == pkv.EUNSUPPORTED
    with pytest.raises(TypeError):
        call(kp=d["kp"].float())
    with pytest.raises(TypeError):
        call(ks=d["ks"].double())
    with pytest.raises(ValueError):
        call(ks=d["ks"][1:])
    with pytest.raises(ValueError):
        call(kp=d["kp"][1:])
    with pytest.raises(TypeError):
        call(out=d["out"].transpose(0, 1))
    with pytest.raises(TypeError):
        call(q=d["q"].cpu())
    lib, h, P = pkv.load(), plan.handle, {k: v.data_ptr() for k, v in d.items()}
    args = [P["q"], P["kp"], P["vp"], P["ks"], P["vs"], P["table"], P["lens"], h, P["out"], P["lse"], None]
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9):
        bad = list(args)
        bad[i] = None
        assert lib.pkv_decode_q8(*bad) == pkv.EINVAL
    for i, off in ((0, 2), (1, 8), (2, 4), (3, 2), (4, 1), (5, 2), (6, 2), (8, 4), (9, 2)):
        bad = list(args)
        bad[i] += off
        assert lib.pkv_decode_q8(*bad) == pkv.EINVAL
    torch.cuda.synchronize()
    assert plan.status() == 0


def test_trace_and_profile_cover_the_8bit_decode():
    c = Cache([400, 30], Hq=4, H=1, D=64, seed=16)
    c.upload()
    plan = c.plan(force_mode="split_queue", num_splits=3)
    plan.trace(True)
    plan.profile(True)
    c.decode(plan)
    c.check()
    rows = plan.read_trace()
    assert len(rows) == plan.info()["grid_ctas"] and (rows[:, pkv.TR_TILES] == 1).all()
    assert (rows[:, pkv.TR_EXIT] >= rows[:, pkv.TR_ENTRY]).all() and (rows[:, pkv.TR_ENTRY] > 0).all()
    ms = plan.profile_read()
    assert len(ms) == 1 and ms[0] > 0


# ------------------------------------------------------------------ appends

class New:
    """New tokens for the rows of a cache."""

    def __init__(self, c, counts, *, fused=False, offsets=True, seed=1, size=1.0):
        rng = np.random.default_rng(seed)
        self.counts = list(counts)
        T = sum(counts)
        self.T = T
        if fused:
            qkv = bf16(size * rng.standard_normal((T, c.Hq + 2 * c.H, c.D)))
            dev = on_gpu(qkv)
            cut = (slice(0, c.Hq), slice(c.Hq, c.Hq + c.H), slice(c.Hq + c.H, None))
            (self.q, self.k, self.v), (self.qd, self.kd, self.vd) = [qkv[:, x] for x in cut], [dev[:, x] for x in cut]
        else:
            self.q, self.k, self.v = (bf16(size * rng.standard_normal((T, h, c.D))) for h in (c.Hq, c.H, c.H))
            self.qd, self.kd, self.vd = on_gpu(self.q), on_gpu(self.k), on_gpu(self.v)
        self.cu = None
        if offsets:
            self.cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        self.pos = np.concatenate([np.arange(n, n + k) for n, k in zip(c.lens, counts)] + [[]]).astype(np.int64)
        self.q_out = torch.full((T, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.after = torch.full((c.B,), -5, dtype=torch.int32, device="cuda")


def freqs(dim, base=10000.0):
    return base ** (-np.arange(0, dim, 2) / dim)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def near_bf16(got_bits, want, x, scale=1.0):
    got = cache8.bf16_to_f64(got_bits)
    ax = np.abs(x)
    pair = ax.max(-1, keepdims=True) * 2   # a bound on |x| + |y| of any pair
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * pair * scale)


ROT = [dict(dim=0), dict(dim=16), dict(dim=64), dict(dim=32, interleaved=True), dict(dim=64, interleaved=True, scale=1.25)]


def rotary_of(dim=0, interleaved=False, scale=1.0):
    if not dim:
        return None, lambda x, pos: cache8.rotate(x, pos, [])
    r = pkv.Rotary(dim, interleaved=interleaved, scale=scale)
    return r, lambda x, pos: cache8.rotate(x, pos, freqs(dim), interleaved, np.float32(scale))


LENS, COUNTS = [0, 5, 16, 31, 100, 7, 48, 0], [1, 11, 16, 33, 0, 250, 1, 0]


@pytest.mark.parametrize("rot", ROT, ids=str)
@pytest.mark.parametrize("D, G, fused", [(64, 4, False), (128, 1, True), (128, 8, False)])
def test_append_rotary(rot, D, G, fused):
    c = Cache(LENS, Hq=2 * G, H=2, D=D, ps=32, seed=20, room=256)
    c.upload()
    n = New(c, COUNTS, fused=fused)
    rng = np.random.default_rng(3)
    kp, vp = (bf16(rng.standard_normal((c.pages, 32, 2, D))) for _ in range(2))
    kd, vd = on_gpu(kp), on_gpu(vp)
    r, turn = rotary_of(**rot)
    plan = c.plan()
    pkv.append_rotary(n.kd, n.vd, kd, vd, c.d["table"], c.d["lens"], n.after, plan, r, q=n.qd, q_out=n.q_out,
                      cu_tokens=n.cu)
    torch.cuda.synchronize()
    assert plan.status() == 0
    assert n.after.tolist() == [a + b for a, b in zip(LENS, COUNTS)] and c.d["lens"].tolist() == LENS
    x = cache8.bf16_to_f64(n.k)
    near_bf16(bits(n.q_out), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q), rot.get("scale", 1))
    want = cache8.append_values(turn(x, n.pos), cache8.bf16_to_f64(kp), c.table, c.lens, COUNTS, 32)
    rows = np.concatenate([cache8.places(c.table, b, c.lens[b], c.lens[b] + k, 32) for b, k in enumerate(COUNTS)])
    got = bits(kd).reshape(want.shape)
    near_bf16(got[rows], want[rows], x, rot.get("scale", 1))
    rest = np.ones(len(got), bool)
    rest[rows] = False
    assert np.array_equal(got[rest], kp.reshape(want.shape)[rest])   # nothing else is written
    vw = vp.reshape(want.shape).copy()
    vw[rows] = n.v
    assert np.array_equal(bits(vd).reshape(want.shape), vw)          # values go in as they are


def check_q8(c, n, turn, before, scale=1.0):
    """The device cache against the oracle's append; `before`: host (kc, ks, vc, vs)."""
    d = c.d
    kx, vx = cache8.bf16_to_f64(n.k), cache8.bf16_to_f64(n.v)
    for x, codes, scales, pages, sc in ((turn(kx, n.pos), before[0], before[1], "kp", "ks"),
                                        (vx, before[2], before[3], "vp", "vs")):
        wc, ws, want = cache8.append_q8(x, codes, scales, c.table, c.lens, n.counts, c.ps)
        assert np.array_equal(d[sc].cpu().numpy().astype(np.float64), ws)
        got = d[pages].view(torch.uint8).cpu().numpy().reshape(want.shape)
        written = ~np.isnan(want)
        assert np.array_equal(got[~written], codes.reshape(want.shape)[~written])
        pair = np.abs(kx if sc == "ks" else vx).max(initial=0) * 2 * scale
        slop = 2.0 ** -20 * pair / np.repeat(ws.reshape(-1, c.H), 16, 0)[..., None]
        off = np.abs(cache8.E4M3[got] - want)
        limit = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + slop
        assert np.all(off[written] <= limit[written])
        # all but the values next to a rounding border have the oracle's own code
        assert np.mean(got != wc.reshape(want.shape)) < 1e-3


@pytest.mark.parametrize("rot", ROT, ids=str)
@pytest.mark.parametrize("D, G, fused", [(64, 4, False), (128, 1, True), (128, 8, False)])
def test_append_q8(rot, D, G, fused):
    c = Cache(LENS, Hq=2 * G, H=2, D=D, ps=32, seed=21, room=256, scales="amax")
    c.upload()
    n = New(c, COUNTS, fused=fused, size=3.0)
    r, turn = rotary_of(**rot)
    plan = c.plan()
    for _ in range(2):   # the second call finds its own result and changes nothing
        pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r,
                      q=n.qd, q_out=n.q_out, cu_tokens=n.cu)
        torch.cuda.synchronize()
        assert plan.status() == 0
        assert n.after.tolist() == [a + b for a, b in zip(LENS, COUNTS)] and c.d["lens"].tolist() == LENS
        near_bf16(bits(n.q_out), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q), rot.get("scale", 1))
        check_q8(c, n, turn, (c.kc, c.ks, c.vc, c.vs), rot.get("scale", 1))


@pytest.mark.parametrize("q8", [False, True])
def test_append_one_token_a_row_without_offsets(q8):
    c = Cache([0, 1, 15, 16, 17, 63], Hq=8, H=4, D=128, seed=22, room=1)
    c.upload()
    n = New(c, [1] * 6, offsets=False)
    r, turn = rotary_of(dim=128)
    plan = c.plan()
    if q8:
        pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r)
        check_q8(c, n, turn, (c.kc, c.ks, c.vc, c.vs))
    else:
        kd = torch.zeros((c.pages, 16, 4, 128), dtype=torch.bfloat16, device="cuda")
        vd = torch.zeros_like(kd)
        pkv.append_rotary(n.kd, n.vd, kd, vd, c.d["table"], c.d["lens"], n.after, plan, r)
        rows = np.array([cache8.places(c.table, b, c.lens[b], c.lens[b] + 1, 16)[0] for b in range(6)])
        near_bf16(bits(kd).reshape(-1, 4, 128)[rows], turn(cache8.bf16_to_f64(n.k), n.pos), cache8.bf16_to_f64(n.k))
        assert np.array_equal(bits(vd).reshape(-1, 4, 128)[rows], n.v)
    assert n.after.tolist() == [1, 2, 16, 17, 18, 64] and plan.status() == 0


def test_append_in_place_queries_and_many_rows():
    """More rows than a CTA has threads, a few with many tokens; q turned in place."""
    rng = np.random.default_rng(23)
    B = 300
    lens, counts = rng.integers(0, 40, B), rng.integers(0, 3, B)
    counts[7], counts[299] = 100, 40
    c = Cache(lens, Hq=2, H=1, D=64, seed=24, room=100)
    c.upload()
    n = New(c, counts.tolist())
    r, turn = rotary_of(dim=64)
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r, q=n.qd,
                  q_out=n.qd, cu_tokens=n.cu)
    torch.cuda.synchronize()
    near_bf16(bits(n.qd), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q))
    check_q8(c, n, turn, (c.kc, c.ks, c.vc, c.vs))
    assert n.after.tolist() == (lens + counts).tolist()


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_turns_the_queries_inside_a_fused_projection(interleaved):
    """q_out is q's own slice of the projection's output: the queries turn in place, keys and values beside them stay."""
    c = Cache([3, 40, 0], Hq=16, H=2, D=128, seed=33, room=80)   # G = 8: two passes over the queries
    c.upload()
    n = New(c, [60, 1, 17], fused=True)
    k, v = n.kd.clone(), n.vd.clone()
    r, turn = rotary_of(dim=64, interleaved=interleaved)
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r, q=n.qd,
                  q_out=n.qd, cu_tokens=n.cu)
    torch.cuda.synchronize()
    near_bf16(bits(n.qd), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q))
    check_q8(c, n, turn, (c.kc, c.ks, c.vc, c.vs))
    assert torch.equal(n.kd, k) and torch.equal(n.vd, v) and plan.status() == 0


@pytest.mark.parametrize("H, G", [(8, 4), (3, 1), (2, 8)])
@pytest.mark.parametrize("q8", [False, True])
def test_append_long_prompts(H, G, q8):
    """Prompts long enough that a CTA takes two KV heads, and an odd number of heads, which it takes one by one."""
    c = Cache([5, 0, 700], Hq=G * H, H=H, D=64, seed=34, room=6000, ps=16)
    c.upload()
    n = New(c, [5000, 1111, 600], fused=True)
    r, turn = rotary_of(dim=64)
    plan = c.plan()
    if q8:
        pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r, q=n.qd,
                      q_out=n.q_out, cu_tokens=n.cu)
        check_q8(c, n, turn, (c.kc, c.ks, c.vc, c.vs))
    else:
        kd, vd = (torch.zeros((c.pages, 16, H, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pkv.append_rotary(n.kd, n.vd, kd, vd, c.d["table"], c.d["lens"], n.after, plan, r, q=n.qd, q_out=n.q_out,
                          cu_tokens=n.cu)
        rows = np.concatenate([cache8.places(c.table, b, c.lens[b], c.lens[b] + k, 16) for b, k in enumerate(n.counts)])
        near_bf16(bits(kd).reshape(-1, H, 64)[rows], turn(cache8.bf16_to_f64(n.k), n.pos), cache8.bf16_to_f64(n.k))
        assert np.array_equal(bits(vd).reshape(-1, H, 64)[rows], n.v)
    near_bf16(bits(n.q_out), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q))
    assert n.after.tolist() == [5005, 1111, 1300] and plan.status() == 0


def test_append_far_positions():
    """Positions up to 2^31: the angles stay exact (an fp32 product would be off by whole turns)."""
    ps, D = 256, 64
    lens = [2 ** 31 - 4 * 256 - 100, 2 ** 30 + 3, 1_000_003]
    wide = (2 ** 31 - 1) // ps
    table = np.full((3, wide), -1, np.int32)
    counts = [90, 2, 20]
    at = 0
    for b, (n, k) in enumerate(zip(lens, counts)):
        for page in range(n // ps, (n + k - 1) // ps + 1):
            table[b, page] = at
            at += 1
    plan = pkv.Plan([0] * 3, None, ps, B=3, Hq=2, Hkv=1, D=D, max_pages=wide, num_pages=at)
    rng = np.random.default_rng(25)
    T = sum(counts)
    k = bf16(rng.standard_normal((T, 1, D)))
    kd = torch.zeros((at, ps, 1, D), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    after = torch.zeros(3, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 90, 92, 112], dtype=torch.int32, device="cuda")
    freq = freqs(64)
    pkv.append_rotary(on_gpu(k), on_gpu(k), kd, vd, torch.from_numpy(table).cuda(),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), after, plan, pkv.Rotary(64, inv_freq=freq),
                      cu_tokens=cu)
    torch.cuda.synchronize()
    assert plan.status() == 0 and after.tolist() == [a + b for a, b in zip(lens, counts)]
    pos = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, counts)])
    # the angle in 64-bit steps of a turn: p * inv_freq / 2 pi with a relative error of 2^-52 is off by up to
    # 2^31 * 2^-2.6 * 2^-52 = 2^-23.6 turns, 2^-21 rad, on either side: |x| + |y| <= 2 max |x| times that
    x = cache8.bf16_to_f64(k)
    want = cache8.rotate(x, pos, freq)
    rows = np.concatenate([cache8.places(table, b, n, n + m, ps) for b, (n, m) in enumerate(zip(lens, counts))])
    got = cache8.bf16_to_f64(bits(kd).reshape(-1, 1, D)[rows])
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(x).max())


@pytest.mark.parametrize("q8", [False, True])
def test_append_flags_bad_rows_and_leaves_them_alone(q8):
    lens = [20, 33, 32, 60, 47, 5, -3, 10]
    c = Cache([20, 33, 32, 60, 47, 5, 0, 10], Hq=4, H=2, D=64, seed=26, max_pages=4, room=0, extra=6)
    counts = [2, 20, 1, 10, 1, 3, 2, 1]
    # row 0 good; 1 runs from page 2 into an unassigned page 3; 2 unassigned; 3 past the table's end; 4 a page past
    # the pool; 5 good; 6 a negative length; 7 good
    table = c.table
    assert table[1, 3] == -1 and table[2, 2] == -1 and table[4, 2] >= 0
    table[4, 2] = c.pages + 5
    c.upload()
    c.d["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = New(c, counts)
    good = [0, 5, 7]
    plan = c.plan()
    q_before = n.q_out.clone()
    r, turn = rotary_of(dim=32)
    if q8:
        pages = [c.d["kp"], c.d["vp"]]
        pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r,
                      q=n.qd, q_out=n.q_out, cu_tokens=n.cu)
    else:
        pages = [torch.zeros((c.pages, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pkv.append_rotary(n.kd, n.vd, *pages, c.d["table"], c.d["lens"], n.after, plan, r, q=n.qd, q_out=n.q_out,
                          cu_tokens=n.cu)
    torch.cuda.synchronize()
    assert plan.status() == pkv.DEV_ROW_FULL | pkv.DEV_PAGE_OOB
    assert n.after.tolist() == [a + b if i in good else a for i, (a, b) in enumerate(zip(lens, counts))]
    start = np.concatenate([[0], np.cumsum(counts)])
    for b in range(8):
        same = torch.equal(n.q_out[start[b]:start[b + 1]], q_before[start[b]:start[b + 1]])
        assert same == (b not in good)
    rows = np.concatenate([cache8.places(table, b, lens[b], lens[b] + counts[b], 16) for b in good])
    old = c.kc.reshape(-1, 2, 64) if q8 else np.zeros((c.pages * 16, 2, 64), np.uint8)
    got = (pages[0].view(torch.uint8) if q8 else pages[0].ne(0).byte()).cpu().numpy().reshape(old.shape)
    blocks = np.unique(rows // 16)
    rest = np.array([i for i in range(c.pages * 16) if i // 16 not in blocks])
    assert np.array_equal(got[rest], old[rest])
    assert (got[rows] != old[rows]).any((1, 2)).all()


def test_append_bad_offsets_are_flagged():
    c = Cache([20, 33, 5], Hq=4, H=2, D=64, seed=27, room=40)
    plan = c.plan()
    r, _ = rotary_of(dim=64)
    for cu, good in (([0, 3, 2, 5], [0, 2]), ([0, 2, 4, 9], [0, 1]), ([-1, 2, 4, 5], [1, 2])):
        d = c.upload()
        n = New(c, [2, 2, 1])
        pkv.append_q8(n.kd, n.vd, *(d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, r,
                      cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert plan.status() == pkv.DEV_PLAN_MISMATCH
        for b in range(3):
            want = c.lens[b] + (cu[b + 1] - cu[b] if b in good else 0)
            assert n.after[b].item() == want, (cu, b)
            if b not in good:
                rows = cache8.places(c.table, b, c.lens[b] // 16 * 16, c.lens[b] // 16 * 16 + 16, 16)
                assert np.array_equal(d["kp"].view(torch.uint8).cpu().numpy().reshape(-1, 2, 64)[rows],
                                      c.kc.reshape(-1, 2, 64)[rows])


def test_append_token_by_token_is_the_chunk_at_once():
    """32 tokens one by one: the chunk's scales, and its codes but for those that fell below the normal range of a
    scale on the way (two roundings of half a subnormal step each)."""
    rng = np.random.default_rng(28)
    grow = 2.0 ** rng.integers(-3, 4, 32)
    c = Cache([13], Hq=4, H=2, D=64, seed=29, room=40)
    c.upload()
    n = New(c, [32], size=1.0)
    n.v = bf16(cache8.bf16_to_f64(n.v) * grow[:, None, None])
    n.vd = on_gpu(n.v)
    plan = c.plan()
    r, _ = rotary_of(dim=64)
    cache = ("kp", "vp", "ks", "vs")
    one = {x: c.d[x].clone() for x in cache}
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in cache), c.d["table"], c.d["lens"], n.after, plan, r, cu_tokens=n.cu)
    at, nxt = c.d["lens"].clone(), torch.empty_like(c.d["lens"])
    for i in range(32):
        pkv.append_q8(n.kd[i:i + 1], n.vd[i:i + 1], *(one[x] for x in cache), c.d["table"], at, nxt, plan, r)
        at, nxt = nxt, at
    torch.cuda.synchronize()
    assert at.tolist() == [45] and plan.status() == 0
    for pages, sc in (("kp", "ks"), ("vp", "vs")):
        assert torch.equal(one[sc], c.d[sc])
        a, b = (cache8.E4M3[x.view(torch.uint8).cpu().numpy()] for x in (one[pages], c.d[pages]))
        assert np.all(np.abs(a - b) <= np.where(np.abs(b) < 2.0 ** -6 * 1.0001, 2.0 ** -9, 0))


def test_append_values_that_are_not_finite_and_zeros():
    """NaN and infinities are stored as NaN and leave the scale to the others; a block of zeros has the least scale,
    which the next token replaces."""
    c = Cache([0, 0], Hq=1, H=1, D=64, seed=30, room=32)
    c.upload()
    n = New(c, [2, 1])
    x = np.zeros((3, 1, 64), np.float32)
    x[0, 0, :4] = [np.nan, np.inf, -np.inf, 3.0]
    x[1, 0, 0] = -5.0
    n.k = n.v = bf16(x)
    n.kd = n.vd = on_gpu(n.k)
    plan = c.plan()
    args = [c.d[x] for x in ("kp", "vp", "ks", "vs", "table")]
    pkv.append_q8(n.kd, n.vd, *args, c.d["lens"], n.after, plan, None, cu_tokens=n.cu)
    torch.cuda.synchronize()
    rows = [cache8.places(c.table, b, 0, 3, 16) for b in range(2)]
    code = c.d["kp"].view(torch.uint8).cpu().numpy().reshape(-1, 64)
    ks = c.d["ks"].cpu().numpy().reshape(-1)
    s = 2.0 ** -6   # 5 / 448 = 2^-6.5
    assert ks[rows[0][0] // 16] == s and ks[rows[1][0] // 16] == 2.0 ** -120
    assert np.isnan(cache8.E4M3[code[rows[0][0], :3]]).all()
    assert cache8.E4M3[code[rows[0][0], 3]] * s == 3.0 and cache8.E4M3[code[rows[0][1], 0]] * s == -5.0
    assert (cache8.E4M3[code[rows[1][0]]] == 0).all()
    # a second token into the zero block
    one = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    y = on_gpu(bf16(np.full((1, 1, 64), 0.5)))
    lens, after = n.after.clone(), torch.empty_like(n.after)
    pkv.append_q8(y, y, *args, lens, after, plan, None, cu_tokens=one)
    torch.cuda.synchronize()
    ks = c.d["ks"].cpu().numpy().reshape(-1)
    code = c.d["kp"].view(torch.uint8).cpu().numpy().reshape(-1, 64)
    assert ks[rows[1][0] // 16] == 2.0 ** -9   # 0.5 / 448 = 2^-9.8
    assert (cache8.E4M3[code[rows[1][1]]] * 2.0 ** -9 == 0.5).all() and after.tolist() == [2, 2]
    assert ks[rows[0][0] // 16] == s           # a row without new tokens is left alone


def test_append_of_no_tokens():
    c = Cache([20, 0], Hq=4, H=2, D=64, seed=31)
    c.upload()
    n = New(c, [0, 0])
    plan = c.plan()
    pkv.append_q8(n.kd, n.vd, *(c.d[x] for x in ("kp", "vp", "ks", "vs", "table", "lens")), n.after, plan, None,
                  cu_tokens=n.cu)
    torch.cuda.synchronize()
    assert n.after.tolist() == [20, 0] and plan.status() == 0
    assert np.array_equal(c.d["kp"].view(torch.uint8).cpu().numpy(), c.kc)


def test_append_refusals():
    c = Cache([20, 3], Hq=4, H=2, D=64, seed=32, room=8)
    d = c.upload()
    n = New(c, [2, 1])
    plan = c.plan()
    r = pkv.Rotary(64)

    def call(k=n.kd, v=n.vd, kp=d["kp"], ks=d["ks"], table=d["table"], lens=d["lens"], after=n.after, rot=r, q=n.qd,
             q_out=n.q_out, cu=n.cu):
        pkv.append_q8(k, v, kp, d["vp"], ks, d["vs"], table, lens, after, plan, rot, q=q, q_out=q_out, cu_tokens=cu)

    for kw, error in ((dict(k=n.kd.float()), TypeError), (dict(k=n.kd.cpu()), TypeError),
                      (dict(v=n.vd[:2]), ValueError), (dict(k=n.kd[..., :32]), ValueError),
                      (dict(k=n.kd.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                      (dict(kp=d["kp"].bfloat16()), TypeError), (dict(kp=d["kp"][1:]), ValueError),
                      (dict(ks=d["ks"].transpose(0, 2)), TypeError), (dict(ks=d["ks"][1:]), ValueError),
                      (dict(table=d["table"].long()), TypeError), (dict(lens=d["lens"][:1]), ValueError),
                      (dict(cu=n.cu[1:]), ValueError), (dict(cu=n.cu.long()), TypeError), (dict(q_out=None), ValueError),
                      (dict(q=n.qd[:2]), ValueError), (dict(after=d["lens"]), pkv.PkvError),
                      (dict(rot=pkv.Rotary(128)), pkv.PkvError), (dict(cu=None), pkv.PkvError)):
        with pytest.raises(error):
            call(**kw)
    # the C entry itself
    lib, h = pkv.load(), plan.handle
    import ctypes

    def raw(change=None, **ptrs):
        t = pkv.Tokens()
        t.q, t.q_out, t.k, t.v = n.qd.data_ptr(), n.q_out.data_ptr(), n.kd.data_ptr(), n.vd.data_ptr()
        t.cu_tokens_d, t.total_tokens = n.cu.data_ptr(), 3
        if change:
            change(t)
        P = {x: d[x].data_ptr() for x in ("kp", "vp", "ks", "vs", "table", "lens")} | {"after": n.after.data_ptr()} | ptrs
        return lib.pkv_append_q8(ctypes.byref(t), ctypes.byref(r.params), P["kp"], P["vp"], P["ks"], P["vs"], P["table"],
                                 P["lens"], P["after"], h, None)

    def setting(**kw):
        def change(t):
            for k, v in kw.items():
                setattr(t, k, v)
        return change

    for kw in (dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(k=n.kd.data_ptr() + 2),
               dict(q=n.qd.data_ptr() + 8), dict(total_tokens=-1), dict(cu_tokens_d=None), dict(k_stride=4),
               dict(k_stride=124), dict(k_stride=120), dict(v_stride=-128), dict(q_stride=128),
               dict(q_out=n.qd.data_ptr(), q_out_stride=512), dict(cu_tokens_d=n.cu.data_ptr() + 2)):
        assert raw(setting(**kw)) == pkv.EINVAL, kw
    for name in ("kp", "vp", "ks", "vs", "table", "lens", "after"):
        assert raw(**{name: None}) == pkv.EINVAL
    assert raw(kp=d["kp"].data_ptr() + 8) == pkv.EINVAL and raw(after=d["lens"].data_ptr() + 4) == pkv.EINVAL
    torch.cuda.synchronize()
    assert plan.status() == 0
    assert np.array_equal(d["kp"].view(torch.uint8).cpu().numpy(), c.kc)   # none of them wrote


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("D, G, ps", [(128, 4, 16), (64, 8, 32)])
def test_prompts_then_steps(D, G, ps):
    """Prompts enter an empty 8-bit cache in two ragged chunks, then every row is decoded token by token: each step's
    attention against the oracle over the cache as the device holds it, and that cache against the oracle's appends."""
    H, dim = 2, 64
    c = Cache([0] * 4, Hq=G * H, H=H, D=D, ps=ps, seed=40, room=200)
    c.upload()
    d = c.d
    r, turn = rotary_of(dim=dim, interleaved=True)
    plan = c.plan()
    after = torch.empty_like(d["lens"])
    chunks = [[70, 1, 0, 33], [3, 40, 100, 0]] + [[1] * 4] * 20
    for i, counts in enumerate(chunks):
        n = New(c, counts, fused=True, offsets=i < 2, seed=50 + i)
        before = [x.copy() for x in (c.kc, c.ks, c.vc, c.vs)]
        q_out = n.q_out
        pkv.append_q8(n.kd, n.vd, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["lens"], after, plan, r, q=n.qd,
                      q_out=q_out, cu_tokens=n.cu)
        check_q8(c, n, turn, before)
        c.kc, c.vc = (d[x].view(torch.uint8).cpu().numpy().copy() for x in ("kp", "vp"))
        c.ks, c.vs = (d[x].cpu().numpy().copy() for x in ("ks", "vs"))
        d["lens"], after = after, d["lens"]
        c.lens = c.lens + np.array(counts, np.int32)
        plan.update(c.lens)
        last = np.maximum(np.cumsum(counts) - 1, 0)   # each row's last token asks
        d["q"] = q_out[torch.from_numpy(last).cuda()].contiguous()
        c.q = bits(d["q"])
        c.decode(plan)
        c.check(what=f"chunk {i}")
    assert plan.status() == 0


def test_step_captured_in_a_graph():
    """Append and decode of two steps, captured with the two length buffers in turn and replayed; an eager run of the
    same steps gives the same bits.  The padded route takes its lengths from the device."""
    c = Cache([30, 64, 1], Hq=8, H=2, D=128, seed=41, room=40)
    r = pkv.Rotary(128)
    steps = [New(c, [1] * 3, offsets=False, seed=60 + i) for i in range(8)]

    def fresh():
        d = c.upload()
        plan = make_plan(c.lens + 40, 16, 8, 2, 128, c.table, c.pages, force_mode="split_padded", num_splits=3)
        return d, plan, torch.empty_like(d["lens"])

    def step(d, plan, x, a, b):
        pkv.append_q8(x.kd, x.vd, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], a, b, plan, r, q=x.qd, q_out=x.q_out)
        pkv.decode_q8(x.q_out, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], b, plan, d["out"], d["lse"])

    d, plan, other = fresh()
    want = []
    for i in range(0, 8, 2):
        for x, a, b in ((steps[i], d["lens"], other), (steps[i + 1], other, d["lens"])):
            step(d, plan, x, a, b)
            want.append((d["out"].clone(), d["lse"].clone()))
    cache = {x: d[x].view(torch.uint8).clone() if x[1] == "p" else d[x].clone() for x in ("kp", "vp", "ks", "vs", "lens")}
    assert plan.status() == 0

    d, plan, other = fresh()
    plan_warm = torch.empty_like(d["out"])
    bufs = [New(c, [1] * 3, offsets=False, seed=70 + i) for i in range(2)]
    pkv.decode_q8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["lens"], plan, plan_warm, d["lse"])  # uploads the plan
    outs = [torch.empty_like(d["out"]) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for x, a, b, o in ((bufs[0], d["lens"], other, outs[0]), (bufs[1], other, d["lens"], outs[1])):
            pkv.append_q8(x.kd, x.vd, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], a, b, plan, r, q=x.qd, q_out=x.q_out)
            pkv.decode_q8(x.q_out, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], b, plan, o, d["lse"])
    for i in range(0, 8, 2):
        for j in range(2):
            for name in ("qd", "kd", "vd"):
                getattr(bufs[j], name).copy_(getattr(steps[i + j], name))
        graph.replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert torch.equal(outs[j], want[i + j][0])
    for name, t in cache.items():
        assert torch.equal(d[name].view(torch.uint8) if name[1] == "p" else d[name], t), name
    assert plan.status() == 0


def test_rotated_append_then_bf16_decode():
    """append_rotary feeds pkv_decode: a prompt and two steps, the attention against a dense fp64 one."""
    H, G, D, ps, dim = 2, 4, 128, 16, 128
    c = Cache([0, 0], Hq=H * G, H=H, D=D, ps=ps, seed=42, room=60)
    c.upload()
    r, turn = rotary_of(dim=dim)
    kp = torch.zeros((c.pages, ps, H, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    lens, after = c.d["lens"], torch.empty_like(c.d["lens"])
    plan = c.plan()
    for i, counts in enumerate(([33, 17], [1, 1], [1, 1])):
        n = New(c, counts, seed=80 + i)
        pkv.append_rotary(n.kd, n.vd, kp, vp, c.d["table"], lens, after, plan, r, q=n.qd, q_out=n.q_out, cu_tokens=n.cu)
        lens, after = after, lens
        c.lens = c.lens + np.array(counts, np.int32)
        plan.update(c.lens)
        q = n.q_out[torch.tensor(np.cumsum(counts) - 1).cuda()].contiguous()
        pkv.decode(q, kp, vp, c.d["table"], lens, plan, c.d["out"], c.d["lse"])
        torch.cuda.synchronize()
        near_bf16(bits(n.q_out), turn(cache8.bf16_to_f64(n.q), n.pos), cache8.bf16_to_f64(n.q))
        import oracle
        ref = oracle.decode(bits(q), bits(kp), bits(vp), c.table, c.lens)
        assert np.max(np.abs(c.d["out"].cpu().numpy() - ref[0])) <= 2e-3
        assert np.max(np.abs(c.d["lse"].cpu().numpy() - ref[1])) <= 1e-4
    assert plan.status() == 0
