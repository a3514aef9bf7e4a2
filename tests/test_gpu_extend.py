"""pkv_extend and pkv_extend_q8 on the GPU against the definition in 64 bits.

Tolerances, element by element.  Let A = sum_t w_t |v_t| with the exact weights w, and n the tokens seen.
* A score is an fp32 dot product: off by at most d = (2 D + 16) 2^-23 max_t sum_e |q_e k_te| / sqrt(D).  In the 8-bit
  cache (exact codes, their scale joins in fp32) the query is two e4m3 numbers, scaled so that its largest element lies
  in [2^7, 2^8): the second holds the first's remainder to half of e4m3's smallest step, 2^-10 of 2^7, which adds
  2^-17 max_e |q_e| sum_e |k_te| / sqrt(D) at most.
* A weight is off by a factor of 2 d + 2^-20 (score and reference, ex2, V scale), then rounded: r = 2^-8 of itself in
  bf16; times its V scale in f16, 2^-11 of itself or half a step of 2^-24 where the largest such product is at least
  2^6 (8-bit; and 2^-16 for the logarithm of the scale).  Sums of n terms in fp32 add n 2^-23.  So |out error| <= (r + 2 (2 d + 2^-20 + n 2^-23)) A (numerator
  and denominator), for 8 bits and n tokens + n 2^-31 448 max_t w_t |scale_t|, and rounding the output to bf16 adds
  2^-8 |out|, or half a subnormal step.
* A weight below 2^-126, fp32's least normal number, against a largest one of 1 or more is 0: n 2^-126 max |v|.
* |lse error| <= 2 d + 2^-20 + n 2^-23 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

from paged_kv_decode_block_gb300 import pkv

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load()


class Problem:
    """Rows of `lens` cached tokens that take `new` more, the last of the row, on scattered pages."""

    def __init__(self, lens, new, *, Hq=8, Hkv=2, D=128, ps=16, q8=False, scales="pow2", seed=0, extra=3, fused=False,
                 size=1.0):
        self.lens, self.new = list(lens), list(new)
        self.after = [a + b for a, b in zip(lens, new)]
        self.B, self.Hq, self.Hkv, self.D, self.ps, self.q8 = len(self.lens), Hq, Hkv, D, ps, q8
        self.gen = torch.Generator("cuda").manual_seed(seed)
        used = [-(-n // ps) for n in self.after]
        self.pages, wide = sum(used) + extra, max(max(used), 1) + 1
        order = torch.randperm(self.pages, generator=self.gen, device="cuda").int()
        self.table = torch.full((self.B, wide), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, ps, Hkv, D)
        if q8:
            blocks = (self.pages, ps // 16, Hkv)
            self.k, self.v = (torch.randint(0, 256, shape, generator=self.gen, device="cuda").to(torch.uint8) for _ in "kv")
            for x in (self.k, self.v):
                x[(x & 0x7f) == 0x7f] = 0x55
            s = torch.rand((2,) + blocks, generator=self.gen, device="cuda") * 0.02 + 0.001
            self.ks, self.vs = torch.exp2(torch.round(torch.log2(s))) if scales == "pow2" else s
            self.k, self.v = self.k.view(FP8), self.v.view(FP8)
        else:
            self.k, self.v = (torch.randn(shape, generator=self.gen, device="cuda").bfloat16() for _ in "kv")
        self.T = sum(self.new)
        x = (torch.randn(self.T, Hq + 2 * Hkv, D, generator=self.gen, device="cuda") * size).bfloat16()
        self.q = x[:, :Hq] if fused else x[:, :Hq].contiguous()
        ints = dict(dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), **ints)
        self.lens_d = torch.tensor(self.after, **ints)
        self.out = torch.full((self.T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, Hq), 7.0, device="cuda")
        self.plan = pkv.Plan(self.after, None, ps, B=self.B, Hq=Hq, Hkv=Hkv, D=D, max_pages=wide, num_pages=self.pages)

    def run(self, **kw):
        kw = {**dict(q=self.q, out=self.out, lse=self.lse, cu_tokens=self.cu, table=self.table, lens=self.lens_d), **kw}
        args = (kw.pop("q"),) + ((self.k, self.v, self.ks, self.vs) if self.q8 else (self.k, self.v)) + \
            (kw.pop("table"), kw.pop("lens"), self.plan, kw.pop("out"))
        (pkv.extend_q8 if self.q8 else pkv.extend)(*args, **kw)
        return self

    def cached(self, b, n):
        t = torch.arange(n, device="cuda")
        flat = self.table[b].long()[t // self.ps] * self.ps + t % self.ps
        if not self.q8:
            return (x.flatten(0, 1)[flat].double() for x in (self.k, self.v))
        return (x.flatten(0, 1).view(torch.uint8)[flat].view(FP8).double() * s.flatten(0, 1)[flat // 16][..., None].double()
                for x, s in ((self.k, self.ks), (self.v, self.vs)))

    def check(self, rows=None, out=None, lse=None):
        out, lse = self.out if out is None else out, self.lse if lse is None else lse
        at, D, G = 0, self.D, self.Hq // self.Hkv
        for b, (n, a) in enumerate(zip(self.after, self.new)):
            here = slice(at, at + a)
            at += a
            if not a or (rows is not None and b not in rows):
                continue
            k, v = self.cached(b, n)
            hidden = torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1)
            for h in range(self.Hq):
                kh, vh, q = k[:, h // G], v[:, h // G], self.q[here, h].double()
                z = (q @ kh.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                size = (q.abs() @ kh.abs().T / math.sqrt(D)).masked_fill(hidden, 0)
                ref_lse = torch.logsumexp(z, 1)
                w = torch.softmax(z, 1)
                ref, A = w @ vh, w @ vh.abs()
                d = (2 * D + 16) * 2.0 ** -23 * size.amax(1)
                if self.q8:
                    far = kh.abs().sum(1).expand(a, n).masked_fill(hidden, 0).amax(1)
                    d = d + 2.0 ** -17 * q.abs().amax(1) * far / math.sqrt(D)
                f = 2 * (2 * d + 2.0 ** -20 + n * 2.0 ** -23)
                r = 2.0 ** -11 + 2.0 ** -16 if self.q8 else 2.0 ** -8   # (2^-16: the logarithm of the V scale)
                tol = (r + f)[:, None] * A + 2.0 ** -8 * ref.abs() + 2.0 ** -133 + n * 2.0 ** -126 * vh.abs().max()
                if self.q8:
                    t = torch.arange(n, device="cuda")
                    blk = (self.table[b].long()[t // self.ps] * self.ps + t % self.ps) // 16
                    heaviest = (w * self.vs.flatten(0, 1)[blk, h // G].double().abs()).amax(1)
                    tol = tol + (n * 2.0 ** -31 * 448 * heaviest)[:, None]
                got = out[here, h].double()
                assert torch.isfinite(got).all(), (b, h)
                over = ((got - ref).abs() / tol).max().item()
                assert over <= 1, (b, h, over)
                err = (lse[here, h].double() - ref_lse).abs()
                assert (err <= 2 * d + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * ref_lse.abs()).all(), (b, h, err.max().item())
        assert self.plan.status() == 0
        return self


BOTH = pytest.mark.parametrize("q8", [False, True], ids=["bf16", "q8"])


@BOTH
@pytest.mark.parametrize("D", [64, 128])
def test_one_block(D, q8):
    Problem([0], [5], D=D, q8=q8).run().check()


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens, new", [([0], [1]), ([0], [128]), ([100], [29]), ([128], [1]), ([300], [64]), ([0], [700])])
def test_one_row(lens, new, D, q8):
    Problem(lens, new, D=D, q8=q8).run().check()


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("ps", [16, 48, 128])
def test_shapes(G, D, ps, q8):
    Problem([0, 130, 1000, 17, 0], [33, 128, 300, 1, 515], Hq=2 * G, Hkv=2, D=D, ps=ps, q8=q8, scales="amax").run().check()


@BOTH
@pytest.mark.parametrize("ps", [32, 64, 80, 112, 256])
def test_pages(ps, q8):
    Problem([7, 0, 513], [40, 300, 2], ps=ps, q8=q8).run().check()


@BOTH
def test_edges(q8):
    """Rows without new tokens, of one token, ends around a block, a page and a tile."""
    new = [0, 1, 1, 63, 64, 65, 127, 128, 129, 0, 31, 33]
    lens = [50, 0, 127, 65, 64, 63, 1, 0, 0, 0, 1000, 2015]
    Problem(lens, new, q8=q8, Hq=4, Hkv=1, D=64).run().check()


@BOTH
@pytest.mark.parametrize("lens, new, Hkv", [([32768 - 5], [5], 8), ([40000], [1], 1), ([9000, 20, 30000], [3, 2, 9], 2)])
def test_few_tokens_over_a_long_cache(lens, new, Hkv, q8):
    """Tiles shared by many CTAs."""
    Problem(lens, new, Hq=4 * Hkv, Hkv=Hkv, q8=q8, extra=1).run().check()


@BOTH
def test_long_chunks(q8):
    Problem([3000, 0], [1500, 2600], Hq=8, Hkv=2, q8=q8).run().check()


@BOTH
def test_many_rows(q8):
    """More rows than a CTA has threads."""
    rng = np.random.default_rng(3)
    lens, new = rng.integers(0, 60, 1300), rng.integers(0, 4, 1300)
    Problem(lens.tolist(), new.tolist(), Hq=2, Hkv=1, D=64, q8=q8).run().check()


@BOTH
def test_no_tokens_at_all(q8):
    Problem([5, 0], [0, 0], q8=q8).run().check()


@BOTH
def test_one_token_a_row_without_offsets(q8):
    Problem([5, 0, 300], [1, 1, 1], q8=q8).run(cu_tokens=None).check()


def test_scales_of_any_kind():
    """Negative scales, zeros, and far apart ones; a scale that is not a number reaches who sees its block."""
    p = Problem([200, 0], [90, 300], q8=True, scales="amax")
    g = torch.Generator("cuda").manual_seed(9)
    for s in (p.ks, p.vs):
        s *= torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.3, -1.0, 1.0)
        s *= torch.exp2(torch.randint(-20, 3, s.shape, generator=g, device="cuda"))
        s[torch.rand(s.shape, generator=g, device="cuda") < 0.2] = 0
    p.run().check()
    was = p.out.clone(), p.lse.clone()
    p.ks[int(p.table[0, 256 // 16])] = math.nan      # tokens 256 to 271 of the first row: new ones from 56 on
    p.run()
    assert p.out[56:90].isnan().all() and p.lse[56:90].isnan().all()
    fine = torch.ones(p.T, dtype=torch.bool, device="cuda")
    fine[56:90] = False
    assert torch.equal(p.out[fine], was[0][fine]) and torch.equal(p.lse[fine], was[1][fine])
    p.ks[int(p.table[0, 256 // 16])] = 0.5
    p.vs[int(p.table[0, 256 // 16])] = math.inf
    p.run()
    assert not p.out[56:90].isfinite().any() and p.lse.isfinite().all() and torch.equal(p.out[fine], was[0][fine])


def test_queries_with_far_elements():
    """8-bit cache: elements from 2^-30 to 2^30 times the others, all small, all zero, and powers of two apart."""
    p = Problem([200], [70], q8=True, Hq=4, Hkv=2)
    p.q[0:10] = (p.q[0:10].float() * 2.0 ** -100).bfloat16()
    p.q[10:20, :, 3] *= 2.0 ** 6
    p.q[20:30] = 0
    p.q[30:40] = (p.q[30:40].float() * torch.exp2(torch.arange(128, device="cuda") % 13 - 12.0)).bfloat16()
    p.q[40:50, :, 5] = (p.q[40:50, :, 5].float() * 2.0 ** -30).bfloat16()
    p.run().check()
    # elements above 2^-10 of the largest are exact: the score of such a query is as good as in fp32
    p.q.copy_((torch.rand(70, 4, 128, device="cuda") + 0.01).bfloat16())
    p.run()
    k, _ = p.cached(0, 270)
    z = torch.einsum("ahd,nhd->han", p.q.double(), k.repeat_interleave(2, 1)) / math.sqrt(128)
    z = z.masked_fill(torch.ones(70, 270, dtype=torch.bool, device="cuda").triu(201), -math.inf)
    ref = torch.logsumexp(z, 2).T
    size = (p.q.double().abs().sum(2) * k.abs().amax() / math.sqrt(128))
    assert ((p.lse.double() - ref).abs() <= 2 * 272 * 2.0 ** -23 * size + 270 * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * ref.abs()).all()


@BOTH
def test_queries_that_are_not_finite(q8):
    """A query with an element that is no number is none itself (with an infinite one too, in the 8-bit cache), and no other."""
    p = Problem([200], [70], q8=q8, Hq=4, Hkv=2).run()
    was = p.out.clone(), p.lse.clone()
    p.q[7, 2, 11] = math.nan
    if q8:
        p.q[33, 1, 0] = -math.inf
    p.run()
    odd = torch.zeros(70, 4, dtype=torch.bool, device="cuda")
    odd[7, 2] = True
    odd[33, 1] = q8
    assert p.out[odd].isnan().all() and p.lse[odd].isnan().all()
    assert torch.equal(p.out[~odd], was[0][~odd]) and torch.equal(p.lse[~odd], was[1][~odd])


def test_one_token_a_row_is_the_decode():
    p = Problem([4096, 77, 0], [1, 1, 1], Hq=8, Hkv=2).run()
    out, lse = torch.empty(3, 8, 128, device="cuda"), torch.empty(3, 8, device="cuda")
    pkv.decode(p.q, p.k, p.v, p.table, p.lens_d, p.plan, out, lse)
    assert (p.lse - lse).abs().max().item() <= 1e-5
    # each within its tolerance of the exact value: weights and output rounded to bf16 here, fp32 there
    assert ((p.out.float() - out).abs() <= 2.0 ** -8 * out.abs() + 2.0 ** -8 * 4).all()


@BOTH
def test_strides(q8):
    """Queries in a projection's output, outputs in a wider tensor, whose other columns are left alone."""
    p = Problem([20, 300], [50, 3], q8=q8, fused=True)
    wide = torch.full((p.T, p.Hq + 3, p.D), 9.0, dtype=torch.bfloat16, device="cuda")
    p.run(out=wide[:, 1:p.Hq + 1]).check(out=wide[:, 1:p.Hq + 1])
    assert (wide[:, 0] == 9).all() and (wide[:, p.Hq + 1:] == 9).all()


@BOTH
@pytest.mark.parametrize("fused", [False, True])
def test_outputs_in_the_queries_place(fused, q8):
    p = Problem([20, 300, 9000], [50, 3, 70], q8=q8, fused=fused).run()
    was, was_lse = p.out.clone(), p.lse.clone()
    p.run(out=p.q)
    assert torch.equal(p.q, was) and torch.equal(p.lse, was_lse)


@BOTH
def test_lse_may_be_left_out(q8):
    p = Problem([20, 9000], [50, 3], q8=q8).run()
    was = p.out.clone()
    p.run(lse=None)
    assert torch.equal(was, p.out)


@BOTH
def test_queries_of_no_row_are_left_alone(q8):
    """Padding behind the last row's tokens (and before the first's)."""
    p = Problem([20, 300, 8], [50, 3, 4], q8=q8)
    cu = p.cu.clone()
    cu[3] = cu[2]
    p.run(cu_tokens=cu)
    assert (p.out[53:] == 7).all() and (p.lse[53:] == 7).all()
    p.check(rows=[0, 1])


@BOTH
def test_large_scores(q8):
    """Scores far apart: the running maximum moves, most weights vanish."""
    Problem([700, 0], [90, 400], q8=q8, size=30.0).run().check()


def test_rising_scores():
    """The maximum rises from block to block, far and near."""
    p = Problem([1000], [40], Hq=4, Hkv=1)
    t = torch.arange(1040, device="cuda")
    for step in (0.01, 0.3):
        flat = p.table[0].long()[t // 16] * 16 + t % 16
        p.k.flatten(0, 1)[flat] = (torch.randn(1040, 1, 128, device="cuda") * 0.1 + (t * step / 12)[:, None, None]).bfloat16()
        p.q.copy_((torch.rand(40, 4, 128, device="cuda") * 0.5 + 0.75).bfloat16())
        p.run().check()


@BOTH
def test_anything_behind_the_last_token(q8):
    p = Problem([3, 100, 0, 250], [2, 30, 1, 6], q8=q8, ps=64)
    p.run()
    was = p.out.clone(), p.lse.clone()
    t = torch.arange(64, device="cuda")
    for b, n in enumerate(p.after):
        if n % 64:
            page, rest = int(p.table[b, n // 64]), t >= n % 64
            for x in (p.k, p.v):
                (x.view(torch.uint8) if q8 else x)[page, rest] = 0x7f if q8 else math.nan
            if q8:
                for s in (p.ks, p.vs):
                    s[page, -(-(n % 64) // 16):] = math.nan
    p.run()
    assert torch.equal(was[0], p.out) and torch.equal(was[1], p.lse)
    p.check()


@BOTH
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_reach_only_who_sees_them(value, q8):
    lens, new, bad = [200, 0], [90, 40], 245   # a token of the chunk, and of V only
    p = Problem(lens, new, q8=q8, Hq=4, Hkv=2)
    p.run()
    was, was_lse = p.out.clone(), p.lse.clone()
    page, at = int(p.table[0, bad // 16]), bad % 16
    if q8:
        p.v.view(torch.uint8)[page, at, 1, 5] = 0x7f
    else:
        p.v[page, at, 1, 5] = value
    p.run()
    want = was.clone()
    want[bad - 200:90, 2:, 5] = math.nan if q8 else value
    assert torch.equal(p.out.isnan(), want.isnan())
    fine = ~want.isnan()
    assert torch.equal(p.out[fine], want[fine]) and torch.equal(p.lse, was_lse)


def test_value_not_finite_before_the_chunk():
    p = Problem([2000], [9], Hq=4, Hkv=2)
    p.v[int(p.table[0, 3]), 2, 0, 7] = math.inf
    p.run()
    odd = torch.zeros_like(p.out, dtype=torch.bool)
    odd[:, :2, 7] = True
    assert torch.equal(~p.out.isfinite(), odd)


def test_keys_that_are_not_finite():
    """A score of NaN makes the query NaN, one of -inf drops out; all -inf give 0 and -inf."""
    p = Problem([40], [3], Hq=1, Hkv=1, D=64)
    p.q.fill_(1.0)
    p.k[int(p.table[0, 42 // 16]), 42 % 16, 0, 0] = math.nan     # seen by the last query only
    p.k[int(p.table[0, 0]), 5, 0, 0] = -math.inf
    p.run()
    assert p.out[:2].isfinite().all() and p.out[2].isnan().all() and p.lse[2].isnan().all()
    p.k[..., 0] = -math.inf
    p.run()
    assert (p.out == 0).all() and (p.lse == -math.inf).all()


@BOTH
def test_repeats_give_the_same_bits(q8):
    p = Problem([9000, 0, 300], [3, 500, 40], q8=q8)
    p.run()
    was = p.out.clone(), p.lse.clone()
    for _ in range(3):
        p.out.zero_(), p.lse.zero_()
        p.run()
        assert torch.equal(was[0], p.out) and torch.equal(was[1], p.lse)


@BOTH
def test_captured_call_replayed_with_other_lengths(q8):
    a = Problem([9000, 50, 7], [3, 200, 0], q8=q8, seed=1)
    b = Problem([20, 8000, 300], [190, 1, 12], q8=q8, seed=2)   # the same number of tokens
    assert a.T == b.T
    a.plan.reserve_extend()
    wide = max(a.table.shape[1], b.table.shape[1])
    pages = max(a.pages, b.pages)
    hold = Problem([9000, 50, 7], [3, 200, 0], q8=q8)
    grow = lambda x, n: torch.cat([x.view(torch.uint8) if q8 else x, torch.zeros((n - x.shape[0],) + x.shape[1:], dtype=torch.uint8 if q8 else x.dtype, device="cuda")])  # noqa: E731
    hold.k, hold.v = grow(a.k, pages), grow(a.v, pages)
    if q8:
        more = torch.ones(pages - a.pages, 1, 2, device="cuda")
        hold.ks, hold.vs = torch.cat([a.ks, more]), torch.cat([a.vs, more])
    hold.table = torch.full((3, wide), -1, dtype=torch.int32, device="cuda")
    hold.plan = pkv.Plan([0, 0, 0], None, 16, B=3, Hq=8, Hkv=2, D=128, max_pages=wide, num_pages=pages)
    hold.plan.reserve_extend()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        hold.run()
    for p in (a, b, a):
        hold.table.fill_(-1)
        hold.table[:, :p.table.shape[1]] = p.table
        for x, y in ((hold.q, p.q), (hold.cu, p.cu), (hold.lens_d, p.lens_d)):
            x.copy_(y)
        for x, y in ((hold.k, p.k), (hold.v, p.v)):
            x[:p.pages] = y.view(torch.uint8) if q8 else y
        if q8:
            hold.ks[:p.pages], hold.vs[:p.pages] = p.ks, p.vs
        hold.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert hold.plan.status() == 0
        p.check(out=hold.out, lse=hold.lse)


def test_first_call_during_a_capture_is_refused():
    p = Problem([20], [4])
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(pkv.PkvError) as e:
            p.run()
    assert e.value.code == pkv.EINVAL
    graph.replay()
    p.plan.reserve_extend()
    p.plan.reserve_extend()
    p.run().check()


@BOTH
def test_another_stream_and_calls_behind_one_another(q8):
    p = Problem([300, 9000], [60, 5], q8=q8)
    o = Problem([50], [400], q8=q8, seed=5)
    p.plan.reserve_extend(), o.plan.reserve_extend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(p.out) for _ in range(4)]
    lses = [torch.empty_like(p.lse) for _ in range(4)]
    with torch.cuda.stream(side):
        for x, y in zip(outs, lses):
            p.run(out=x, lse=y)
    o.run()   # another plan, at the same time
    torch.cuda.synchronize()
    for x, y in zip(outs, lses):
        p.check(out=x, lse=y)
    o.check()
    p.run(stream=side)
    torch.cuda.synchronize()
    p.check()


@BOTH
def test_pages_outside_the_pool(q8):
    p = Problem([300, 9000, 40], [60, 5, 30], q8=q8)
    for page in (p.pages, -1, 2 ** 31 - 1):
        table = p.table.clone()
        table[1, 17] = page
        p.run(table=table)
        assert p.plan.status() == pkv.DEV_PAGE_OOB
        assert p.out[60:65].isnan().all() and p.lse[60:65].isnan().all()
        p.check(rows=[0, 2])
    table = p.table.clone()     # entries behind the row's last token are not looked at
    table[0, -1] = 2 ** 31 - 1
    table[2, 5:] = p.pages
    p.run(table=table).check()


@BOTH
def test_lengths_that_cannot_be(q8):
    p = Problem([300, 100, 40], [60, 5, 30], q8=q8)
    for n in (4, -1, 0, p.table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        lens = p.lens_d.clone()
        lens[1] = n
        p.run(lens=lens)
        assert p.plan.status() == pkv.DEV_PLAN_MISMATCH
        assert p.out[60:65].isnan().all() and p.lse[60:65].isnan().all()
        p.check(rows=[0, 2])


@BOTH
def test_offsets_that_cannot_be(q8):
    p = Problem([300, 100, 40], [60, 5, 30], q8=q8)
    for cu in ([0, 60, 65, 96], [-3, 60, 65, 95], [0, 60, 59, 95], [0, 2 ** 31 - 1, 65, 95]):
        p.out.fill_(7.0)
        p.run(cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert p.plan.status() == pkv.DEV_PLAN_MISMATCH, cu
    p.run().check()


def test_refusals():
    p = Problem([20], [6], Hq=4, Hkv=2)
    for bad in (dict(q=p.q[:5]), dict(q=p.q.float()), dict(out=p.out.float()), dict(lse=p.lse[:, :2]), dict(lse=p.lse.half()),
                dict(cu_tokens=p.cu.long()), dict(cu_tokens=p.cu[:1]), dict(table=p.table[:, :1]), dict(lens=p.lens_d.cpu()),
                dict(q=p.q[:1].expand(6, 4, 128)), dict(out=p.out.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            p.run(**bad)
    with pytest.raises(pkv.PkvError):      # six tokens, one row, no offsets
        p.run(cu_tokens=None)
    odd = torch.zeros(p.q.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:1 + p.q.numel()].view(p.q.shape)
    with pytest.raises(pkv.PkvError):      # not on a 16-byte boundary
        p.run(q=odd)
    wide = torch.zeros(6, 4 * 128 + 4, dtype=torch.bfloat16, device="cuda")[:, :512].view(6, 4, 128)
    with pytest.raises(pkv.PkvError):      # tokens 8 bytes off it
        p.run(out=wide)
    p.run().check()


def test_offsets_past_32_bits():
    """Pages of a pool of more than 2^32 bytes and 2^31 elements."""
    ps, Hkv, D = 256, 8, 128
    pages = 2 ** 31 // (ps * Hkv * D) + 40
    p = Problem([300, 1000], [20, 3], Hq=16, Hkv=Hkv, D=D, ps=ps)
    k, v = (torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k[-p.pages:], v[-p.pages:] = p.k, p.v
    p.k, p.v = k, v
    p.table = torch.where(p.table >= 0, p.table + pages - p.pages, p.table)
    p.plan = pkv.Plan(p.after, None, ps, B=2, Hq=16, Hkv=Hkv, D=D, max_pages=p.table.shape[1], num_pages=pages)
    p.run().check()


@pytest.mark.parametrize("G", [1, 4])
@BOTH
def test_a_row_of_almost_two_to_the_31(G, q8):
    """A table as long as a plan takes, whose tokens before the last 32 lie in one page and weigh nothing (scores of
    -448, the others within a few tens of 0): lengths and positions that a sign bit or a rounding up could break."""
    p = Problem([12], [20], Hq=G, Hkv=1, D=64, q8=q8)
    used = p.table[0, :2].clone()
    far = next(i for i in range(p.pages) if i not in used.tolist())
    p.q[..., 0] = 8.0
    if q8:
        p.k.view(torch.uint8)[far] = 0
        p.k.view(torch.uint8)[far, ..., 0] = 0xfe
        p.ks[far] = 1.0
    else:
        p.k[far] = 0.0
        p.k[far, ..., 0] = -448.0
    wide = 2 ** 27 - 1
    table = torch.full((1, wide), far, dtype=torch.int32, device="cuda")
    table[0, -2:] = used
    lens = torch.full((1,), wide * 16, dtype=torch.int32, device="cuda")
    plan = pkv.Plan([32], None, 16, B=1, Hq=G, Hkv=1, D=64, max_pages=wide, num_pages=p.pages)
    short, p.plan = p.plan, plan
    p.run(table=table, lens=lens)
    torch.cuda.synchronize()
    assert plan.status() == 0
    p.plan = short
    p.check()


def test_decode_of_the_same_plan_at_the_same_time():
    p = Problem([3000, 200, 8000], [40, 1, 300])
    q = torch.randn(3, 8, 128, generator=p.gen, device="cuda").bfloat16()
    alone, out = (torch.empty(3, 8, 128, device="cuda") for _ in range(2))
    lse = torch.empty(3, 8, device="cuda")
    pkv.decode(q, p.k, p.v, p.table, p.lens_d, p.plan, alone, lse)
    p.plan.reserve_extend()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        p.run()
        pkv.decode(q, p.k, p.v, p.table, p.lens_d, p.plan, out, lse, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, alone)
    p.check()
