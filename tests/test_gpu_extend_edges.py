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


def far_scores(p, b, c):
    """Token t of row b gets score c[t]: D = 64, queries of 8 in element 0, keys of scale 1."""
    assert p.D == 64 and len(c) == p.after[b]
    k = torch.zeros(len(c), p.Hkv, 64, device="cuda")
    k[..., 0] = torch.tensor(c, dtype=torch.float32, device="cuda")[:, None]
    p.k.flatten(0, 1).view(torch.uint8)[slots(p, b, len(c))] = k.to(FP8).view(torch.uint8)


@pytest.mark.parametrize("lens, new", [([200], [3]), ([130, 0], [200, 300]), ([20000], [5])])
def test_values_of_scale_zero_or_far_apart(lens, new):
    """8-bit: scales of V that are 0, where scores are high, and scales so far apart that the factor on a weight is out of
    fp32's range where the weight itself is 0."""
    p = Problem(lens, new, q8=True, Hq=4, Hkv=1, D=64)
    p.q.zero_()
    p.q[..., 0] = 8.0
    p.ks.fill_(1.0)
    was = p.vs.clone()
    rng = torch.Generator().manual_seed(11)

    def blocks(b, lo, hi):   # the scales' places of the row's tokens [lo, hi), both multiples of 16
        return slots(p, b, p.after[b])[lo:hi:16] // 16

    def scales(s):
        p.vs.flatten(0, 1)[:] = s
        return p.vs.flatten(0, 1)

    for b, n in enumerate(p.after):
        # high scores, and no scale of V but 0 in the first block of 128, or anywhere
        far_scores(p, b, [240.0] * n)
    s = scales(was.flatten(0, 1))
    for b in range(p.B):
        s[blocks(b, 0, 128)] = 0
    p.run().check()
    s.zero_()
    p.run().check()
    assert (p.out == 0).all()
    # the heaviest token has a scale of V of 0, and all others weigh nothing
    for b, n in enumerate(p.after):
        far_scores(p, b, [448.0 if t == 5 else float(t % 11) for t in range(n)])
    s = scales(was.flatten(0, 1))
    for b in range(p.B):
        s[blocks(b, 0, 16)] = 0
    p.run().check()
    # the heaviest token's scale is small, and those of tokens that weigh next to nothing are large; and the other way round
    for heavy, light in ((2.0 ** -100, 2.0 ** 110), (2.0 ** 110, 2.0 ** -100), (2.0 ** -140, 1.0), (0.0, 2.0 ** 110)):
        for far, near in ((60.0, 0.0), (80.0, 0.0), (88.0, 1.5), (104.0, 0.0)):
            for b, n in enumerate(p.after):
                far_scores(p, b, [far if t % 150 == 5 else near for t in range(n)])
            s = scales(light)
            for b, n in enumerate(p.after):
                at = slots(p, b, n)[5::150] // 16
                s[at] = heavy
            p.run().check()
    # anything
    for b, n in enumerate(p.after):
        far_scores(p, b, (torch.rand(n, generator=rng) * 160 - 80).tolist())
    s = scales(torch.exp2(torch.rand(was.flatten(0, 1).shape, generator=rng).cuda() * 220 - 110))
    s[::7] = 0
    p.run().check()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_scales_of_v_that_are_not_finite(value):
    """8-bit: who sees a token of the scale's block answers no number, whatever the codes; the logarithm is K's alone."""
    p = Problem([200, 0, 9000], [90, 300, 4], q8=True, scales="amax").run()
    was = p.out.clone(), p.lse.clone()
    odd = torch.zeros_like(p.out, dtype=torch.bool)
    p.vs[int(p.table[0, 256 // 16]), 0, 1] = value    # tokens 256 to 271 of the first row, the second KV head
    odd[56:90, 4:] = True
    p.vs[int(p.table[2, 7]), 0, 0] = value            # seen by all of the third row's new tokens, in whole blocks
    odd[390:394, :4] = True
    p.v.view(torch.uint8)[int(p.table[2, 7])] = 0
    p.run()
    assert torch.equal(~p.out.isfinite(), odd)
    assert torch.equal(p.out[:390][~odd[:390]], was[0][:390][~odd[:390]]) and torch.equal(p.lse, was[1])
    p.check(rows=[1])


@BOTH
@pytest.mark.parametrize("new", [3, 35])
def test_a_row_does_not_depend_on_the_next_rows_queries(new, q8):
    """A tile's box of queries goes on into the next row's.  Scores that rise by 2^3 a block move the reference now and
    then; queries that are not the row's, in the same warp, have no say in when: the same bits."""
    p = Problem([30000, 0], [new, 60], Hq=32, Hkv=8, q8=q8)
    n = p.after[0]
    ramp = (torch.arange(n, device="cuda") - (n - 1540)).clamp(min=0) * 0.00144
    k = torch.randn(n, 8, 128, generator=p.gen, device="cuda") * 0.1 + ramp[:, None, None]
    at = slots(p, 0, n)
    if q8:
        p.k.flatten(0, 1).view(torch.uint8)[at] = (k * 64).to(FP8).view(torch.uint8)
        p.ks.fill_(2.0 ** -6)
    else:
        p.k.flatten(0, 1)[at] = k.bfloat16()
    q = torch.rand(p.q.shape, generator=p.gen, device="cuda") * 0.5 + 0.75
    results = []
    for size in (0.0, 20.0, 1.0):
        x = q.clone()
        x[new:] *= size
        p.q.copy_(x.bfloat16())
        p.out.fill_(7.0), p.lse.fill_(7.0)
        p.run().check()
        results.append((p.out[:new].clone(), p.lse[:new].clone()))
    for out, lse in results[1:]:
        assert torch.equal(lse, results[0][1]) and torch.equal(out, results[0][0])
    p.run(out=p.q)   # (the next row's outputs are being written over its queries)
    assert torch.equal(p.q[:new], results[0][0]) and torch.equal(p.lse[:new], results[0][1])


def test_elements_of_a_query_that_are_exact():
    """8-bit: elements down to 2^-9 of the largest, a power of two here, are exact, and so is the score as far as fp32 is;
    K is 0 where the largest element is.  The next ones below are off by at most 2^-17 of the largest."""
    p = Problem([200], [70], q8=True, Hq=4, Hkv=2)
    p.k.view(torch.uint8)[..., 0] = 0
    for low, exact in ((2.0 ** -9, True), (2.0 ** -10, False)):
        q = 128 * low * (1 + torch.randint(0, 128, (70, 4, 128), generator=p.gen, device="cuda") / 128)
        q *= torch.where(torch.rand(q.shape, generator=p.gen, device="cuda") < 0.5, -1, 1)
        q[..., 0] = 128
        p.q.copy_(q.bfloat16())
        assert torch.equal(p.q.float(), q.float())
        p.run().check()
        k, _ = p.cached(0, 270)
        k = k.repeat_interleave(2, 1)
        hidden = torch.ones(70, 270, dtype=torch.bool, device="cuda").triu(201)
        z = torch.einsum("ahd,nhd->han", p.q.double(), k) / math.sqrt(128)
        ref = torch.logsumexp(z.masked_fill(hidden, -math.inf), 2).T
        size = torch.einsum("ahd,nhd->han", p.q.double().abs(), k.abs()).masked_fill(hidden, 0).amax(2).T / math.sqrt(128)
        tol = 2 * 272 * 2.0 ** -23 * size + 270 * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * ref.abs()
        if not exact:
            tol = tol + 128 * 2.0 ** -17 * k.abs().sum(2).amax(0) / math.sqrt(128)
        assert ((p.lse.double() - ref).abs() <= tol).all()


@BOTH
def test_what_bad_offsets_leave_alone(q8):
    """Rows with offsets that cannot be are left out: tokens of no other row keep what they held, and the other rows are
    answered."""
    p = Problem([300, 100, 40], [60, 5, 30], q8=q8)
    whole = {0: range(0, 60), 1: range(60, 65), 2: range(65, 95)}
    for cu, good in (([0, 60, 65, 96], [0, 1]), ([-3, 60, 65, 95], [1, 2]), ([0, 60, 50, 50], [0]),
                     ([0, 2 ** 31 - 1, 65, 95], [2]), ([0, 60, 2 ** 31 - 1, 2 ** 31 - 1], [0])):
        p.out.fill_(7.0), p.lse.fill_(7.0)
        p.run(cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert p.plan.status() == pkv.DEV_PLAN_MISMATCH, cu
        p.check(rows=good)
        left = torch.ones(p.T, dtype=torch.bool, device="cuda")
        for b in good:
            left[list(whole[b])] = False
        assert (p.out[left] == 7).all() and (p.lse[left] == 7).all(), cu


@BOTH
@pytest.mark.parametrize("lens, new", [(0, 700), (9000, 60)])
def test_each_token_in_its_turn(lens, new, q8):
    """Queries that single a token out: its V is the answer, and nothing else can make up for it."""
    p = Problem([lens], [new], Hq=8, Hkv=2, q8=q8, size=1.0)
    n = lens + new
    # (keys alike in size, so that a query along one of them scores highest there)
    k = torch.where(torch.rand(n, 2, 128, generator=p.gen, device="cuda") < 0.5, -1.0, 1.0)
    at = slots(p, 0, n)
    if q8:
        p.k.flatten(0, 1).view(torch.uint8)[at] = k.to(FP8).view(torch.uint8)
        p.ks.fill_(1.0)
    else:
        p.k.flatten(0, 1)[at] = k.bfloat16()
    limit = torch.arange(lens, n, device="cuda")
    for part in range(4):   # the token itself, the first ones, and others it sees
        pick = (limit if part == 0 else (limit - lens) if part == 1 else
                (torch.rand(new, generator=p.gen, device="cuda") * (limit + 1)).long()).clamp(max=n - 1)
        p.q.copy_((k[pick] * 4).repeat_interleave(4, 1).bfloat16())
        p.run().check()
        _, v = p.cached(0, n)
        # 128 * 4 / sqrt(128) = 45 for the token, and few others above 20
        assert ((p.out.double() - v[pick].repeat_interleave(4, 1)).abs() <= 2.0 ** -6 * v.abs().max()).all()
