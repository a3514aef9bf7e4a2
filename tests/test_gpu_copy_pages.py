"""pkv_copy_pages on the GPU, and sessions that share a prefix: fork, copy, append, extend, compact, decode."""
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


def pools_of(kind, pages, ps, H, D, layers=1, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=gen, device="cuda", dtype=torch.int64).int()  # noqa: E731
    out = []
    for _ in range(2 * layers):
        if kind == "bf16":
            out.append(rnd(pages, ps, H, D // 2).view(torch.bfloat16))
        else:
            out += [rnd(pages, ps, H, D // 4).view(FP8), rnd(pages, ps // 16, H).view(torch.float32)]
    return out


def expected(pools, copies, ps):
    out = []
    for p in pools:
        x = p.view(torch.int8).clone()
        unit = ps // p.shape[1]
        for a, b, n in copies:
            x[b, :-(-n // unit)] = p.view(torch.int8)[a, :-(-n // unit)]
        out.append(x)
    return out


def same(pools, want):
    return all(torch.equal(p.view(torch.int8), w) for p, w in zip(pools, want))


def random_copies(rng, pages, n, ps, whole=False):
    ids = rng.permutation(pages)[:2 * n]
    return np.stack([ids[:n], ids[n:], np.full(n, ps) if whole else rng.integers(0, ps + 1, n)], 1).astype(np.int32)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("ps, H, D", [(16, 1, 64), (16, 8, 128), (48, 1, 64), (256, 2, 128), (64, 3, 64)])
def test_copies(kind, ps, H, D):
    rng = np.random.default_rng(ps + H)
    pools = pools_of(kind, 90, ps, H, D)
    for n in (1, 7, 45):
        copies = random_copies(rng, 90, n, ps, whole=n == 7)
        want = expected(pools, copies, ps)
        pkv.copy_pages(pools, copies, ps)
        assert same(pools, want)


def test_one_source_for_many_targets():
    pools = pools_of("bf16", 40, 16, 2, 64)
    copies = [(5, b, b % 17) for b in range(40) if b != 5]
    want = expected(pools, copies, 16)
    pkv.copy_pages(pools, copies, 16)
    assert same(pools, want)


def test_more_copies_and_pools_than_one_launch_takes():
    rng = np.random.default_rng(1)
    pools = pools_of("q8", 10001, 16, 1, 64, layers=1) + pools_of("bf16", 10001, 16, 1, 64, layers=98, seed=2)
    assert len(pools) == 200
    copies = random_copies(rng, 10001, 5000, 16)
    want = expected(pools[:5] + pools[-2:], copies, 16)
    pkv.copy_pages(pools, copies, 16)
    assert same(pools[:5] + pools[-2:], want)


def test_nothing_to_copy():
    pools = pools_of("bf16", 4, 16, 1, 64)
    want = expected(pools, [], 16)
    pkv.copy_pages(pools, np.zeros((0, 3), np.int32), 16)
    pkv.copy_pages(pools, [], 16)
    pkv.copy_pages([], [(0, 1, 16)], 16)
    pkv.copy_pages(pools, [(0, 1, 0)], 16)
    assert same(pools, want)


def test_pools_off_a_16_byte_boundary():
    """Scales of one KV head lie 4 bytes apart; a pool may begin anywhere on 4."""
    buf = torch.arange(40 * 3 + 1, dtype=torch.float32, device="cuda")
    pool = buf[1:].view(40, 3, 1)
    was = pool.clone()
    pkv.copy_pages([pool], [(3, 5, 40), (7, 8, 16)], 48)
    was[5], was[8, :1] = was[3].clone(), was[7, :1].clone()
    assert torch.equal(pool, was) and buf[0] == 0


def test_offsets_past_32_bits():
    ps, H, D = 256, 8, 128
    pages = 2 ** 32 // (ps * H * D * 2) + 20
    pool = torch.zeros(pages, ps, H, D, dtype=torch.bfloat16, device="cuda")
    pool[pages - 3] = torch.randn(ps, H, D, device="cuda").bfloat16()
    pkv.copy_pages([pool], [(pages - 3, pages - 1, 200), (pages - 3, 1, 256)], ps)
    assert torch.equal(pool[pages - 1, :200], pool[pages - 3, :200]) and (pool[pages - 1, 200:] == 0).all()
    assert torch.equal(pool[1], pool[pages - 3]) and (pool[0] == 0).all() and (pool[2] == 0).all()


def test_in_a_graph_and_on_another_stream():
    pools = pools_of("q8", 20, 32, 2, 64)
    first = [p.clone() for p in pools]
    copies = random_copies(np.random.default_rng(4), 20, 9, 32)
    want = expected(pools, copies, 32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.copy_pages(pools, copies, 32)
    graph.replay()
    torch.cuda.synchronize()
    assert same(pools, want)
    for p, f in zip(pools, first):
        p.view(torch.int8).copy_(f.view(torch.int8))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.copy_pages(pools, copies, 32, stream=side)
    side.synchronize()
    assert same(pools, want)


def test_calls_behind_one_another():
    """A page copied on from where the call before has put it."""
    pools = pools_of("bf16", 64, 64, 8, 128)
    first = pools[0][0].clone()
    for i in range(60):
        pkv.copy_pages(pools, [(i, i + 1, 64)], 64)
    assert torch.equal(pools[0][60].view(torch.int16), first.view(torch.int16))


def test_refusals():
    pools = pools_of("bf16", 8, 16, 2, 64)
    for bad in (dict(pools=[pools[0][:, ::2]]), dict(pools=[pools[0].cpu()])):
        with pytest.raises(TypeError):
            pkv.copy_pages(bad["pools"], [(0, 1, 2)], 16)
    for bad in (dict(pools=[pools[0], pools[1][:7]]), dict(page_size=24), dict(copies=[(0, 1)]), dict(pools=[pools[0].flatten()])):
        with pytest.raises(ValueError):
            pkv.copy_pages(bad.get("pools", pools), bad.get("copies", [(0, 1, 2)]), bad.get("page_size", 16))
    want = expected(pools, [], 16)
    for bad in ([(0, 8, 1)], [(0, 1, 17)], [(0, 1, 2), (1, 3, 2)]):
        with pytest.raises(pkv.PkvError):
            pkv.copy_pages(pools, bad, 16)
    torch.cuda.synchronize()
    assert same(pools, want)


# ------------------------------------------------------------------ run together

def attention(q, k, v):
    """q [a][Hq][D], the last a of the n tokens of k / v [n][Hkv][D], in 64 bits."""
    a, Hq, D = q.shape
    n, H, _ = k.shape
    k, v = (x.double().repeat_interleave(Hq // H, 1) for x in (k, v))
    z = torch.einsum("ahd,nhd->han", q.double(), k) / math.sqrt(D)
    z = z.masked_fill(torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1), -math.inf)
    return torch.einsum("han,nhd->ahd", torch.softmax(z, -1), v), torch.einsum("han,nhd->ahd", torch.softmax(z, -1), v.abs())


@pytest.mark.parametrize("q8", [False, True], ids=["bf16", "q8"])
@pytest.mark.parametrize("ps", [16, 48])
def test_sessions_that_share_a_prefix(ps, q8):
    """A prompt enters the cache; three sessions fork from it (one inside a page, one at a page's end, one from nothing),
    go on with chunks of their own, the pool is compacted, and each answers a token: always the attention over the keys
    and values that its own history put there."""
    Hq, Hkv, D, pages, wide = 8, 2, 128, 64, 16
    gen = torch.Generator("cuda").manual_seed(ps)
    pool = pkv.Pool(np.random.default_rng(0).permutation(pages).astype(np.int32), pages)
    rotary = pkv.Rotary(D)
    if q8:
        blocks = (pages, ps // 16, Hkv)
        k, v = (torch.zeros(pages, ps, Hkv, D, device="cuda").to(FP8) for _ in "kv")
        ks, vs = (torch.zeros(blocks, device="cuda") for _ in "kv")
        cache, scales = [k, v, ks, vs], (ks, vs)
    else:
        k, v = (torch.full((pages, ps, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        cache, scales = [k, v], ()

    def gathered(row, n):
        t = torch.arange(n, device="cuda")
        flat = torch.from_numpy(row).cuda().long()[t // ps] * ps + t % ps
        if not q8:
            return [x.flatten(0, 1)[flat].double() for x in (k, v)]
        return [x.flatten(0, 1).view(torch.uint8)[flat].view(FP8).double() * s.flatten(0, 1)[flat // 16][..., None].double()
                for x, s in ((k, ks), (v, vs))]

    def go_on(table, lens, new):
        """Appends new[b] tokens to each row and attends; returns the lengths after."""
        B = len(lens)
        for b, (n, a) in enumerate(zip(lens, new)):
            for page in range(-(-n // ps), -(-(n + a) // ps)):
                one = np.full((1, 1), -1, np.int32)
                pool.reserve([0], one, ps)
                table[b, page] = one[0, 0]
        after = [n + a for n, a in zip(lens, new)]
        plan = pkv.Plan(after, table, ps, B=B, Hq=Hq, Hkv=Hkv, D=D, max_pages=wide, num_pages=pages)
        ints = dict(dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **ints)
        before, after_d, table_d = torch.tensor(lens, **ints), torch.empty(B, **ints), torch.from_numpy(table).cuda()
        T = sum(new)
        x = torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=gen).bfloat16()
        q, kn, vn = x.split([Hq, Hkv, Hkv], 1)
        rotated, out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        args = (kn, vn, *cache[:2], *scales, table_d, before, after_d, plan, rotary)
        held = [gathered(table[b], n) for b, n in enumerate(lens)]
        (pkv.append_q8 if q8 else pkv.append_rotary)(*args, q=q, q_out=rotated, cu_tokens=cu)
        (pkv.extend_q8 if q8 else pkv.extend)(rotated, *cache[:2], *scales, table_d, after_d, plan, out, cu_tokens=cu)
        at = 0
        for b, (n, a) in enumerate(zip(after, new)):
            kk, vv = gathered(table[b], n)
            # (in the 8-bit cache a later token may move the open block's scale: whole blocks stay)
            keep = lens[b] // 16 * 16 if q8 else lens[b]
            assert torch.equal(kk[:keep], held[b][0][:keep]) and torch.equal(vv[:keep], held[b][1][:keep])
            if a:
                ref, size = attention(rotated[at:at + a], kk, vv)
                # weights and output rounded to bf16; fp32 terms are far below the rest
                assert ((out[at:at + a].double() - ref).abs() <= 2.0 ** -8 * (size + ref.abs()) + 2.0 ** -16 * size).all(), b
            at += a
        assert plan.status() == 0
        return after, plan, table_d, after_d

    prompt = np.full((1, wide), -1, np.int32)
    go_on(prompt, [0], [2 * ps + 5])
    forked, copies = pool.fork(prompt, [0, 0, 0, 0], [2 * ps + 5, ps, 0, ps + 3], ps)
    assert len(copies) == 2
    pkv.copy_pages(cache, copies, ps)
    table = np.ascontiguousarray(np.concatenate([prompt, forked]))
    lens = [2 * ps + 5, 2 * ps + 5, ps, 0, ps + 3]
    history = [gathered(table[b], n) for b, n in enumerate(lens)]
    for b in (1, 2, 4):     # what the forks begin with is the prompt's
        assert all(torch.equal(x, y[:lens[b]]) for x, y in zip(history[b], history[0]))
    lens, *_ = go_on(table, lens, [3, 40, 1, 130, 0])
    lens, *_ = go_on(table, lens, [1, 5, ps, 1, 2])
    # the prompt's own session ends; the rest moves to the front
    pool.release(table[0][table[0] >= 0])
    table, lens = np.ascontiguousarray(table[1:]), lens[1:]
    before = [gathered(table[b], n) for b, n in enumerate(lens)]
    copies = pool.compact(table, ps)
    assert len(copies) > 0
    pkv.copy_pages(cache, copies, ps)
    assert table.max() < len(np.unique(table[table >= 0]))
    for b, n in enumerate(lens):
        assert all(torch.equal(x, y) for x, y in zip(gathered(table[b], n), before[b]))
    lens, plan, table_d, lens_d = go_on(table, lens, [4, 1, 60, 1])
    # and the decode reads the same cache
    q = torch.randn(4, Hq, D, device="cuda", generator=gen).bfloat16()
    out, lse = torch.empty(4, Hq, D, device="cuda"), torch.empty(4, Hq, device="cuda")
    (pkv.decode_q8 if q8 else pkv.decode)(q, *cache[:2], *scales, table_d, lens_d, plan, out, lse)
    for b, n in enumerate(lens):
        ref, size = attention(q[b:b + 1], *gathered(table[b], n))
        assert ((out[b:b + 1].double() - ref).abs() <= 2.0 ** -14 * size).all()


def test_session_and_shared_pages():
    """A session's rows may be forked and evicted; it is not compacted, and pages that are shared do not go to the device."""
    B, ps, pages = 2, 16, 16
    pool = pkv.Pool(list(range(4, pages)), pages)
    table = np.full((B, 4), -1, np.int32)
    table[0, :2], table[1, :2] = [0, 1], [2, 3]
    lens = [20, 32]
    plan = pkv.Plan(lens, table, ps, B=B, Hq=4, Hkv=1, D=64, max_pages=4, num_pages=pages, force_mode="persistent", num_splits=1)
    table_d, lens_d = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    session = pkv.Session(plan, pool, lens, table, table_d, lens_d)
    with pytest.raises(pkv.PkvError):
        pool.compact(table.copy(), ps)
    new, copies = pool.fork(session.table(), [0, 1], [20, 32], ps)
    assert new[:, :2].tolist() == [[0, 4], [2, 3]] and copies.tolist() == [[1, 4, 4]]
    with pytest.raises(pkv.PkvError):
        session.device_plan()
    session.evict([0, 1])
    assert session.free_pages()[0].tolist() == list(range(5, 16)) + [1]
    pool.release(new[new >= 0])
    session.device_plan()
    with pytest.raises(pkv.PkvError):
        pool.fork(np.zeros((1, 4), np.int32), [0], [16], ps)
