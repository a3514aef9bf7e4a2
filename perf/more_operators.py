"""Attention of a chunk of new tokens over the paged cache, and the copies that fork and compact its pages, as cases
to be measured.

Three operators and one run of them together:
  extend       causal grouped-query attention of each row's new tokens over its pages of a bf16 cache
  extend_q8    the same over an e4m3 cache with one scale for each block of 16 tokens and KV head
  copy_pages   pages, or their first tokens, copied to other pages in every pool of a cache
  fork_extend  sessions forked from one prefix go on: the tail pages' copies, the rotated append, extend

`run` computes them in plain torch operations, or, where `own` is true, through this repository's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens that share a scale
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _attend(name, op, *, B, Hq, Hkv, D, ps, lens, new, fused=False, scales="pow2", rows=1):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "lens": lens, "new": new,
            "fused": fused, "scales": scales, "rows": rows}


def _copy(name, *, cache, layers, Hkv, D, ps, pages, copies, tokens, rows=1):
    return {"name": name, "op": "copy_pages", "cache": cache, "layers": layers, "Hkv": Hkv, "D": D, "ps": ps,
            "pages": pages, "copies": copies, "tokens": tokens, "rows": rows}


def listed():
    return [
        # the tiny configuration: two short rows, one KV head; all latency
        _attend("extend tiny", "extend", B=2, Hq=4, Hkv=1, D=64, ps=16, lens="37,100", new="3,17"),
        # the mixed batch, each row with a few drafted tokens to be verified: bound by reading the cache
        _attend("extend drafts", "extend", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="log:512:32768", new="5",
                rows=20260623),
        # eight prompts answered from an empty cache, queries in the fused projection's output
        _attend("extend prompts", "extend", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="0", new="log:128:4096", fused=True,
                rows=20260624),
        # the last chunk of a long prompt: one row that ends at the batch-1 configuration's length
        _attend("extend long chunk", "extend", B=1, Hq=32, Hkv=8, D=128, ps=16, lens="30720", new="2048"),
        # odd rows (no new tokens, one, around a block and a tile), eight queries a KV head, pages of three blocks
        _attend("extend odd rows", "extend", B=7, Hq=16, Hkv=2, D=64, ps=48, lens="0,4097,15,129,1000,0,0",
                new="0,1,17,33,127,1,515", fused=True),
        # 56 sessions over the 8-bit cache, four drafted tokens each
        _attend("extend q8 drafts", "extend_q8", B=56, Hq=32, Hkv=8, D=128, ps=16, lens="uniform:1024:8192", new="4",
                rows=20260623),
        # chunks of 512 tokens of eight prompts that are under way, mixed lengths
        _attend("extend q8 chunks", "extend_q8", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="log:512:16384", new="512",
                fused=True, rows=20260625),
        # odd rows over a cache quantised by somebody else, one query head a KV head
        _attend("extend q8 odd rows", "extend_q8", B=6, Hq=4, Hkv=4, D=64, ps=32, lens="0,1,2049,16,300,77",
                new="1,0,2,300,255,129", scales="amax"),
        # one session forked, one layer: its tail page
        _copy("copy one tail", cache="bf16", layers=1, Hkv=8, D=128, ps=16, pages=64, copies=1, tokens="7"),
        # 64 sessions forked inside a page, the caches of 32 layers in one call
        _copy("copy forks", cache="bf16", layers=32, Hkv=8, D=128, ps=16, pages=192, copies=64, tokens="uniform:1:16",
              rows=20260627),
        # an 8-bit cache compacted: whole pages move to the front, eight layers
        _copy("copy compaction", cache="q8", layers=8, Hkv=8, D=128, ps=64, pages=3000, copies=1237, tokens="64",
              rows=20260628),
        # 16 sessions forked from one prefix that ends inside a page, each with its own next 100 tokens
        _attend("fork and go on", "fork_extend", B=16, Hq=32, Hkv=8, D=128, ps=16, lens="1000", new="100", fused=True),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["extend", "extend", "extend_q8", "extend_q8", "copy_pages", "fork_extend"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    ps = rng.choice([16, 16, 32, 48, 64, 128])
    rows = rng.randrange(1 << 30)
    if op == "copy_pages":
        cache = rng.choice(["bf16", "q8"])   # (two pools a layer, or four)
        layers = log(1, 32 if cache == "bf16" else 16)
        copies = log(1, max(1, min(2000, (1 << 30) // (layers * ps * Hkv * D * 4))))
        c = _copy("", cache=cache, layers=layers, Hkv=Hkv, D=D, ps=ps,
                  pages=2 * copies + log(1, 256), copies=copies,
                  tokens=rng.choice(["%d" % ps, "uniform:1:%d" % ps, "uniform:0:%d" % ps]), rows=rows)
        del c["name"]
        return c
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = log(1, 64)
    # lengths within the padded size of the largest listed cache, products within those of the largest listed case
    top = max(64, min(49152, 56 * 8192 * 1024 // (B * Hkv * D)))
    hi = log(64, top)
    many = int(1.0e12 / (4.0 * Hq * D * B * hi))
    most = max(1, min(hi, 4096, many))
    short = rng.random() < 0.4
    new = log(1, max(1, min(16, most))) if short else log(1, most)
    if op == "fork_extend":
        c = _attend("", op, B=B, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lens="%d" % log(1, hi), new="%d" % new,
                    fused=rng.random() < 0.5, rows=rows)
    else:
        lens = rng.choice(["0", "uniform:0:%d" % hi, "log:1:%d" % hi])
        c = _attend("", op, B=B, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lens=lens,
                    new=rng.choice(["%d" % new, "uniform:0:%d" % new, "log:1:%d" % new]) if B > 1 else "%d" % new,
                    fused=rng.random() < 0.5, scales=rng.choice(["pow2", "amax"]), rows=rows)
    del c["name"]
    return c


def _spread(spec, count, rng):
    kind, _, rest = spec.partition(":")
    if kind in ("uniform", "log"):
        lo, hi = (int(x) for x in rest.split(":"))
        if kind == "uniform":
            return [rng.randint(lo, hi) for _ in range(count)]
        return [int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) for _ in range(count)]
    given = [int(x) for x in spec.split(",")]
    return given if len(given) == count else given * count


def _rows(case):
    """(tokens in the cache, new tokens) of each row: a matter of the case, not of the inputs' seed."""
    rng = random.Random(case["rows"])
    lens = _spread(case["lens"], case["B"], rng)
    new = _spread(case["new"], case["B"], rng)
    if not any(new):
        new[0] = 1
    return lens, new


def _copies(case):
    """[(source page, target page, tokens)]: sources and targets scattered, no page twice."""
    rng = random.Random(case["rows"])
    ids = rng.sample(range(case["pages"]), 2 * case["copies"])
    return list(zip(ids[::2], ids[1::2], _spread(case["tokens"], case["copies"], rng)))


def work(case):
    op = case["op"]
    if op == "copy_pages":
        row = case["Hkv"] * case["D"]
        one = (lambda n: n * row * 4) if case["cache"] == "bf16" else (  # noqa: E731
            lambda n: n * row * 2 + -(-n // BLOCK) * case["Hkv"] * 8)
        return {"bytes": 2 * case["layers"] * sum(one(n) for _, _, n in _copies(case)), "flops": 0}
    lens, new = _rows(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(new)
    # queries in, outputs out (bf16), lse out (fp32); keys and values of the rows that have new tokens
    nbytes = T * Hq * (2 * D * 2 + 4)
    flops = 4 * Hq * D * sum(n * a + a * (a + 1) // 2 for n, a in zip(lens, new))
    after = [n + a for n, a in zip(lens, new) if a]
    if op == "extend_q8":
        nbytes += sum(n * Hkv * D * 2 + -(-n // BLOCK) * Hkv * 8 for n in after)
    elif op == "extend":
        nbytes += sum(after) * Hkv * D * 4
    else:
        # the shared prefix once, the tails' copies out, the new tokens' keys and values in and out into the pages,
        # the rotated queries out
        nbytes += (lens[0] + len(lens) * (lens[0] % case["ps"]) + T * 2) * Hkv * D * 4 + T * Hq * D * 2
        flops += 3 * T * D * (Hq + Hkv)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _filled(pages, ps, Hkv, D, kind, gen):
    """A pool of e4m3 codes and its scales, as a cache holds them: normal values of another size in each block."""
    n = pages * ps // BLOCK
    x = torch.randn(n, BLOCK, Hkv, D, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(n, 1, Hkv, 1, device="cuda", generator=gen))
    s = x.abs().amax((1, 3)) / 448
    if kind == "pow2":
        s = torch.exp2(torch.ceil(torch.log2(s)))
    codes = (x / s[:, None, :, None]).clamp(-448, 448).to(FP8).view(pages, ps, Hkv, D)
    return codes, s.view(pages, ps // BLOCK, Hkv)


def _inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    Hkv, D, ps, op = (case[k] for k in ("Hkv", "D", "ps", "op"))
    ints = dict(dtype=torch.int32, device="cuda")
    if op == "copy_pages":
        pools = []
        for _ in range(case["layers"]):
            for _ in "kv":
                if case["cache"] == "bf16":
                    pools.append(torch.randn(case["pages"], ps, Hkv, D, device="cuda", generator=gen).bfloat16())
                else:
                    pools.extend(_filled(case["pages"], ps, Hkv, D, "pow2", gen))
        copies = _copies(case)
        return {"op": op, "ps": ps, "pools": pools, "copies": copies,
                "copies_t": torch.tensor(copies, dtype=torch.int32).view(-1, 3)}
    lens, new = _rows(case)
    B, Hq = case["B"], case["Hq"]
    after = [n + a for n, a in zip(lens, new)]
    used = [-(-n // ps) for n in after]
    pages, wide = sum(used) + 5, max(used) + 1
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    T = sum(new)
    s = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "T": T, "table": table, "lens_h": lens, "new_h": new,
         "after_h": after, "lens": torch.tensor(lens, **ints), "after": torch.tensor(after, **ints)}
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], **ints)
    if op == "extend_q8":
        s["kp"], s["ks"] = _filled(pages, ps, Hkv, D, case["scales"], gen)
        s["vp"], s["vs"] = _filled(pages, ps, Hkv, D, case["scales"], gen)
    else:
        s["kp"] = torch.randn(pages, ps, Hkv, D, device="cuda", generator=gen).bfloat16()
        s["vp"] = torch.randn(pages, ps, Hkv, D, device="cuda", generator=gen).bfloat16()
    size = torch.exp(0.5 * torch.randn(1, Hq + 2 * Hkv, 1, device="cuda", generator=gen))
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=gen) * size).bfloat16()
    parts = qkv.split([Hq, Hkv, Hkv], 1)   # views of the projection's output, or tensors of their own
    s["q"], s["k"], s["v"] = parts if case["fused"] else [x.contiguous() for x in parts]
    if op == "fork_extend":
        # row b's full pages of the prefix are the parent's, whose tail page is one more page of the pool; its own
        # tail page, which the copy fills, and those of its new tokens it has already
        whole, tail = lens[0] // ps, lens[0] % ps
        table[:, :whole] = table[0, :whole].clone()
        parent, to = order[at], table[:, whole] if tail else table[:, 0]
        s["copies_t"] = torch.stack((parent.expand(B), to, torch.full((B,), tail, **ints)), 1)[:B if tail else 0].cpu()
        s["copies"] = s["copies_t"].tolist()
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = s["op"]
    if op != "copy_pages":
        T, Hq, D = s["T"], s["Hq"], s["D"]
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(T, Hq, device="cuda")
    if op == "fork_extend":
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["new_lens"] = torch.empty_like(s["lens"])
        s["inv_freq_d"] = s["inv_freq"].cuda()
    if own:
        from paged_kv_decode_block_gb300 import pkv
        s["pkv"] = pkv
        if op != "copy_pages":
            s["plan"] = pkv.Plan(s["after_h"], None, s["ps"], B=s["B"], Hq=Hq, Hkv=s["Hkv"], D=D,
                                 max_pages=s["table"].shape[1], num_pages=s["kp"].shape[0])
            s["plan"].reserve_extend()
        if op == "fork_extend":
            s["rotary"] = pkv.Rotary(D, inv_freq=s["inv_freq"].numpy())
        if "copies_t" in s:
            s["copies_np"] = s["copies_t"].numpy()   # the page pool hands out its copies as such an array
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        pkv = s["pkv"]
        if op == "copy_pages":
            pkv.copy_pages(s["pools"], s["copies_np"], s["ps"])
        if op == "fork_extend":
            pkv.copy_pages([s["kp"], s["vp"]], s["copies_np"], s["ps"])
            pkv.append_rotary(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], s["new_lens"], s["plan"],
                              s["rotary"], q=s["q"], q_out=s["q_out"], cu_tokens=s["cu"])
        if op in ("extend", "fork_extend"):
            pkv.extend(s["q"] if op == "extend" else s["q_out"], s["kp"], s["vp"], s["table"],
                       s["after"] if op == "extend" else s["new_lens"], s["plan"], s["out"], s["lse"],
                       cu_tokens=s["cu"])
        if op == "extend_q8":
            pkv.extend_q8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["after"], s["plan"], s["out"],
                          s["lse"], cu_tokens=s["cu"])
    else:
        if op == "copy_pages":
            _plain_copy(s["pools"], s["copies"], s["ps"])
        if op == "fork_extend":
            _plain_copy([s["kp"], s["vp"]], s["copies"], s["ps"])
            _plain_append(s)
        if op != "copy_pages":
            _plain_extend(s, s["q_out"] if op == "fork_extend" else s["q"])
    if op == "copy_pages":
        return list(s["pools"])
    result = {"out": s["out"], "lse": s["lse"]}
    if op == "fork_extend":
        result.update(k_pages=s["kp"], v_pages=s["vp"], lens=s["new_lens"], q=s["q_out"])
    return result


def _plain_copy(pools, copies, ps):
    """All sources are read before any target is written, pool by pool."""
    if not copies:
        return
    for unit in sorted({ps // p.shape[1] for p in pools}):   # tokens of one entry of a page: 1, or a block's scale
        at = [(a * (ps // unit) + i, b * (ps // unit) + i) for a, b, n in copies for i in range(-(-n // unit))]
        src, dst = torch.tensor(at, dtype=torch.int64, device="cuda").view(-1, 2).unbind(1)
        for p in pools:
            if ps // p.shape[1] == unit:
                flat = p.flatten(0, 1)
                if p.dtype == FP8:
                    flat = flat.view(torch.uint8)
                flat[dst] = flat[src]


def _plain_append(s):
    """New keys and queries turned by their positions in 32 bits, the angles in 64; pages written in bf16."""
    n = s["cu"][1:] - s["cu"][:-1]
    row = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), n.long(), output_size=s["T"])
    pos = s["lens"].long()[row] + torch.arange(s["T"], device="cuda") - s["cu"].long()[row]
    s["new_lens"].copy_(s["lens"] + n)
    flat = s["table"].long()[row, pos // s["ps"]] * s["ps"] + pos % s["ps"]
    angle = pos[:, None].double() * s["inv_freq_d"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    s["q_out"].copy_(turned(s["q"]))
    s["kp"].flatten(0, 1)[flat] = turned(s["k"]).bfloat16()
    s["vp"].flatten(0, 1)[flat] = s["v"]


def _plain_extend(s, q):
    Hq, Hkv, D, ps = (s[k] for k in ("Hq", "Hkv", "D", "ps"))
    at = 0
    for b, (n, a) in enumerate(zip(s["lens_h"], s["new_h"])):
        if not a:
            continue
        here = slice(at, at + a)
        at += a
        t = torch.arange(n + a, device="cuda")
        flat = s["table"].long()[b, t // ps] * ps + t % ps
        if s["op"] == "extend_q8":
            k, v = (s[p].flatten(0, 1).view(torch.uint8)[flat].view(FP8).float() *
                    s[c].flatten(0, 1)[flat // BLOCK][..., None] for p, c in (("kp", "ks"), ("vp", "vs")))
        else:
            k, v = (s[p].flatten(0, 1)[flat].float() for p in ("kp", "vp"))
        x = q[here].float().view(a, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)           # [Hkv][G][a][D]
        score = x @ k.permute(1, 2, 0)[:, None] / math.sqrt(D)                       # [Hkv][G][a][n + a]
        seen = t <= n + torch.arange(a, device="cuda")[:, None]
        score = torch.where(seen, score, -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        o = p @ v.permute(1, 0, 2)[:, None] / total
        s["out"][here] = o.permute(2, 0, 1, 3).reshape(a, Hq, D).bfloat16()
        s["lse"][here] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(a, Hq)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Row by row and head by head, from the definitions; bf16 outputs as the values before their rounding."""
    if case["op"] == "copy_pages":
        s = _inputs(case, seed)
        result = []
        for p in s["pools"]:
            was, now, per = p.double(), p.double(), case["ps"] // p.shape[1]
            for a, b, n in s["copies"]:
                now[b, :-(-n // per)] = was[a, :-(-n // per)]
            result.append(now)
        return result
    if work(case)["flops"] > 4e12:
        return None
    s = _inputs(case, seed)
    B, Hq, Hkv, D, ps, op = (s[k] for k in ("B", "Hq", "Hkv", "D", "ps", "op"))
    lens, new = _rows(case)
    table = s["table"].cpu().tolist()
    q, k_new, v_new = s["q"].double(), s["k"].double(), s["v"].double()
    pool = {x: s[x].reshape(-1, Hkv, D) for x in ("kp", "vp")}
    result = {}
    if op == "fork_extend":
        pool = {x: p.double() for x, p in pool.items()}
        for a, b, n in s["copies"]:
            for p in pool.values():
                p[b * ps:b * ps + n] = p[a * ps:a * ps + n].clone()
        q, k_new = q.clone(), k_new.clone()
        at = 0
        for b in range(B):
            z = torch.polar(torch.ones(new[b], D // 2, dtype=torch.float64),
                            torch.arange(lens[b], lens[b] + new[b], dtype=torch.float64)[:, None] * s["inv_freq"])
            for x in (q, k_new):
                y = torch.complex(x[at:at + new[b], :, :D // 2], x[at:at + new[b], :, D // 2:]) * z.cuda()[:, None]
                x[at:at + new[b]] = torch.cat((y.real, y.imag), -1)
            rows = torch.tensor([table[b][t // ps] * ps + t % ps for t in range(lens[b], lens[b] + new[b])],
                                dtype=torch.int64, device="cuda")
            pool["kp"][rows], pool["vp"][rows] = k_new[at:at + new[b]], v_new[at:at + new[b]]
            at += new[b]
        result.update(k_pages=pool["kp"].view(s["kp"].shape), v_pages=pool["vp"].view(s["vp"].shape),
                      lens=torch.tensor([n + a for n, a in zip(lens, new)], dtype=torch.int32), q=q)
        # what the attention reads is what the queries and the cache hold: rounded to bf16
        q = q.bfloat16().double()
        pool = {x: p.bfloat16() for x, p in pool.items()}
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(B):
        n, a = lens[b] + new[b], new[b]
        if not a:
            continue
        rows = torch.tensor([table[b][t // ps] * ps + t % ps for t in range(n)], dtype=torch.int64, device="cuda")
        hidden = torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1)
        for h in range(Hkv):
            k, v = (pool[x].view(torch.uint8)[rows, h].view(FP8).double() * s[c].view(-1, Hkv)[rows // BLOCK, h, None]
                    if op == "extend_q8" else pool[x][rows, h].double() for x, c in (("kp", "ks"), ("vp", "vs")))
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = (q[at:at + a, g] @ k.T * D ** -0.5).masked_fill_(hidden, -math.inf)
                lse[at:at + a, g] = torch.logsumexp(z, 1)
                out[at:at + a, g] = torch.softmax(z, 1) @ v
        at += a
    # in the run of all three a rotated query or key may round to bf16 the other way, which moves the sum by more
    # than 32 bits do
    result.update(out=out, lse=lse if op != "fork_extend" else None)
    return result
