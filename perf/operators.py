"""The paged 8-bit KV cache's operators and the rotated append, as cases to be measured.

Three operators and one run of them together:
  append_rotary  new keys and values, rotated by their positions, into a bf16 paged cache (queries rotated on the way)
  append_q8      the same into an e4m3 paged cache with one scale for each block of 16 tokens and KV head
  decode_q8      single-token grouped-query attention over that e4m3 cache
  step_q8        one decode step of continuous sessions: append_q8, the re-planning, decode_q8

`run` computes them in plain torch operations, or, where `own` is true, through this repository's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens that share a scale
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _case(name, op, *, B, Hq, Hkv, D, ps, lens, new="1", rot=0, interleaved=False, base=10000.0, fused=False,
          scales="pow2", rows=1):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "lens": lens, "new": new,
            "rot": rot, "interleaved": interleaved, "base": base, "fused": fused, "scales": scales, "rows": rows}


def listed():
    return [
        # the tiny configuration: two short rows, one KV head; all latency
        _case("decode tiny", "decode_q8", B=2, Hq=4, Hkv=1, D=64, ps=16, lens="37,100"),
        # one long context being answered: the batch-1 configuration
        _case("decode batch-1 32k", "decode_q8", B=1, Hq=32, Hkv=8, D=128, ps=16, lens="32768"),
        # a mixed batch of short and long contexts
        _case("decode mixed", "decode_q8", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="log:512:32768", rows=20260623),
        # a full server: many equal contexts
        _case("decode high batch", "decode_q8", B=64, Hq=32, Hkv=8, D=128, ps=16, lens="4096"),
        # odd rows (empty, one token, around a block), eight queries a KV head, a cache quantised by somebody else
        _case("decode odd rows", "decode_q8", B=7, Hq=16, Hkv=2, D=64, ps=32, lens="0,1,15,16,17,1000,4097",
              scales="amax"),
        # one session's next token, nothing else on the GPU
        _case("append one", "append_rotary", B=1, Hq=32, Hkv=8, D=128, ps=16, lens="32767", rot=128),
        # a decode step of 56 sessions, from the fused projection's output
        _case("append step", "append_rotary", B=56, Hq=32, Hkv=8, D=128, ps=16, lens="uniform:1024:8192", rot=128,
              fused=True, rows=20260623),
        # eight prompts enter the cache
        _case("append prompts", "append_rotary", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="0", new="log:128:4096",
              rot=128, fused=True, rows=20260624),
        # a decode step of 64 sessions into the 8-bit cache
        _case("append q8 step", "append_q8", B=64, Hq=32, Hkv=8, D=128, ps=16, lens="log:512:32768", rot=128,
              fused=True, rows=20260625),
        # chunks of eight prompts go on where the last chunk ended, inside a block
        _case("append q8 prompts", "append_q8", B=8, Hq=32, Hkv=8, D=128, ps=16, lens="uniform:1:512",
              new="log:128:4096", rot=128, fused=True, rows=20260626),
        # far positions, half of the head rotated in neighbouring pairs, rows of zero to a few new tokens
        _case("append q8 far", "append_q8", B=5, Hq=8, Hkv=1, D=64, ps=48, lens="200003,131071,77777,9,0",
              new="0,1,7,16,33", rot=32, interleaved=True, base=500000.0),
        # the continuous sessions' whole step over the 8-bit cache
        _case("step 56 sessions", "step_q8", B=56, Hq=32, Hkv=8, D=128, ps=16, lens="uniform:1024:8192", rot=128,
              fused=True, rows=20260623),
    ]


def draw(rng):
    op = rng.choice(["decode_q8", "decode_q8", "append_rotary", "append_q8", "step_q8"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    ps = rng.choice([16, 16, 32, 48, 64])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    B = log(1, 64)
    # the longest row: within the padded size of the largest listed case
    top = max(2, min(65536, 64 * 4096 * 1024 // (B * Hkv * D)))
    hi = log(64, top)
    kind = rng.choice(["uniform", "log"])
    lens = "%s:%d:%d" % (kind, rng.choice([0 if kind == "uniform" and B > 1 else 1, 1, hi // 8]), hi)
    new = "1"
    if op.startswith("append") and rng.random() < 0.6:
        new = "log:1:%d" % log(2, min(4096, max(2, 8192 // B)))
    rot = rng.choice([r for r in (16, 32, 64, 128) if r <= D])
    c = _case("", op, B=B, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lens=lens, new=new, rot=0 if op == "decode_q8" else rot,
              interleaved=rng.random() < 0.4, base=rng.choice([10000.0, 500000.0]), fused=rng.random() < 0.5,
              scales=rng.choice(["pow2", "amax"]), rows=rng.randrange(1 << 30))
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
    new = _spread(case["new"], case["B"], rng) if case["op"] != "decode_q8" else [0] * case["B"]
    return lens, new


def work(case):
    lens, new = _rows(case)
    Hq, Hkv, D, op = case["Hq"], case["Hkv"], case["D"], case["op"]
    nbytes, flops, T = 0, 0, sum(new)
    if op != "decode_q8":
        # queries in and out, keys and values in (bf16), and out into the pages
        nbytes += T * (2 * Hq * D * 2 + 2 * Hkv * D * (2 + (2 if op == "append_rotary" else 1)))
        flops += 3 * T * case["rot"] * (Hq + Hkv)
    if op in ("append_q8", "step_q8"):
        nbytes += sum(math.ceil((n % BLOCK + a) / BLOCK) if a else 0 for n, a in zip(lens, new)) * Hkv * 8
    if op in ("decode_q8", "step_q8"):
        after = [n + a for n, a in zip(lens, new)]
        nbytes += sum(n * Hkv * D * 2 + math.ceil(n / BLOCK) * Hkv * 8 for n in after)
        nbytes += case["B"] * Hq * (D * 2 + D * 4 + 4)
        flops += 4 * sum(after) * Hq * D
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _power_of_two(amax):
    """The least power of two s (from 2^-120 to 2^120) with amax / s <= 448, as a float32 tensor."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -120)).clamp(-120, 120)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _filled(pages, ps, Hkv, D, kind, gen):
    """A pool of e4m3 codes and its scales, as a cache holds them: normal values of another size in each block."""
    n = pages * ps // BLOCK
    x = torch.randn(n, BLOCK, Hkv, D, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(n, 1, Hkv, 1, device="cuda", generator=gen))
    amax = x.abs().amax((1, 3))
    s = _power_of_two(amax) if kind == "pow2" else amax / 448
    codes = (x / s[:, None, :, None]).clamp(-448, 448).to(FP8).view(pages, ps, Hkv, D)
    return codes, s.view(pages, ps // BLOCK, Hkv)


def _inputs(case, seed):
    lens, new = _rows(case)
    B, Hq, Hkv, D, ps, op = (case[k] for k in ("B", "Hq", "Hkv", "D", "ps", "op"))
    gen = torch.Generator("cuda").manual_seed(int(seed))
    after = [n + a for n, a in zip(lens, new)]
    used = [-(-n // ps) for n in after]
    pages, wide = sum(used) + 4, max(used) + 1
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    T = sum(new) if op != "decode_q8" else B
    ints = dict(dtype=torch.int32, device="cuda")
    s = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "T": T, "table": table, "lens_h": lens,
         "after_h": after, "lens": torch.tensor(lens, **ints), "interleaved": case["interleaved"], "rot": case["rot"]}
    if op == "append_rotary":
        s["kp"] = torch.randn(pages, ps, Hkv, D, device="cuda", generator=gen).bfloat16()
        s["vp"] = torch.randn(pages, ps, Hkv, D, device="cuda", generator=gen).bfloat16()
    else:
        s["kp"], s["ks"] = _filled(pages, ps, Hkv, D, case["scales"], gen)
        s["vp"], s["vs"] = _filled(pages, ps, Hkv, D, case["scales"], gen)
    size = torch.exp(0.5 * torch.randn(1, Hq + 2 * Hkv, 1, device="cuda", generator=gen))
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=gen) * size).bfloat16()
    parts = qkv.split([Hq, Hkv, Hkv], 1)   # views of the projection's output, or tensors of their own
    s["q"], s["k"], s["v"] = parts if case["fused"] else [x.contiguous() for x in parts]
    if op != "decode_q8":
        s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], **ints) if case["new"] != "1" else None
        s["inv_freq"] = case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
        # the scheduler's knowledge: the rows whose new tokens begin inside a block that holds tokens already
        s["open"] = torch.tensor([b for b in range(B) if lens[b] % BLOCK and new[b]], dtype=torch.int64, device="cuda")
        s["base"] = case["base"]
    else:
        s["q"] = s["q"].contiguous()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    B, Hq, Hkv, D, T, op = (s[k] for k in ("B", "Hq", "Hkv", "D", "T", "op"))
    if op != "decode_q8":
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["new_lens"] = torch.empty_like(s["lens"])
        s["inv_freq_d"] = s["inv_freq"].cuda()
    if op in ("decode_q8", "step_q8"):
        s["out"] = torch.empty(B, Hq, D, device="cuda")
        s["lse"] = torch.empty(B, Hq, device="cuda")
    if own:
        from paged_kv_decode_block_gb300 import pkv
        s["pkv"] = pkv
        s["plan"] = pkv.Plan(s["after_h"], None, s["ps"], B=B, Hq=Hq, Hkv=Hkv, D=D, max_pages=s["table"].shape[1],
                             num_pages=s["kp"].shape[0])
        if op != "decode_q8":
            s["rotary"] = pkv.Rotary(s["rot"], inv_freq=s["inv_freq"].numpy(), interleaved=s["interleaved"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        pkv = s["pkv"]
        if op == "append_rotary":
            pkv.append_rotary(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], s["new_lens"], s["plan"],
                              s["rotary"], q=s["q"], q_out=s["q_out"], cu_tokens=s["cu"])
        if op in ("append_q8", "step_q8"):
            pkv.append_q8(s["k"], s["v"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"], s["new_lens"],
                          s["plan"], rotary=s["rotary"], q=s["q"], q_out=s["q_out"], cu_tokens=s["cu"])
        if op == "step_q8":
            s["plan"].update(s["after_h"])
        if op in ("decode_q8", "step_q8"):
            pkv.decode_q8(s["q"] if op == "decode_q8" else s["q_out"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"],
                          s["lens"] if op == "decode_q8" else s["new_lens"], s["plan"], s["out"], s["lse"])
    else:
        if op == "append_rotary":
            _plain_append(s)
        if op in ("append_q8", "step_q8"):
            _plain_append_q8(s)
        if op in ("decode_q8", "step_q8"):
            _plain_decode(s, s["q"] if op == "decode_q8" else s["q_out"],
                          s["lens"] if op == "decode_q8" else s["new_lens"])
    result = {}
    if op != "decode_q8":
        result.update(k_pages=s["kp"], v_pages=s["vp"], lens=s["new_lens"], q=s["q_out"])
    if op in ("append_q8", "step_q8"):
        result.update(k_scales=s["ks"], v_scales=s["vs"])
    if op == "decode_q8":
        result.update(out=s["out"], lse=s["lse"])
    if op == "step_q8":   # the output projection that comes next takes bf16
        result.update(out=s["out"].bfloat16(), lse=s["lse"])
    return result


def _places(s):
    """Of each new token: its position, and its token row in the pool."""
    B, T, ps = s["B"], s["T"], s["ps"]
    if s["cu"] is None:
        row, pos = torch.arange(B, device="cuda"), s["lens"].long()
        s["new_lens"].copy_(s["lens"] + 1)
    else:
        n = s["cu"][1:] - s["cu"][:-1]
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), n.long(), output_size=T)
        pos = s["lens"].long()[row] + torch.arange(T, device="cuda") - s["cu"].long()[row]
        s["new_lens"].copy_(s["lens"] + n)
    return pos, s["table"].long()[row, pos // ps] * ps + pos % ps


def _rotated(s, x, pos):
    """x (bf16 [T][heads][D]) turned by its tokens' positions, in 32 bits; the angles in 64."""
    rot = s["rot"]
    angle = pos[:, None].double() * s["inv_freq_d"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    pos, flat = _places(s)
    s["q_out"].copy_(_rotated(s, s["q"], pos))
    s["kp"].flatten(0, 1)[flat] = _rotated(s, s["k"], pos).bfloat16()
    s["vp"].flatten(0, 1)[flat] = s["v"]


def _plain_append_q8(s):
    pos, flat = _places(s)
    s["q_out"].copy_(_rotated(s, s["q"], pos))
    _plain_store(s, _rotated(s, s["k"], pos), s["kp"], s["ks"], flat)
    _plain_store(s, s["v"].float(), s["vp"], s["vs"], flat)


def _plain_store(s, x, pages, scales, flat):
    """Quantises x (fp32 [T][Hkv][D]) into the pool rows `flat`: a block's scale is the least power of two that holds
    its new tokens, but not below the scale of the tokens that it holds already, which are requantised to it."""
    codes = pages.flatten(0, 1).view(torch.uint8)
    scale = scales.flatten(0, 1)
    blk = flat // BLOCK
    amax = torch.zeros_like(scale).index_reduce_(0, blk, x.abs().amax(-1), "amax")
    grown = _power_of_two(amax)
    # the block that each open row goes on with
    tail = s["lens"].long()[s["open"]]
    first = s["table"].long()[s["open"], tail // s["ps"]] * s["ps"] + tail % s["ps"]
    held, count = first // BLOCK, first % BLOCK
    old = scale[held]
    grown[held] = torch.maximum(grown[held], old)
    scale[blk] = grown[blk]
    slots = torch.arange(BLOCK, device="cuda")
    at = held[:, None] * BLOCK + slots
    before = codes[at]
    again = (before.view(FP8).float() * (old / grown[held])[:, None, :, None]).to(FP8).view(torch.uint8)
    codes[at] = torch.where((slots < count[:, None])[..., None, None], again, before)
    codes[flat] = (x / scale[blk][..., None]).to(FP8).view(torch.uint8)


def _plain_decode(s, q, lens):
    B, Hq, Hkv, D, ps = (s[k] for k in ("B", "Hq", "Hkv", "D", "ps"))
    G = Hq // Hkv
    t = torch.arange(max(max(s["after_h"]), 1), device="cuda")
    live = t < lens[:, None]
    row = torch.where(live, s["table"].long()[:, t // ps] * ps + t % ps, 0)   # [B][L]
    k = s["kp"].flatten(0, 1).view(torch.uint8)[row].view(FP8).float() * s["ks"].flatten(0, 1)[row // BLOCK][..., None]
    score = q.float().view(B, Hkv, G, D) @ k.permute(0, 2, 3, 1) / math.sqrt(D)
    del k
    score = torch.where(live[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    some = top > -math.inf
    p = torch.exp(score - torch.where(some, top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = s["vp"].flatten(0, 1).view(torch.uint8)[row].view(FP8).float() * s["vs"].flatten(0, 1)[row // BLOCK][..., None]
    out = p @ torch.where(live[..., None, None], v, 0.0).permute(0, 2, 1, 3)
    s["out"].copy_((out / torch.where(some, total, 1.0)).view(B, Hq, D))
    s["lse"].copy_((top + torch.log(total)).view(B, Hq))


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Row by row, from the definitions; 8-bit and bf16 outputs as the values before their rounding."""
    s = _inputs(case, seed)
    B, Hq, Hkv, D, ps, op = (s[k] for k in ("B", "Hq", "Hkv", "D", "ps", "op"))
    lens, new = _rows(case)
    table = s["table"].cpu().tolist()
    place = lambda b, lo, hi: torch.tensor([table[b][p // ps] * ps + p % ps for p in range(lo, hi)],  # noqa: E731
                                           dtype=torch.int64, device="cuda")
    result = {}
    q = s["q"].double()
    pool = {x: s[x].reshape(-1, Hkv, D).double() for x in ("kp", "vp")}
    scale = {x: s[x].reshape(-1, Hkv).double() for x in ("ks", "vs") if x in s}
    if op != "decode_q8":
        rot, half = s["rot"], s["rot"] // 2
        first = torch.arange(half) * 2 if s["interleaved"] else torch.arange(half)
        second = first + 1 if s["interleaved"] else first + half

        def turn(x, pos):
            w = torch.polar(torch.ones(len(pos), half, dtype=torch.float64),
                            torch.tensor(pos, dtype=torch.float64)[:, None] * s["inv_freq"]).cuda()
            y = x.clone()
            z = torch.complex(x[..., first], x[..., second]) * w[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        q, at = q.clone(), 0
        for b in range(B):
            n, pos = new[b], list(range(lens[b], lens[b] + new[b]))
            if not n:
                continue
            here = slice(at, at + n)
            q[here] = turn(q[here], pos)
            rows = place(b, pos[0], pos[-1] + 1)
            for src, pages, sc in ((turn(s["k"][here].double(), pos), "kp", "ks"), (s["v"][here].double(), "vp", "vs")):
                if op == "append_rotary":
                    pool[pages][rows] = src
                    continue
                for lo in range(pos[0] - pos[0] % BLOCK, pos[-1] + 1, BLOCK):
                    a, z = max(lo, pos[0]), min(lo + BLOCK, pos[-1] + 1)
                    x = src[a - pos[0]:z - pos[0]]
                    block = int(rows[a - pos[0]]) // BLOCK
                    peak = x.abs().amax((0, 2))
                    e = torch.ceil(torch.log2(peak / 448))
                    e = torch.where(torch.exp2(e - 1) * 448 >= peak, e - 1, e)   # log2 next to a whole number
                    e = torch.where(torch.exp2(e) * 448 < peak, e + 1, e)
                    size = torch.exp2(e.clamp(-120, 120))
                    if a > lo:
                        size = torch.maximum(size, scale[sc][block])
                        pool[pages][block * BLOCK:block * BLOCK + a - lo] *= (scale[sc][block] / size)[:, None]
                    scale[sc][block] = size
                    pool[pages][rows[a - pos[0]:z - pos[0]]] = x / size[:, None]
            at += n
        result.update(k_pages=pool["kp"].view(s["kp"].shape), v_pages=pool["vp"].view(s["vp"].shape),
                      lens=torch.tensor([n + a for n, a in zip(lens, new)], dtype=torch.int32), q=q)
        if scale:
            result.update(k_scales=scale["ks"].view(s["ks"].shape), v_scales=scale["vs"].view(s["vs"].shape))
    if op in ("decode_q8", "step_q8"):
        if op == "step_q8":   # what the attention reads is what the cache holds: rounded to 8 bits
            q = q.bfloat16().double()
            pool = {x: p.to(FP8).double() for x, p in pool.items()}
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = lens[b] + new[b]
            if not n:
                continue
            rows = place(b, 0, n)
            k = pool["kp"][rows] * scale["ks"][rows // BLOCK][..., None]
            v = pool["vp"][rows] * scale["vs"][rows // BLOCK][..., None]
            for h in range(Hkv):
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                z = (k[:, h] @ q[b, heads].T) * D ** -0.5
                lse[b, heads] = torch.logsumexp(z, 0)
                out[b, heads] = torch.softmax(z, 0).T @ v[:, h]
        # in a step a rotated query may round to bf16 the other way, which moves the sum by more than 32 bits do
        result.update(out=out, lse=lse if op == "decode_q8" else None)
    return result
