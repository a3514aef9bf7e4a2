"""The barriers of pkv_extend, as a model on the CPU whose counts and arrivals come from the kernel's source.

A wait for a barrier's phase names the phase's parity only: it is right as long as the barrier is in that phase or the one
behind it.  So whoever waits for `full` of a ring's place has to be among those who free it (`empty`), however late it is.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_block_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "pkv_extend.cu")) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def count(barrier, q8):
    """Arrivals of a phase, from `mbar_init(&c-><barrier>, n)` or `..., Q8 ? n : m)`."""
    init = re.search(r"mbar_init\(&c->%s, ([^;]*)\);" % re.escape(barrier), source()).group(1)
    if "?" in init:
        init = re.fullmatch(r"Q8 \? (.*) : (.*)", init).group(1 if q8 else 2)
    return eval(init, {})   # (a number or a sum of some)


def body(function):
    text = source()
    at = text.index("{", re.search(r"__device__ __forceinline__ \w+ %s\(" % function, text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]


class Barrier:
    def __init__(self, arrivals):
        self.arrivals, self.pending, self.phase = arrivals, arrivals, 0   # phase: the one that is not complete

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.arrivals, self.phase + 1


def play(actors, rng, slow):
    """Runs the actors (generators of (barrier, phase) waits) in a random order, those in `slow` seldom."""
    waits = {name: next(a) for name, a in actors.items()}
    while waits:
        for name, (barrier, phase) in waits.items():
            assert barrier.phase <= phase + 1, f"{name} waits for phase {phase}, the barrier is in {barrier.phase}"
        free = [name for name, (barrier, phase) in waits.items() if barrier.phase % 2 != phase % 2]
        assert free, "all wait: " + ", ".join(waits)
        name = rng.choice([n for n in free if n not in slow] or free)
        try:
            waits[name] = actors[name].send(None)
        except StopIteration:
            del waits[name]


@pytest.mark.parametrize("stages", [5, 10])
@pytest.mark.parametrize("slow", [[], ["cleaning"], ["cleaning", "product 1"], ["product 0"], ["loads"]])
def test_the_cleaning_warp_never_falls_a_ring_behind(stages, slow):
    """bf16: keys and values of 60 blocks, the last 3 with masked places, through the ring."""
    blocks, masked = 60, 57
    frees = "mbar_arrive(&c->empty[" in body("clean")
    full = [Barrier(count("full[i]", False)) for _ in range(stages)]
    empty = [Barrier(count("empty[i]", False)) for _ in range(stages)]
    fixed = [Barrier(count("fixed[i]", False)) for _ in range(stages)]

    def loads():
        for n in range(2 * blocks):
            if n >= stages:
                yield empty[n % stages], n // stages - 1
            full[n % stages].arrive()

    def product():
        cleaned = [0] * stages
        for n in range(2 * blocks):
            st = n % stages
            if n % 2 and n // 2 >= masked:
                yield fixed[st], cleaned[st]
                cleaned[st] += 1
            else:
                yield full[st], n // stages
            empty[st].arrive()

    def cleaning():
        for n in range(2 * blocks):
            st = n % stages
            yield full[st], n // stages
            if n % 2 and n // 2 >= masked:
                fixed[st].arrive()
            if frees:
                empty[st].arrive()

    for seed in range(20):
        for x in full + empty + fixed:
            x.pending, x.phase = x.arrivals, 0
        play({"loads": loads(), "product 0": product(), "product 1": product(), "cleaning": cleaning()}, random.Random(seed), slow)


@pytest.mark.parametrize("slow", [[], ["softmax 5"], ["softmax 4", "softmax 7"], ["softmax 0"], ["product 1"], ["loads"]])
def test_the_second_group_never_falls_two_queries_behind(slow):
    """8-bit: pieces of one block and few rows, in which the second group's warps have nothing to do but wait."""
    pieces, ring = 40, 4
    frees = "mbar_arrive(&c->q_empty)" in body("attend")
    q_full, q_empty = Barrier(count("q_full", True)), Barrier(count("q_empty", True))
    told, done = [Barrier(1) for _ in range(ring)], [Barrier(10) for _ in range(ring)]   # (the readers that matter here)
    scores, outputs = Barrier(1), Barrier(4)   # of the first group

    def loads():
        for i in range(pieces):
            if i >= ring:
                yield done[i % ring], i // ring - 1
            told[i % ring].arrive()
            if i > 0:
                yield q_empty, i - 1
            q_full.arrive()

    def product(g):
        for i in range(pieces):
            yield told[i % ring], i // ring
            done[i % ring].arrive()
            yield q_full, i
            if g == 0:
                if i > 0:
                    yield outputs, i - 1
                scores.arrive()
            q_empty.arrive()

    def softmax(g):
        for i in range(pieces):
            yield told[i % ring], i // ring
            yield q_full, i
            if frees:
                q_empty.arrive()
            if g == 0:
                yield scores, i
                outputs.arrive()
            done[i % ring].arrive()

    for seed in range(20):
        for x in [q_full, q_empty, scores, outputs] + told + done:
            x.pending, x.phase = x.arrivals, 0
        play({"loads": loads(), **{f"product {g}": product(g) for g in range(2)}, **{f"softmax {w}": softmax(w // 4) for w in range(8)}},
             random.Random(seed), slow)


def test_the_warps_roles_have_no_wait_without_a_limit():
    """A wait that runs out makes every warp return; one in a barrier of the hardware (bar.sync), which the warps that have
    returned never reach, would stay there for ever."""
    assert not re.search(r"named_barrier_sync|bar\.sync|barrier\.sync|barrier\.cta", source())
    assert source().count("mbar_try_wait(") == 1 and "mbar_try_wait(" in body("wait_for")
    for role in ("load", "load_values", "clean", "widen", "multiply", "split_query", "attend"):
        assert "__syncthreads" not in body(role), role
