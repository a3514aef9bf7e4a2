"""Pages with several users: pkv_pool_fork, pkv_pool_release, pkv_pool_compact, and what pkv_copy_pages refuses, on the CPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from paged_kv_decode_block_gb300 import pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Model:
    """A cache as a dictionary: what each page's slots hold.  Rows are lists of tokens."""

    def __init__(self, pages, ps):
        self.ps, self.slots = ps, [[None] * ps for _ in range(pages)]

    def copy(self, copies):
        new = [(dst, self.slots[src][:n]) for src, dst, n in copies.tolist()]
        for dst, tokens in new:
            self.slots[dst][:len(tokens)] = tokens

    def write(self, row, tokens):
        for i, t in enumerate(tokens):
            self.slots[row[i // self.ps]][i % self.ps] = t

    def read(self, row, n):
        return [self.slots[row[i // self.ps]][i % self.ps] for i in range(n)]


def test_fork_shares_whole_pages_and_copies_the_tail():
    pool = pkv.Pool([7, 3, 9, 1], num_pages=10)
    table = np.array([[4, 5, 6, -1], [8, -1, -1, -1]], np.int32)
    new, copies = pool.fork(table, [0, 0, 1, 1], [40, 32, 0, 3], 16)
    assert new.tolist() == [[4, 5, 7, -1], [4, 5, -1, -1], [-1] * 4, [3, -1, -1, -1]]
    assert copies.tolist() == [[6, 7, 8], [8, 3, 3]]
    assert pool.free_count() == 2
    pool.release([4, 5])                      # the parent's uses
    pool.release([5, 4])
    assert pool.free_count() == 2
    pool.release([4, 7])                      # the last use of 4, the only one of 7
    assert pool.free_count() == 4
    with pytest.raises(pkv.PkvError):
        pool.release([4])
    pool.release([5])
    assert pool.free_count() == 5


def test_release_of_more_uses_than_there_are_changes_nothing():
    pool = pkv.Pool([0], num_pages=4)
    pool.fork(np.array([[2]], np.int32), [0, 0], [16, 16], 16)   # page 2: three users
    for pages in ([2, 2, 2, 2], [1, 2, 2, 2, 1], [2, 0], [3, 2, 3]):
        with pytest.raises(pkv.PkvError) as e:
            pool.release(pages)
        assert e.value.code == pkv.EINVAL and pool.free_count() == 1
    pool.release([2, 1, 2, 2])
    assert pool.free_count() == 3
    table = np.full((3, 1), -1, np.int32)
    pool.reserve([0, 0, 0], table, 16)
    assert table[:, 0].tolist() == [0, 1, 2]  # in the order in which they became free


def test_fork_refusals_change_nothing():
    pool = pkv.Pool([7, 3], num_pages=10)
    table = np.array([[4, 5, -1], [7, 2, 11]], np.int32)
    for parents, lens in (([2], [1]), ([-1], [1]), ([0], [-1]), ([0], [49]), ([0], [33]), ([1], [1]), ([0, 1], [16, 48])):
        with pytest.raises(pkv.PkvError) as e:
            pool.fork(table, parents, lens, 16)
        assert e.value.code == pkv.EINVAL, (parents, lens)
    with pytest.raises(pkv.PkvError) as e:
        pool.fork(table, [0, 0, 0], [17, 18, 19], 16)
    assert e.value.code == pkv.ENOSPACE
    assert pool.free_count() == 2
    pool.release([4, 5])                      # each has one user still
    with pytest.raises(ValueError):
        pool.fork(table, [0, 0], [16], 16)
    lib, n = pkv.load(), ctypes.c_int32(0)
    t = np.array([[4, 5, -1]] * 2, np.int32)
    p = t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    rows, lens, copies = (np.zeros(6, np.int32) for _ in range(3))
    r, ln = (x.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for x in (rows, lens))
    assert lib.pkv_pool_fork(pool._h, p, 2, r, ln, 1, 3, 16, p, copies.ctypes.data, ctypes.byref(n)) == pkv.EINVAL   # overlap
    assert lib.pkv_pool_fork(None, p, 2, r, ln, 1, 3, 16, p, copies.ctypes.data, ctypes.byref(n)) == pkv.EINVAL
    assert lib.pkv_pool_fork(pool._h, p, 2, r, ln, 1, 3, 16, None, copies.ctypes.data, ctypes.byref(n)) == pkv.EINVAL
    assert lib.pkv_pool_compact(None, p, 2, 3, 16, None, 0, ctypes.byref(n)) == pkv.EINVAL


def test_compact_moves_pages_to_the_front():
    pool = pkv.Pool([0, 2, 5], num_pages=8)
    table = np.array([[7, 1, -1], [6, 3, 4]], np.int32)
    copies = pool.compact(table, 16)
    assert table.tolist() == [[2, 1, -1], [0, 3, 4]]
    assert sorted(copies.tolist()) == [[6, 0, 16], [7, 2, 16]]
    fresh = np.full((3, 1), -1, np.int32)
    pool.reserve([0, 0, 0], fresh, 16)
    assert fresh[:, 0].tolist() == [5, 6, 7]
    assert len(pool.compact(np.concatenate([table.ravel(), fresh.ravel()])[None].copy(), 16)) == 0


def test_compact_refusals_change_nothing():
    pool = pkv.Pool([0, 2], num_pages=6)
    table = np.array([[1, 3, -1], [4, 5, -1]], np.int32)
    for bad in ([[1, 3, -1], [4, -1, -1]], [[1, 3, 3], [4, 5, -1]], [[1, 3, 0], [4, 5, -1]], [[1, 3, 6], [4, 5, -1]]):
        t = np.array(bad, np.int32)
        with pytest.raises(pkv.PkvError) as e:
            pool.compact(t, 16)
        assert e.value.code == pkv.EINVAL and t.tolist() == bad
    n = ctypes.c_int32(0)
    p = table.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    copies = np.zeros((2, 3), np.int32)
    lib = pkv.load()
    assert lib.pkv_pool_compact(pool._h, p, 2, 3, 16, copies.ctypes.data, 1, ctypes.byref(n)) == pkv.ENOSPACE and n.value == 2
    assert table.tolist() == [[1, 3, -1], [4, 5, -1]] and pool.free_count() == 2
    with pytest.raises(TypeError):
        pool.compact(table.astype(np.int64), 16)
    assert len(pool.compact(table, 16)) == 2


@pytest.mark.parametrize("seed", range(4))
def test_rows_keep_their_tokens_through_forks_growth_and_compaction(seed):
    """Random sessions against rows held as lists: fork, grow, end, compact."""
    rng = np.random.default_rng(seed)
    ps, pages, wide = 4, 60, 12
    pool, cache = pkv.Pool(rng.permutation(pages).astype(np.int32), pages), Model(pages, ps)
    table, rows, stamp = np.full((0, wide), -1, np.int32), [], 0
    for _ in range(300):
        kind = rng.integers(0, 10)
        if kind < 2 and len(rows) < 8:                       # a new session
            table = np.concatenate([table, np.full((1, wide), -1, np.int32)])
            rows.append([])
        elif kind < 4 and rows:                              # forks, the same parent several times among them
            parents = rng.integers(0, len(rows), rng.integers(1, 4))
            lens = [int(rng.integers(0, len(rows[p]) + 1)) for p in parents]
            try:
                new, copies = pool.fork(table, parents, lens, ps)
            except pkv.PkvError as e:
                assert e.code == pkv.ENOSPACE
                continue
            cache.copy(copies)
            table = np.concatenate([table, new])
            rows += [rows[p][:n] for p, n in zip(parents, lens)]
        elif kind < 8 and rows:                              # every row grows by a token
            table = np.ascontiguousarray(table)
            at = np.array([len(r) for r in rows], np.int32)
            if at.max() >= wide * ps:
                continue
            try:
                pool.reserve(at, table, ps)
            except pkv.PkvError as e:
                assert e.code == pkv.ENOSPACE
                kind = 8
            else:
                for b, r in enumerate(rows):
                    stamp += 1
                    r.append(stamp)
                    cache.slots[table[b, (len(r) - 1) // ps]][(len(r) - 1) % ps] = stamp
        if kind == 8 and rows:                               # a session ends
            b = int(rng.integers(0, len(rows)))
            pool.release(table[b][table[b] >= 0])
            table, rows = np.delete(table, b, 0), rows[:b] + rows[b + 1:]
        elif kind == 9:
            table = np.ascontiguousarray(table)
            cache.copy(pool.compact(table, ps))
            used = np.unique(table[table >= 0])
            assert used.tolist() == list(range(len(used))) and pool.free_count() == pages - len(used)
        for b, r in enumerate(rows):
            assert cache.read(table[b], len(r)) == r
        assert pool.free_count() == pages - len(np.unique(table[table >= 0]))


def test_struct_layouts_match_the_header(tmp_path):
    lines = []
    for name, cls in (("pkv_page_copy", pkv.PageCopy), ("pkv_page_pool", pkv.PagePool)):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in (pkv.PageCopy, pkv.PagePool):
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want


@pytest.mark.parametrize("many", [False, True])
def test_copies_refused_before_a_device_is_touched(many):
    lib = pkv.load()
    rest = [(100 + 2 * i, 101 + 2 * i, 1) for i in range(40)] if many else []   # (beyond 32 copies another check)

    def call(copies, num_pages=200, page_size=16, data=4096, page_bytes=512, unit=1, n_pools=1):
        c = np.array(copies + rest, np.int32).reshape(-1, 3)
        p = pkv.PagePool(data, page_bytes, unit)
        return lib.pkv_copy_pages(ctypes.byref(p), n_pools, c.ctypes.data, len(c), num_pages, page_size, None)

    for bad in ([(0, 200, 1)], [(-1, 2, 1)], [(200, 2, 1)], [(0, -1, 1)], [(0, 1, 17)], [(0, 1, -1)], [(3, 3, 2)],
                [(0, 1, 2), (5, 1, 3)], [(0, 1, 2), (1, 2, 3)], [(1, 2, 2), (0, 1, 3)]):
        assert call(bad) == pkv.EINVAL, bad
    good = [(0, 1, 2), (0, 3, 16)]
    for bad in (dict(num_pages=0), dict(page_size=0), dict(data=0), dict(data=4098), dict(page_bytes=0), dict(page_bytes=520),
                dict(page_bytes=96), dict(unit=0), dict(unit=5), dict(unit=257), dict(n_pools=-1), dict(page_bytes=1 << 25)):
        assert call(good, **bad) == pkv.EINVAL, bad
    assert lib.pkv_copy_pages(None, 1, None, 0, 8, 16, None) == pkv.EINVAL
    if not many:
        assert call(good, n_pools=0) == pkv.OK and call([]) == pkv.OK   # nothing to do


def test_cpu_tensors_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for bad in ([torch.zeros(4, 16, 2, 64)], [None], [np.zeros((4, 16))]):
        with pytest.raises(TypeError):
            pkv.copy_pages(bad, [(0, 1, 2)], 16)
    with pytest.raises(ValueError):
        pkv.copy_pages([], [(0, 1)], 16)
    with pytest.raises(TypeError):
        pkv.copy_pages([], [(0.5, 1, 2)], 16)
    pkv.copy_pages([], [(0, 1, 2)], 16)
