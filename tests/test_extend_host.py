"""pkv_extend without a GPU: the sharing-out of its work, its structures and what it refuses."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_kv_decode_block_gb300 import pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_decode_block_gb300", "csrc")

# Every part is walked as a CTA walks it; each block of each tile has to be covered once, in the order of the CTAs, with
# at most one shared tile at either end of a part, and the first CTA of a shared tile has to know how many there are.
WALK = r"""
#include "pkv_extend_schedule.h"
#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>
using namespace pkv;
#define REQUIRE(x) do { if (!(x)) { printf("%s (problem %d)\n", #x, it); return 1; } } while (0)
int main() {
    std::mt19937 gen(7);
    auto rnd = [&](int n) { return static_cast<int>(gen() % n); };
    for (int it = 0; it < 6000; ++it) {
        const int G = 1 << rnd(4), tt = kExtRows / G, B = 1 + rnd(9), Hkv = 1 + rnd(4), ctas = 1 + rnd(160);
        const int big = rnd(4) == 0 ? 20000 : rnd(2) ? 700 : 40;
        std::vector<int> cu{0}, len;
        for (int b = 0; b < B; ++b) {
            const int n = rnd(3) ? rnd(big) : 0, ctx = rnd(3) ? rnd(big * 4) : 0;
            cu.push_back(cu.back() + n);
            len.push_back(rnd(20) == 0 ? n - 1 : ctx + n);
        }
        std::vector<ExtRow> rows;
        std::vector<int64_t> start;
        int64_t W = 0;
        for (int b = 0; b < B; ++b) {
            rows.push_back(ext_row(cu[b], cu[b + 1], len[b], cu[B], 1 << 30, tt));
            REQUIRE(rows[b].bad == (cu[b + 1] > cu[b] && len[b] < cu[b + 1] - cu[b]));
            start.push_back(W);
            int64_t units = 0;
            for (int i = 0; i < rows[b].tiles; ++i) {
                REQUIRE(ext_units_before(rows[b], tt, i) == units);
                REQUIRE(ext_tile_at(rows[b], tt, units) == i);
                units += ext_tile_blocks(rows[b], tt, i) + kTileUnits;
                REQUIRE(ext_tile_at(rows[b], tt, units - 1) == i);
            }
            REQUIRE(rows[b].units == units);
            W += units * Hkv;
        }
        if (W == 0) continue;
        const ExtParts ps = ext_parts(W, ctas);
        const int parts = ps.parts;
        REQUIRE(parts >= 1 && parts <= ctas && ps.begin(0) == 0 && ps.begin(parts) == W);
        auto get = [&](int b) { return rows[b]; };
        std::map<std::tuple<int, int, int>, std::vector<std::pair<int, ExtPiece>>> seen;
        for (int c = 0; c < parts; ++c) {
            const int64_t first = ps.begin(c);
            REQUIRE(ps.of(first) == c && ps.of(ps.begin(c + 1) - 1) == c);
            int b0 = 0;
            while (!(start[b0] <= first && first < start[b0] + rows[b0].units * Hkv)) ++b0;
            ExtWalk w;
            w.begin(ps, c, B, Hkv, tt, b0, rows[b0], start[b0]);
            ExtPiece p;
            int begun = 0, gone_on = 0;
            while (w.next(p, get)) {
                REQUIRE(p.r.tok0 == cu[p.b] && p.r.len == len[p.b] && p.b < B && p.kvh < Hkv && p.tile < rows[p.b].tiles && p.lo < p.hi);
                begun += p.lo == 0 && p.hi < p.blocks;
                gone_on += p.lo > 0;
                seen[{p.b, p.kvh, p.tile}].push_back({c, p});
            }
            REQUIRE(begun <= 1 && gone_on <= 1);
        }
        size_t tiles = 0;
        for (int b = 0; b < B; ++b)
            for (int h = 0; h < Hkv; ++h)
                for (int i = 0; i < rows[b].tiles; ++i, ++tiles) {
                    const auto& v = seen[{b, h, i}];
                    const int nb = ext_tile_blocks(rows[b], tt, i);
                    int at = 0;
                    for (size_t k = 0; k < v.size(); ++k) {
                        const ExtPiece& p = v[k].second;
                        REQUIRE(p.lo == at && p.blocks == nb && v[k].first == v[0].first + static_cast<int>(k));
                        REQUIRE(p.parts == (k == 0 && v.size() > 1 ? static_cast<int>(v.size()) : 0));
                        at = p.hi;
                    }
                    REQUIRE(at == nb);
                }
        REQUIRE(tiles == seen.size());
    }
    // lengths at the ends of their types
    for (int G = 1, it = 0; G <= 8; G *= 2) {
        const ExtRow r = ext_row(0, 2147483647, 2147483647, 2147483647, 2147483647, kExtRows / G);
        REQUIRE(!r.bad && r.tiles > 0 && r.units > 0 && ext_tile_at(r, kExtRows / G, r.units - 1) == r.tiles - 1);
        REQUIRE(ext_row(5, 2, 9, 9, 9, 64).tiles == 0 && ext_row(-1, 2, 9, 9, 9, 64).tiles == 0);
        REQUIRE(ext_row(0, 2, -2147483647 - 1, 9, 9, 64).bad && ext_row(0, 2, 10, 9, 9, 64).bad);
    }
    puts("ok");
}
"""


def test_every_block_is_somebodys(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_struct_layout_matches_the_header(tmp_path):
    lines = ['printf("%zu\\n", sizeof(pkv_queries));']
    lines += [f'printf("%zu\\n", offsetof(pkv_queries, {f[0]}));' for f in pkv.Queries._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(pkv.Queries)] + [getattr(pkv.Queries, f[0]).offset for f in pkv.Queries._fields_]
    packed = pkv._pack_queries(1, 2, 3, 4, 5, 6, 7)
    q = pkv.Queries.from_buffer_copy(packed)
    assert [getattr(q, f[0]) for f in pkv.Queries._fields_] == [1, 2, 3, 4, 5, 6, 7]


def test_calls_without_a_plan_are_refused():
    lib, t = pkv.load(), pkv.Queries()
    assert lib.pkv_extend_reserve(None) == pkv.EINVAL
    assert lib.pkv_extend(ctypes.byref(t), None, None, None, None, None, None) == pkv.EINVAL
    assert lib.pkv_extend_q8(ctypes.byref(t), None, None, None, None, None, None, None, None) == pkv.EINVAL


def test_cpu_tensors_are_refused():
    class FakePlan:   # the checks come before the plan is used
        geom = pkv.Geom(1, 4, 1, 64, 4, 8)
        page_size, D, Hq, Hkv, handle, device = 16, 64, 4, 1, None, 0
        pool_shape, scales_shape, table_shape, rows_shape = (8, 16, 1, 64), (8, 1, 1), (1, 4), (1,)

    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pages, i = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.extend(q, pages, pages, table, i, FakePlan, q.clone())
    with pytest.raises(TypeError):
        pkv.extend_q8(q, pages, pages, i, i, table, i, FakePlan, q.clone())
    with pytest.raises(TypeError):
        pkv.extend(None, pages, pages, table, i, FakePlan, q.clone())
