// pkv_extend_schedule.h -- how the work of pkv_extend is shared out among CTAs.
//
// Plain arithmetic, compiled for the device and, by the CPU tests, for the host.
//
// Row b has n new tokens, the last n of its len.  Its G query heads of one KV
// head lie next to each other in a token, so a tile packs tile_tokens = 256 / G
// tokens x G heads into 256 rows of scores, and reads the KV blocks (128 tokens
// each) up to its last token.  Work is counted in units: one per KV block, and
// kTileUnits more per tile for what a tile costs besides (loading its queries,
// filling and draining the pipeline).  Row by row, KV head by KV head, tile by
// tile the units form one line of W, of which each of P CTAs takes an equal
// part: nothing has to be known on the host, short and long rows balance, and
// few tiles over a long cache are split.  A part begins and ends anywhere, so a
// CTA has at most two tiles that it shares with others (its first and its last):
// it leaves their partial states in its two workspace slots.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

constexpr int kExtBlock = 128;      // tokens of a KV block
constexpr int kExtBlockLog2 = 7;
constexpr int kExtRows = 256;       // rows of scores of a tile: two groups of 128
// Units of a tile besides its blocks: 8 prompts of 128-4096 take 244 / 224 / 231 us with 1 / 3 / 5, 8-bit
// chunks of 512 over 8 rows 452 / 419 / 409, 2048 tokens after 30720 725 / 724 / 722.
constexpr int kTileUnits = 3;
// A CTA takes at least this much, and fewer CTAs work otherwise: with larger shares the smallest calls
// wait longer than joining the parts takes (3 and 17 tokens after 37 and 100: 10.7 us, with larger ones 13.2).
constexpr int kMinShareUnits = 2;

struct ExtRow {
    int32_t tok0;    // the row's first new token in q / out
    int32_t n;       // its new tokens
    int32_t len;     // its tokens, the new ones among them
    int32_t tiles;   // tiles of one KV head
    int32_t bad;     // lengths that cannot be: the tiles only write NaN
    int64_t units;   // units of one KV head
};

// (tokens are counted without a sign where they are divided: shifts, not divisions)
PKV_HD uint32_t ext_blocks(uint32_t tokens) { return (tokens + (kExtBlock - 1)) >> kExtBlockLog2; }

// Blocks of the first i tiles of a row whose new tokens begin at position ctx,
// none of them its last: sum over k = 1..i of ceil((ctx + k * tt) / 128).
PKV_HD int64_t ext_blocks_before(uint32_t ctx, int tt, uint32_t i) {
    if (tt >= kExtBlock) {
        const uint64_t s = static_cast<uint32_t>(tt) >> kExtBlockLog2;
        return static_cast<int64_t>(static_cast<uint64_t>(i) * ext_blocks(ctx) + s * ((static_cast<uint64_t>(i) * (i + 1)) >> 1));
    }
    const uint32_t log2m = tt == 64 ? 1 : 2;   // 2^log2m tiles of a block: k = 2^log2m * a + r adds a to the r-th
    uint64_t sum = 0;
    for (uint32_t r = 1; r <= 1u << log2m; ++r) {
        const uint64_t cnt = i >= r ? ((i - r) >> log2m) + 1 : 0;
        sum += cnt * ext_blocks(ctx + r * tt) + ((cnt * (cnt - 1)) >> 1);
    }
    return static_cast<int64_t>(sum);
}

PKV_HD int32_t ext_tile_blocks(const ExtRow& r, int tt, int32_t i) {
    if (r.bad) return 1;
    const uint32_t upto = static_cast<uint32_t>(r.len - r.n) + static_cast<uint32_t>(i + 1) * tt, len = r.len;
    return static_cast<int32_t>(ext_blocks(upto < len ? upto : len));
}

// Units of the tiles before tile i of one KV head.
PKV_HD int64_t ext_units_before(const ExtRow& r, int tt, int32_t i) {
    if (r.bad) return static_cast<int64_t>(i) * (1 + kTileUnits);
    return ext_blocks_before(r.len - r.n, tt, i) + static_cast<int64_t>(i) * kTileUnits;
}

// Row of tokens [lo, hi) with `len` tokens in all, of T tokens and at most
// `cap` in a table.  Offsets that do not lie ascending in [0, T] leave no tiles.
PKV_HD ExtRow ext_row(int32_t lo, int32_t hi, int32_t len, int32_t T, int64_t cap, int tt) {
    ExtRow r;
    r.tok0 = lo;
    r.len = len;
    r.n = lo >= 0 && hi <= T && hi > lo ? hi - lo : 0;
    r.bad = (r.n > 0 && (len < r.n || len > cap)) ? 1 : 0;
    int shift = 8;   // tt = 2^shift, 32 to 256
    while (1 << shift > tt) --shift;
    r.tiles = static_cast<int32_t>((static_cast<uint32_t>(r.n) + tt - 1) >> shift);
    r.units = r.tiles == 0 ? 0
                           : ext_units_before(r, tt, r.tiles - 1) + ext_tile_blocks(r, tt, r.tiles - 1) + kTileUnits;
    return r;
}

// The tile of one KV head that holds unit `off` (0 <= off < units).
PKV_HD int32_t ext_tile_at(const ExtRow& r, int tt, int64_t off) {
    int32_t lo = 0, hi = r.tiles - 1;
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (ext_units_before(r, tt, mid) <= off)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// W units in equal parts for at most `ctas` CTAs: the first `rest` parts have q + 1.
struct ExtParts {
    int64_t W, q;
    int32_t parts, rest;
    PKV_HD int64_t begin(int32_t c) const { return c * q + (c < rest ? c : rest); }
    PKV_HD int32_t of(int64_t unit) const {
        return static_cast<int32_t>(unit < rest * (q + 1) ? unit / (q + 1) : rest + (unit - rest * (q + 1)) / q);
    }
};
PKV_HD ExtParts ext_parts(int64_t W, int32_t ctas) {
    ExtParts p;
    const int64_t most = W / kMinShareUnits;
    p.W = W;
    p.parts = static_cast<int32_t>(most < 1 ? 1 : (most < ctas ? most : ctas));
    if (W <= 0xffffffffll) {
        p.q = static_cast<uint32_t>(W) / static_cast<uint32_t>(p.parts);
        p.rest = static_cast<int32_t>(static_cast<uint32_t>(W) % static_cast<uint32_t>(p.parts));
    } else {
        p.q = W / p.parts;
        p.rest = static_cast<int32_t>(W % p.parts);
    }
    return p;
}

// One CTA's stretch of one tile.
struct ExtPiece {
    int32_t b, kvh, tile;
    int32_t lo, hi;    // its KV blocks
    int32_t blocks;    // the tile's
    int32_t parts;     // lo == 0 and hi < blocks: CTAs (from this one on) that share the tile; else 0
    ExtRow r;          // its row
};

// Walks one CTA's part of the line.  `rows` gives ExtRow by index.
struct ExtWalk {
    ExtParts ps;
    int64_t unit, first, end;   // unit: the current tile's first
    int32_t cta, B, Hkv, tt;
    int32_t b, kvh, tile;
    ExtRow r;

    // The part of `cta`, which begins in row b0 = `row`, whose first unit is row_unit.
    PKV_HD void begin(const ExtParts& parts, int32_t cta_, int32_t B_, int32_t Hkv_, int tt_, int32_t b0, const ExtRow& row,
                      int64_t row_unit) {
        ps = parts, cta = cta_, B = B_, Hkv = Hkv_, tt = tt_;
        first = ps.begin(cta);
        end = ps.begin(cta + 1);
        b = b0;
        r = row;
        unit = row_unit;
        for (kvh = 0; first - unit >= r.units; ++kvh) unit += r.units;
        tile = ext_tile_at(r, tt, first - unit);
        unit += ext_units_before(r, tt, tile);
    }

    // The next stretch with blocks in it; false at the end of the part.
    template <class Rows>
    PKV_HD bool next(ExtPiece& p, const Rows& rows) {
        while (unit < end) {
            const int32_t nb = ext_tile_blocks(r, tt, tile);
            const int64_t b0 = unit + kTileUnits;   // the unit of block 0
            p.b = b, p.kvh = kvh, p.tile = tile, p.blocks = nb, p.parts = 0, p.r = r;
            p.lo = first > b0 ? static_cast<int32_t>(first - b0) : 0;
            p.hi = end < b0 + nb ? static_cast<int32_t>(end - b0) : nb;
            if (p.lo == 0 && p.hi > 0 && p.hi < nb) p.parts = ps.of(b0 + nb - 1) - cta + 1;
            unit = b0 + nb;
            if (++tile == r.tiles) {
                tile = 0;
                if (++kvh == Hkv) {
                    kvh = 0;
                    do ++b;
                    while (unit < end && b < B && (r = rows(b)).tiles == 0);
                }
            }
            if (p.hi > p.lo) return true;
        }
        return false;
    }
};

}  // namespace pkv
