// pkv_attention_q8.cu -- paged GQA decode attention over an e4m3 cache with one
// scale per 16-token block and KV head.
//
// The method, the tiles and the merges are those of pkv_attention.cu
// ("PersistentKV: Page-Aware Decode Scheduling for Long-Context LLM Serving on
// Commodity GPUs", gist.science summary, Methodology section 1); the plan is
// the same object, and every route and merge of it runs.
//
// Mathematics.  With codes k, v and block scales ks, vs of token t's block B:
//     s_t = (ks_B * log2(e) / sqrt(D)) * <q, k_t>,   out = sum_t 2^(s_t - m) vs_B v_t / sum_t 2^(s_t - m).
// e4m3 codes are exact in f16, so both products run on f16 tensor cores
// (mma.m16n8k16, fp32 accumulation).  q (bf16) is scaled per head by the power
// of two that brings its largest element to [1, 2), so it is exact in f16 down to
// 2^-14 of that element and rounded by at most 2^-25 of it below.  A query head has
// two references: m for its weights 2^(s - m), fp32, and m - lift for what goes into
// O, because a light token may lie in a block of large scale and the heaviest in one
// of small scale.  w = 2^(s - m + lift) * vs_B is split into f16 hi + 2^-11 lo, 22
// bits, and 2^-36 is the least that is not rounded to zero; the parts are columns of
// the products' right operand (with G = 8, of a second one).  Statistics and sums are
// fp32.  The references follow their running maxima lazily: w may grow to 2^14 (within
// f16) before O moves to a reference that puts the block's largest w at 2^6 or more,
// so what a token adds whose w is 2^42 times smaller than the largest is still there.
//
// What bounds it: HBM, 2 * D + 1/2 bytes per token and KV head against 4 * G * D
// flops (2 G flop per byte).  Measured at 32 / 8 heads, D = 128, back to back: 64 x 4096
// tokens 84-90 us by box (6.0-6.4 TB/s), 38 x 8192 96-100 us (6.4-6.7 TB/s), one row of
// 32768 17.3 us from twelve caches in turn (3.9 TB/s: ramp, merge and launch gap are two
// fifths) and 14.6-15.0 us from three, whose 201 MB L2 holds in part.  Next to
// HBM a warp's own time counts: about 310 instructions a block, 64 of them widening
// codes, and a loop that does not quite fit the instruction cache.  tcgen05 is not
// used: it would want the widened codes back in shared memory, for products of 8
// columns.  Staging with TMA boxes and mbarriers measured slower than cp.async
// (64 x 4096 90 against 86 us, D = 64 106 against 88 us).  Layout of the work:
//   * one CTA per tile, eight warps; warp w owns blocks w, w + 8, ... of the tile
//     with a private softmax state, so the loop has no barrier and no shared state;
//   * a warp copies its blocks by whole rows (cp.async, 16 bytes a lane) into a ring
//     of its own and waits for its own copies only; ldmatrix brings the codes out
//     conflict-free, four per register, in the order the fragments need (K as it
//     lies, V transposed), the contraction order being free; the ring slot is
//     refilled before the block's softmax;
//   * S^T = K Q^T and O^T += V^T P^T, with the query group as the 8 columns: no row
//     of a product is padding; P^T goes from one to the other through movmatrix;
//   * the block table and the scales are fetched 32 blocks at a time, one per lane.
// Bad page ids set PKV_DEV_PAGE_OOB and poison the tile; page 0 is read in place
// of such a page.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_merge.cuh"

namespace pkv {
namespace {

constexpr int kWarps = kThreads / 32;
// m, the reference of the weights, puts the largest weight of the block that moves it at 2^5 to 2^6 and
// holds until one would pass 2^13; O's reference does the same with weights times V scales, 2^6 to 2^8
// and 2^14.
constexpr float kHeadroom = 6.f, kGrowth = 13.f, kHeadroomV = 8.f, kGrowthV = 14.f;
// Most that O's reference lies below m, in powers of two: 2^13 * 2^104 is finite, and a sum of 2^28
// weights brings m another 2^41 above, 2^145 in all, whose reciprocal fp32 just holds.
constexpr float kMaxLift = 104.f;
constexpr float kLoUp = 2048.f, kLoDown = 1.f / 2048.f;   // P's lo parts are held times 2^11

template <int D, int G>
struct Q8Cfg {
    static constexpr int kBlockBytes = 2 * kBlockRows * D;   // K and V codes of one block
    static constexpr int kStages = D == 128 ? 3 : 5;         // 12 or 10 KB in flight per warp, 80-96 KB per CTA
    static constexpr int kMatBytes = kBlockRows * D;         // one K or V block: 16 rows of D bytes
    static constexpr int kChunks = D / 16;                   // 16-byte chunks of a row
    static constexpr int kPairFrom = D == 128 ? 40 : 4;     // blocks a warp from which two are reduced at a time
    static constexpr int kParts = G == 8 ? 2 : 1;            // P^T column tiles: the lo parts share one while 2G <= 8
    static_assert(D == 64 || D == 128, "head_dim");
};

template <int D, int G>
struct Q8Smem {
    static constexpr int kRing = Q8Cfg<D, G>::kStages * Q8Cfg<D, G>::kBlockBytes;   // one warp's ring
    static constexpr int kScratchBytes = kWarps * kRing;
    static constexpr int kAccRow = D + 4;   // floats of one head's partial (padded against bank conflicts)
    __device__ uint8_t* scratch() { return &ring[0][0]; }
    alignas(1024) uint8_t ring[kWarps][kRing];   // staged blocks; at the tile's end each warp's partial
    float m[kWarps][G], l[kWarps][G];
    int poisoned[kWarps];
    float merge_m[G], merge_inv[G];
    int merge_nan_h[G];
    int abort;
    int tile_slot[2];
    int tile_fin, tile_splits, tile_base;
    uint64_t tr[kTraceWords];
    static_assert(G * kAccRow * 4 <= kRing, "a warp's partial fits its ring");
    static_assert(kRing % 512 == 0 && Q8Cfg<D, G>::kBlockBytes % 512 == 0, "chunk addresses are formed by exclusive or");
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk `c` of row `r` in a staged block.  Chunks are
// exchanged within a row (by r mod 8 in 128-byte rows, by r / 2 mod 4 in 64-byte
// rows) so that one chunk index of eight neighbouring rows hits eight distinct
// bank groups.
template <int D>
__device__ __forceinline__ uint32_t chunk_offset(int r, int c) {
    return static_cast<uint32_t>(r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
}

// Four e4m3 codes to two f16x2: bytes 0, 1 and bytes 2, 3.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// D (16x8 fp32) += A (16x16 f16, row-major) * B (16x8 f16, column-major)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// 2^x (ex2.approx: about 2^-22 relative; results below 2^-126 are zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// An 8 x 8 tile of 16-bit values held as mma fragments (row lane / 4, columns
// 2 (lane % 4) and + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 2^e for a whole e from -126 to 127.
__device__ __forceinline__ float exp2i(float e) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<int>(e) + 127) << 23);
}

// The least whole number e with |x| < 2^e (-126 for zero and subnormals).
__device__ __forceinline__ float exponent_above(float x) {
    const uint32_t biased = (__float_as_uint(x) >> 23) & 0xffu;
    return __uint_as_float(0x4b000000u | biased) - (8388608.f + 126.f);   // 2^23 + biased, exactly
}

// One tile: every warp reduces its blocks, then the eight states are combined
// and written (to out / lse, or to the workspace for a split).
// Fragment coordinates: g = lane / 4 (a row of A and C: tokens g, g + 8 of K,
// two dimensions of V^T; a column of B: a head), t = lane % 4 (k pairs of A and
// B, columns 2t, 2t + 1 of C).
template <int D, int G>
__device__ void run_tile_q8(Q8Smem<D, G>& sm, const AttnQ8Params& qp, TileWork tw) {
    using C = Q8Cfg<D, G>;
    const AttnParams& p = qp.attn;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, t = lane & 3;
    // A queue tile's planned pages are copied at once; the row's length, which masks
    // its last block, is read meanwhile.
    const int nplan = (max(tw.t_stream - tw.t0, 0) + kBlockRows - 1) / kBlockRows;
    int mine = nplan > warp ? (nplan - warp + kWarps - 1) / kWarps : 0;   // this warp's blocks: warp + 8 i

    // the lane's share of a copy: 16-byte chunk lane % kChunks of rows lane /
    // kChunks, + kRows, ... (a warp moves whole rows)
    constexpr int kRows = 32 / C::kChunks;
    const uint32_t pitch = static_cast<uint32_t>(p.Hkv) * D;   // bytes between tokens
    const uint32_t lane_off = tw.kvh * D + (lane / C::kChunks) * pitch + (lane % C::kChunks) * 16;
    const uint32_t step = kRows * pitch;
    const uint32_t lane_chunk = chunk_offset<D>(lane / C::kChunks, lane % C::kChunks);   // below the ring's alignment
    const uint8_t* kpool = reinterpret_cast<const uint8_t*>(p.k_pages) + lane_off;
    const uint8_t* vpool = reinterpret_cast<const uint8_t*>(p.v_pages) + lane_off;
    const uint32_t ring = smem_addr(sm.ring[warp]);
    const uint64_t policy = l2_evict_first_policy();
    const int32_t* bt_row = p.block_table + static_cast<size_t>(tw.b) * p.max_pages;

    // 32 of the warp's blocks at a time: lane i holds block i's token row in the
    // pool and its scales.  The copies run ahead of the arithmetic, so the scales
    // of the batch being copied (k/v_next) and of the one being reduced differ for
    // a few blocks; the table entries are read one batch further ahead.
    int row_i = 0, entry = 0, poisoned = 0;
    float k_next = 0.f, v_next = 0.f, k_now = 0.f, v_now = 0.f;
    auto row_block = [&](int i) { return tw.t0 / kBlockRows + warp + kWarps * i; };   // 16-token block of the row
    auto page_of = [&](int blk) {   // blk / (blocks per page)
        return qp.page_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(blk), qp.page_magic)) : blk;
    };
    auto read_entry = [&](int i0) {
        if (i0 + lane < mine) entry = bt_row[page_of(row_block(i0 + lane))];
    };
    auto fetch_batch = [&](int i0) {
        if (i0 + lane < mine) {
            int page = entry;
            if (page < 0 || page >= p.num_pages) {
                atomicOr(&p.ctr->status, static_cast<uint32_t>(PKV_DEV_PAGE_OOB));
                poisoned = 1;
                page = 0;
            }
            const int blk = row_block(i0 + lane);
            row_i = page * p.page_size + blk * kBlockRows - page_of(blk) * p.page_size;
            const size_t s = static_cast<size_t>(row_i / kBlockRows) * p.Hkv + tw.kvh;
            k_next = qp.k_scales[s];
            v_next = qp.v_scales[s];
        }
        read_entry(i0 + 32);
    };
    auto issue = [&](int i, int stage) {   // block i of the current batch into `stage`
        const size_t off = static_cast<size_t>(__shfl_sync(kFull, row_i, i & 31)) * pitch;
        const uint32_t dst = (ring + stage * C::kBlockBytes) ^ lane_chunk;
        const uint8_t* ksrc = kpool + off;
        const uint8_t* vsrc = vpool + off;
#pragma unroll
        for (int x = 0; x < kBlockRows / kRows; ++x) {
            // (128-byte rows: row + 4 flips the exchange's bit 2)
            const uint32_t at = (D == 128 && (x & 1) ? dst ^ 64u : dst) + x * kRows * D;
            cp_async16(at, ksrc, policy);
            cp_async16(at + C::kMatBytes, vsrc, policy);
            ksrc += step;
            vsrc += step;
        }
    };

    // the first table entries, q and the row's length in one round trip
    read_entry(0);
    uint2 q_raw[D / 16];   // head g % G: elements 16 j + 4 t .. + 3
    {
        const uint16_t* qh = p.q + (static_cast<size_t>(tw.b) * p.Hq + tw.kvh * G + g % G) * D + t * 4;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) q_raw[j] = *reinterpret_cast<const uint2*>(qh + 16 * j);
    }
    if (tw.lazy) tile_finish(p, tw);
    // the ring's first blocks
    fetch_batch(0);
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
        if (s < mine) issue(s, s);
        cp_async_commit();
    }
    if (threadIdx.x == 0) {
        sm.tile_fin = tw.finalize;
        sm.tile_splits = tw.splits;
        sm.tile_base = tw.slot - tw.split;
    }
    const int ntok = tw.t1 > tw.t0 ? tw.t1 - tw.t0 : 0;
    const int nblk = (ntok + kBlockRows - 1) / kBlockRows;   // at most nplan
    mine = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;
    poisoned |= tw.poisoned;
    // B fragments of Q^T: column g is query head g % G (so with G <= 4 the columns
    // repeat the group: one copy serves P's hi parts, the next its lo parts).  A K
    // word is four neighbouring elements, 16 j + 4 t on for k-step j, so q's fragments
    // hold the same four
    uint32_t qb[D / 16][2];
    float qs[2];   // what the dot products of columns 2t, 2t + 1 are multiplied by, before ks
    {
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            big = max(big, max((q_raw[j].x & 0x7fffu) << 16, q_raw[j].x & 0x7fff0000u));
            big = max(big, max((q_raw[j].y & 0x7fffu) << 16, q_raw[j].y & 0x7fff0000u));
        }
        big = max(big, __shfl_xor_sync(kFull, big, 1));
        big = max(big, __shfl_xor_sync(kFull, big, 2));
        const int e = max(-126, min(126, static_cast<int>(big >> 23) - 127));
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        qs[0] = __shfl_sync(kFull, back, 8 * t);     // column 2t: the lanes of g = 2t hold its head
        qs[1] = __shfl_sync(kFull, back, 8 * t + 4);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            qb[j][0] = pack_half(__uint_as_float(q_raw[j].x << 16) * down, __uint_as_float(q_raw[j].x & 0xffff0000u) * down);
            qb[j][1] = pack_half(__uint_as_float(q_raw[j].y << 16) * down, __uint_as_float(q_raw[j].y & 0xffff0000u) * down);
        }
    }
    // Where the parts share a column tile, columns 2t and 2t + 1 carry whole * w - part * f16(w):
    // P's hi parts (whole 1, part 0) or its lo parts (both 2^11)
    const float whole0 = 2 * t < G ? 1.f : kLoUp, whole1 = 2 * t + 1 < G ? 1.f : kLoUp;
    const float part0 = 2 * t < G ? 0.f : kLoUp, part1 = 2 * t + 1 < G ? 0.f : kLoUp;

    // columns 2t, 2t + 1: the reference m (a whole number; before the first block less than any), this
    // lane's share of the sum of the weights 2^(s - m), and up = 2^lift, by which a weight is multiplied
    // on its way into O: O's reference is m - lift
    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, up[2] = {1.f, 1.f}, lift[2] = {0.f, 0.f};
    float o[C::kParts][D / 16][4];     // O^T accumulators
#pragma unroll
    for (int x = 0; x < C::kParts; ++x)
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[x][n][i] = 0.f;

    // a lane's row address for ldmatrix: matrices 0, 1 are rows 0-7 and 8-15 of a chunk, 2, 3 of the next chunk
    const uint32_t frag_off = chunk_offset<D>((lane & 7) + (lane & 8), lane >> 4);
    int stage = 0;
    // U blocks at a time; of a last, incomplete turn the missing block is masked whole.
    auto reduce = [&](auto u_blocks) {
        constexpr int U = decltype(u_blocks)::value;
        for (int i = 0; i < mine; i += U) {
            cp_async_wait<C::kStages - U>();
            __syncwarp();   // every lane's copies of the blocks have landed
            if (i == 0 && p.trace && threadIdx.x == 0 && sm.tr[kTrFirstBlock] == 0) sm.tr[kTrFirstBlock] = globaltimer_ns();
            if ((i & 31) == 0) {
                k_now = k_next;
                v_now = v_next;
            }
            float z[U][4], vs[U];
            int valid[U], slot[U];
            uint32_t src[U], vf[C::kChunks / 2][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                valid[u] = ntok - (warp + kWarps * (i + u)) * kBlockRows;   // tokens of the block (16 or more: all)
                slot[u] = stage;
                src[u] = ring + stage * C::kBlockBytes + frag_off;
                stage = stage + 1 == C::kStages ? 0 : stage + 1;
            }
            // V to registers, and the stage is free for its next block
            auto take_v = [&](int u) {
#pragma unroll
                for (int c = 0; c < C::kChunks; c += 2) ldsm_x4_trans(vf[c / 2], (src[u] ^ (c << 4)) + C::kMatBytes);
                __syncwarp();
                const int next = i + u + C::kStages;
                if (next < mine) {
                    if ((U == 1 || (u + C::kStages) % U == 0) && (next & 31) == 0) fetch_batch(next);
                    issue(next, slot[u]);
                }
                cp_async_commit();
            };
            // S^T = K Q^T: rows g and g + 8 are tokens g and g + 8
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};   // two chains, for the product's latency
#pragma unroll
                for (int c = 0; c < C::kChunks; c += 2) {
                    uint32_t w[4], a0, a1, a2, a3;
                    ldsm_x4(w, src[u] ^ (c << 4));
                    widen4(w[0], a0, a2);
                    widen4(w[1], a1, a3);
                    mma_f16(s, a0, a1, a2, a3, qb[c][0], qb[c][1]);
                    widen4(w[2], a0, a2);
                    widen4(w[3], a1, a3);
                    mma_f16(U == 1 ? s2 : s, a0, a1, a2, a3, qb[c + 1][0], qb[c + 1][1]);
                }
                const float ks = __shfl_sync(kFull, k_now, (i + u) & 31);
                vs[u] = __shfl_sync(kFull, v_now, (i + u) & 31);
                if (U > 1 && i + u >= mine) vs[u] = 0.f;
                const float sc0 = ks * qs[0], sc1 = ks * qs[1];
                z[u][0] = (U == 1 ? s[0] + s2[0] : s[0]) * sc0;
                z[u][1] = (U == 1 ? s[1] + s2[1] : s[1]) * sc1;
                z[u][2] = (U == 1 ? s[2] + s2[2] : s[2]) * sc0;
                z[u][3] = (U == 1 ? s[3] + s2[3] : s[3]) * sc1;
                if (valid[u] < kBlockRows) {
                    if (g >= valid[u]) z[u][0] = z[u][1] = -INFINITY;
                    if (g + 8 >= valid[u]) z[u][2] = z[u][3] = -INFINITY;
                }
            }
            if constexpr (U == 1) take_v(0);

            // A reference moves when a weight would pass 2^13, or a weight times V scale 2^14 in O's
            // units; neither happens often, so the exact maxima are found only then
            float t0 = -INFINITY, t1 = -INFINITY, y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float ev = exponent_above(vs[u]);
                const float a0 = fmaxf(z[u][0], z[u][2]) - m[0], a1 = fmaxf(z[u][1], z[u][3]) - m[1];
                t0 = fmaxf(t0, a0);
                t1 = fmaxf(t1, a1);
                y0 = fmaxf(y0, a0 + ev);
                y1 = fmaxf(y1, a1 + ev);
            }
            if (__any_sync(kFull, t0 > kGrowth || t1 > kGrowth || y0 + lift[0] > kGrowthV || y1 + lift[1] > kGrowthV)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(z[0][c], z[0][2 + c]);
                    if constexpr (U == 2) top = fmaxf(top, fmaxf(z[1][c], z[1][2 + c]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
                    const float mn = top - m[c] > kGrowth ? ceilf(top) - kHeadroom : m[c];
                    float most = fmaxf(z[0][c], z[0][2 + c]) - mn + exponent_above(vs[0]);
                    if constexpr (U == 2) most = fmaxf(most, fmaxf(z[1][c], z[1][2 + c]) - mn + exponent_above(vs[1]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, x));
                    const float moved = m[c] == mn ? 0.f : mn - m[c];
                    float ln = fminf(lift[c] + moved, kMaxLift);   // O's reference stays where it is ...
                    if (most + ln > kGrowthV) ln = fmaxf(kHeadroomV - ceilf(most), -126.f);   // ... or moves up too
                    l[c] *= exp2f(-moved);
                    const float f = exp2f(ln - lift[c] - moved);
                    m[c] = mn;
                    lift[c] = ln;
                    up[c] = exp2i(ln);
#pragma unroll
                    for (int x = 0; x < C::kParts; ++x)
#pragma unroll
                        for (int n = 0; n < D / 16; ++n) {
                            o[x][n][c] *= f;
                            o[x][n][2 + c] *= f;
                        }
                }
            }
            // B fragments of P^T: the 8 x 8 transposes of the token-major tiles
            uint32_t pb[U][C::kParts][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p0 = ex2(z[u][0] - m[0]), p1 = ex2(z[u][1] - m[1]);   // token g (masked: 0)
                const float p2 = ex2(z[u][2] - m[0]), p3 = ex2(z[u][3] - m[1]);   // token g + 8
                l[0] += p0 + p2;
                l[1] += p1 + p3;
                // (in this order no product overflows, whatever the scale of a block that weighs nothing)
                const float w0 = p0 * up[0] * vs[u], w1 = p1 * up[1] * vs[u];
                const float w2 = p2 * up[0] * vs[u], w3 = p3 * up[1] * vs[u];
                const uint32_t ha = pack_half(w0, w1), hb = pack_half(w2, w3);
                const float2 ua = unpack_half(ha), ub = unpack_half(hb);
                if constexpr (C::kParts == 2) {
                    pb[u][0][0] = transpose8(ha);
                    pb[u][0][1] = transpose8(hb);
                    pb[u][1][0] = transpose8(pack_half((w0 - ua.x) * kLoUp, (w1 - ua.y) * kLoUp));
                    pb[u][1][1] = transpose8(pack_half((w2 - ub.x) * kLoUp, (w3 - ub.y) * kLoUp));
                } else {
                    pb[u][0][0] = transpose8(pack_half(fmaf(-part0, ua.x, w0 * whole0), fmaf(-part1, ua.y, w1 * whole1)));
                    pb[u][0][1] = transpose8(pack_half(fmaf(-part0, ub.x, w2 * whole0), fmaf(-part1, ub.y, w3 * whole1)));
                }
            }

            // O^T += V^T P^T: rows g and g + 8 of tile c are dimensions 16 c + 2 g and + 1.  A
            // transposed word holds (token 2t: both dimensions), (token 2t + 1: both)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (U > 1) take_v(u);
                if (valid[u] < kBlockRows) {   // slots past the row's end may hold anything, NaN codes too (0 * NaN = NaN)
                    const uint32_t lo = (2 * t < valid[u] ? 0xffffu : 0u) | (2 * t + 1 < valid[u] ? 0xffff0000u : 0u);
                    const uint32_t hi = (2 * t + 8 < valid[u] ? 0xffffu : 0u) | (2 * t + 9 < valid[u] ? 0xffff0000u : 0u);
#pragma unroll
                    for (int c = 0; c < C::kChunks / 2; ++c) {
                        vf[c][0] &= lo;
                        vf[c][1] &= hi;
                        vf[c][2] &= lo;
                        vf[c][3] &= hi;
                    }
                }
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) {
                    uint32_t a0, a1, a2, a3;
                    widen4(__byte_perm(vf[c / 2][2 * (c & 1)], 0, 0x3120), a0, a1);
                    widen4(__byte_perm(vf[c / 2][2 * (c & 1) + 1], 0, 0x3120), a2, a3);
#pragma unroll
                    for (int x = 0; x < C::kParts; ++x) mma_f16(o[x][c], a0, a1, a2, a3, pb[u][x][0], pb[u][x][1]);
                }
            }
        }
    };
    // Two blocks at a time share a turn's bookkeeping and overlap their latencies; one
    // at a time starts earlier and has its loads out earlier.  Measured, one / two at a
    // time, by blocks a warp (G = 4; the other G differ alike, by up to 2 % from these):
    // D = 128, 4 blocks (200 x 500 tokens) 46.1 / 50.0 us, 7 (1 x 32768) 16.7 / 17.5, 8 (128
    // x 1024) 52.1 / 55.3, 14 on average (8 rows of 512-32768) 25.4 / 24.9, 32 (64 x 4096)
    // 85.7 / 86.5, 64 (38 x 8192) 109.4 / 100.0; D = 64, 2 blocks (64 x 300) 11.1 / 11.4, 4
    // 32.8 / 31.9, 7 14.6 / 14.5, 8 32.6 / 31.4, 14 18.4 / 17.5, 32 51.3 / 48.5.
    if (nblk >= C::kPairFrom * kWarps)
        reduce(std::integral_constant<int, 2>{});
    else
        reduce(std::integral_constant<int, 1>{});
    trace_stamp(sm, p, kTrStreamEnd);

    // publish the warp's state, divided by the power of two that brings the sum of its
    // weights to [1, 2), or to [1/16, 1/8) where large scales are about, so that the
    // eight partials together are no larger than the output: fold the lo parts into the
    // hi parts; a lane then holds D / 8 neighbouring dimensions of its columns' heads
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        l[0] += __shfl_xor_sync(kFull, l[0], x);
        l[1] += __shfl_xor_sync(kFull, l[1], x);
    }
    float down[2];   // from O's reference to m, and the division
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float e = l[c] > 0.f ? fminf(exponent_above(l[c]) + (lift[c] > 0.f ? -1.f : 3.f), 126.f) : 0.f;
        down[c] = exp2f(-lift[c] - e);
        l[c] *= exp2i(-e);
        m[c] += e;
    }
    poisoned = __any_sync(kFull, poisoned) ? 1 : 0;
    cp_async_wait<0>();   // (planned blocks past the row's end may still be on their way)
    __syncwarp();         // every lane has read its slots: the ring takes the partial
    float* acc = reinterpret_cast<float*>(sm.ring[warp]) + 2 * g;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
        float f[4];   // column 2t: dimensions 16 n + 2 g and + 1; column 2t + 1: the same
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = o[0][n][(k >> 1) + 2 * (k & 1)];
            if constexpr (C::kParts == 2) f[k] = fmaf(o[1][n][(k >> 1) + 2 * (k & 1)], kLoDown, f[k]);
            else if constexpr (G > 1) f[k] = fmaf(__shfl_xor_sync(kFull, f[k], G / 2), kLoDown, f[k]);   // (hi columns' lanes)
        }
        if constexpr (G == 1) {
            f[0] = fmaf(f[2], kLoDown, f[0]);
            f[1] = fmaf(f[3], kLoDown, f[1]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (2 * t + c < G)
                *reinterpret_cast<float2*>(acc + (2 * t + c) * Q8Smem<D, G>::kAccRow + 16 * n) =
                    make_float2(f[2 * c] * down[c], f[2 * c + 1] * down[c]);
    }
    if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (2 * t + c < G) {
                sm.m[warp][2 * t + c] = m[c];
                sm.l[warp][2 * t + c] = l[c];
            }
    }
    if (lane == 0) sm.poisoned[warp] = poisoned;
    __syncthreads();

    // exact combine of the eight states, one float4 (head h, d .. d+3) per thread and pass
    bool any_poison = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) any_poison |= sm.poisoned[w] != 0;
    for (int i = threadIdx.x; i < G * D / 4; i += kThreads) {
        const int h = i / (D / 4), d = (i % (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][h]);
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        float lse2 = -INFINITY;
        if (nblk > 0) {
            float lsum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sm.m[w][h];
                const float f = exp2f(mw - M);   // idle warp: 0
                lsum = fmaf(sm.l[w][h], f, lsum);
                const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w]) +
                                                                  h * Q8Smem<D, G>::kAccRow + d);
                r.x = fmaf(a.x, f, r.x);
                r.y = fmaf(a.y, f, r.y);
                r.z = fmaf(a.z, f, r.z);
                r.w = fmaf(a.w, f, r.w);
            }
            const float inv = lsum == 0.f ? 0.f : 1.f / lsum;   // (every score -inf: as no token at all)
            r = make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
            lse2 = M + log2f(lsum);
        }
        if (any_poison) {
            r = make_float4(NAN, NAN, NAN, NAN);
            lse2 = NAN;
        }
        if (tw.finalize) {
            const int qh = tw.kvh * G + h;
            *reinterpret_cast<float4*>(p.out + (static_cast<size_t>(tw.b) * p.Hq + qh) * D + d) = r;
            if (d == 0) p.lse[static_cast<size_t>(tw.b) * p.Hq + qh] = lse2 * kLn2;
        } else {
            *reinterpret_cast<float4*>(p.ws_o + (static_cast<size_t>(tw.slot) * G + h) * D + d) = r;
            if (d == 0) p.ws_lse[static_cast<size_t>(tw.slot) * G + h] = lse2;
        }
    }
    if (p.trace && threadIdx.x == 0) {
        sm.tr[kTrCombineEnd] = globaltimer_ns();
        sm.tr[kTrLastTile] = (static_cast<uint64_t>(tw.b) << 40) | (static_cast<uint64_t>(tw.kvh) << 20) |
                             static_cast<uint64_t>(tw.split);
        sm.tr[kTrTiles] += 1;
    }
}

// The row whose length is the rank-th largest (of equal lengths the lower row
// first), for B <= kThreads rows; all CTA threads call this.
template <int D, int G>
__device__ int row_by_length(Q8Smem<D, G>& sm, const AttnParams& p, int rank) {
    int* lens = reinterpret_cast<int*>(sm.scratch());   // the idle ring
    const int r = threadIdx.x, n = r < p.B ? p.seq_lens[r] : INT_MIN;
    lens[r] = n;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < p.B; i += 4) {   // (past B: INT_MIN, before no row)
        const int4 x = *reinterpret_cast<const int4*>(lens + i);
        before += (x.x > n || (x.x == n && i < r)) + (x.y > n || (x.y == n && i + 1 < r)) +
                  (x.z > n || (x.z == n && i + 2 < r)) + (x.w > n || (x.w == n && i + 3 < r));
    }
    if (r < p.B && before == rank) sm.tile_slot[1] = r;
    __syncthreads();
    return sm.tile_slot[1];
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 2) attention_q8_kernel(const __grid_constant__ AttnQ8Params qp) {
    // (aligned by its declaration: through an address rounded up at run time the
    // compiler would lose sight of the memory being shared)
    extern __shared__ __align__(1024) uint8_t smem_q8[];
    Q8Smem<D, G>& sm = *reinterpret_cast<Q8Smem<D, G>*>(smem_q8);
    const AttnParams& p = qp.attn;
    if (p.trace && threadIdx.x == 0) {
        for (int i = 0; i < kTraceWords; ++i) sm.tr[i] = 0;
        sm.tr[kTrEntry] = globaltimer_ns();
        sm.tr[kTrSm] = smid();
    }
    if (threadIdx.x == 0) sm.abort = 0;
    // Before the grid dependency wait, only what no kernel writes may be used: a
    // host-staged queue entry.  L2 is warmed with the blocks the ring starts with,
    // through a speculative read of the block table; prefetches change no value.
    const bool staged = p.route == kRouteQueue && p.queue_host_staged && static_cast<int>(blockIdx.x) < p.num_tiles;
    pkv_work_item item{};
    if (staged) {
        item = p.queue[blockIdx.x];
        if (item.b >= 0 && item.b < p.B && item.kvh >= 0 && item.kvh < p.Hkv && item.page_begin >= 0 &&
            item.page_end <= p.max_pages) {
            const int t0 = item.page_begin * p.page_size;
            const int t_end = min(item.page_end * p.page_size, t0 + kWarps * Q8Cfg<D, G>::kStages * kBlockRows);
            const int32_t* bt_row = p.block_table + static_cast<size_t>(item.b) * p.max_pages;
            for (int tok = t0 + static_cast<int>(threadIdx.x); tok < t_end; tok += kThreads) {
                const int page = ld_volatile_i32(bt_row + tok / p.page_size);
                if (page < 0 || page >= p.num_pages) continue;
                const size_t row = static_cast<size_t>(page) * p.page_size + tok % p.page_size;
                const size_t off = (row * p.Hkv + item.kvh) * D;
                prefetch_l2(reinterpret_cast<const uint8_t*>(p.k_pages) + off);
                prefetch_l2(reinterpret_cast<const uint8_t*>(p.v_pages) + off);
                if (row % kBlockRows == 0) {
                    prefetch_l2(qp.k_scales + row / kBlockRows * p.Hkv + item.kvh);
                    prefetch_l2(qp.v_scales + row / kBlockRows * p.Hkv + item.kvh);
                }
            }
        }
    }
    grid_dependency_wait();
    trace_stamp(sm, p, kTrWaitDone);
    __syncthreads();
    auto trace_flush = [&]() {
        if (p.trace && threadIdx.x == 0) {
            sm.tr[kTrExit] = globaltimer_ns();
            uint64_t* row = p.trace + static_cast<size_t>(blockIdx.x) * kTraceWords;
            for (int i = 0; i < kTraceWords; ++i) row[i] = sm.tr[i];
        }
    };
    auto neutral_rows = [&]() {   // rows with no tokens get no tiles
        if (p.no_empty_rows) return;
        for (int b = blockIdx.x; b < p.B; b += gridDim.x)
            if (p.row_splits[b] == 0) write_neutral_row(p, b, threadIdx.x, blockDim.x);
    };

    if (p.route == kRoutePersistent) {
        while (true) {
            if (threadIdx.x == 0) sm.tile_slot[0] = static_cast<int>(atomicAdd(&p.ctr->next_tile, 1u));
            __syncthreads();
            const int i = sm.tile_slot[0];
            if (i >= p.num_tiles) break;
            const TileWork tw = tile_from_item(p, p.queue[p.order[i]]);
            run_tile_q8<D, G>(sm, qp, tw);
            __syncthreads();
            if (!sm.tile_fin && p.fused_merge) merge_if_last<D, G>(sm, p, tw.b, tw.kvh, sm.tile_splits);
            __syncthreads();
        }
        launch_dependents();
        neutral_rows();
        if (threadIdx.x == 0 && atomicAdd(&p.ctr->done_ctas, 1u) == gridDim.x - 1) {
            p.ctr->next_tile = 0;   // the last CTA out rewinds the queue for the next launch
            p.ctr->done_ctas = 0;
        }
        trace_flush();
        return;
    }

    TileWork tw{};
    if (p.route == kRouteDirect) {
        tw.b = blockIdx.x / p.Hkv;
        tw.kvh = blockIdx.x % p.Hkv;
        if (qp.longest_first) tw.b = row_by_length(sm, p, tw.b);
        tw.t1 = p.seq_lens[tw.b];
        tw.finalize = 1;
        tw.splits = 1;
        if (tw.t1 < 0 || tw.t1 > p.max_pages * p.page_size) {   // would read past the table row
            tw.poisoned = 1;
            tw.t1 = 0;
            if (threadIdx.x == 0) atomicOr(&p.ctr->status, static_cast<uint32_t>(PKV_DEV_PLAN_MISMATCH));
        }
        tw.t_stream = tw.t1;
    } else if (p.route == kRouteQueue) {
        if (static_cast<int>(blockIdx.x) >= p.num_tiles) {   // launched only for the neutral rows
            launch_dependents();
            neutral_rows();
            trace_flush();
            return;
        }
        tw = tile_from_item(p, staged ? item : p.queue[blockIdx.x]);
    } else {   // padded grid: (b, kvh, s) from the block index, ranges from the device lengths
        const int per_row = p.Hkv * p.max_splits;
        tw.b = blockIdx.x / per_row;
        tw.kvh = (blockIdx.x % per_row) / p.max_splits;
        tw.split = blockIdx.x % p.max_splits;
        const int n = p.seq_lens[tw.b];
        const int pages = (n + p.page_size - 1) / p.page_size;
        tw.poisoned = n < 0 || pages > p.max_splits * p.chunk_pages || n > p.max_pages * p.page_size;
        if (tw.poisoned && threadIdx.x == 0) atomicOr(&p.ctr->status, static_cast<uint32_t>(PKV_DEV_PLAN_MISMATCH));
        const int pb = max(0, min(tw.split * p.chunk_pages, pages));
        const int pe = max(0, min((tw.split + 1) * p.chunk_pages, pages));
        tw.t0 = pb * p.page_size;
        tw.t1 = tw.poisoned ? tw.t0 : min(pe * p.page_size, n);
        tw.t_stream = tw.t1;
        tw.finalize = p.max_splits == 1;
        tw.splits = p.max_splits;
        tw.slot = blockIdx.x;
    }
    run_tile_q8<D, G>(sm, qp, tw);
    __syncthreads();
    launch_dependents();   // the next grid may start its CTAs in the slots this tail frees
    if (!sm.tile_fin && p.fused_merge) {
        if (p.all_merge)
            merge_all_splits<D, G>(sm, p, tw.b, tw.kvh, tw.split, sm.tile_splits);
        else
            merge_if_last<D, G>(sm, p, tw.b, tw.kvh, sm.tile_splits);
    }
    if (p.route == kRouteQueue) neutral_rows();
    trace_flush();
}

template <int D, int G>
cudaError_t launch_q8_t(const AttnQ8Params& p, int grid, cudaStream_t stream, bool cooperative) {
    constexpr size_t smem = sizeof(Q8Smem<D, G>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    if (cooperative) {
        attr[n].id = cudaLaunchAttributeCooperative;
        attr[n].val.cooperative = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    // Devices on which the kernel has been allowed that much shared memory; a device
    // that was reset since forgets it, and the launch is refused.
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (configured.load(std::memory_order_relaxed) & bit) {
        e = cudaLaunchKernelEx(&cfg, attention_q8_kernel<D, G>, p);
        if (e != cudaErrorInvalidValue) return e;
        (void)cudaGetLastError();
    }
    e = cudaFuncSetAttribute(attention_q8_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, attention_q8_kernel<D, G>, p);
}

}  // namespace

cudaError_t launch_attention_q8(const AttnQ8Params& p, int grid, cudaStream_t stream, bool cooperative) {
    const int G = p.attn.Hq / p.attn.Hkv;
    switch (p.attn.D * 16 + G) {
        case 64 * 16 + 1: return launch_q8_t<64, 1>(p, grid, stream, cooperative);
        case 64 * 16 + 2: return launch_q8_t<64, 2>(p, grid, stream, cooperative);
        case 64 * 16 + 4: return launch_q8_t<64, 4>(p, grid, stream, cooperative);
        case 64 * 16 + 8: return launch_q8_t<64, 8>(p, grid, stream, cooperative);
        case 128 * 16 + 1: return launch_q8_t<128, 1>(p, grid, stream, cooperative);
        case 128 * 16 + 2: return launch_q8_t<128, 2>(p, grid, stream, cooperative);
        case 128 * 16 + 4: return launch_q8_t<128, 4>(p, grid, stream, cooperative);
        case 128 * 16 + 8: return launch_q8_t<128, 8>(p, grid, stream, cooperative);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
