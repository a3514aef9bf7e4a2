// pkv_append_tokens.cu -- ragged append of rotated keys and values to a paged
// cache, in bf16 or quantised to e4m3 with one scale per 16-token block and KV
// head.
//
// Layout and role as in pkv_append.cu ("PersistentKV: Page-Aware Decode
// Scheduling for Long-Context LLM Serving on Commodity GPUs", gist.science
// summary, Methodology section 1 "Layout"; the KV-cache update and rotary
// operators of "GPUOS", arXiv 2604.17861, section 4).
//
// Mathematics.  Token i of row b has position p = seq_lens[b] + i.  Of its first
// `dim` elements the pair (x, y) number m turns by the angle p * inv_freq[m]:
//     (x, y) -> scale * (x cos - y sin, y cos + x sin).
// The angle is reduced in integers: step[m] is inv_freq[m] / 2 pi in units of
// 2^-64 turns, so p * step[m] mod 2^64 is the phase, exact but for step's own
// rounding however far the position; its nearest quarter turn is taken off in
// integers too, which leaves at most an eighth of a turn for the series of sin
// and cos.
// An e4m3 block stores x / s with s the least power of two that brings the
// largest finite |x| of the block's new tokens to at most 448, and at least the
// scale of the tokens the block already holds.  e4m3 keeps four significant
// bits at any scale, so a power of two costs no precision, and when a later
// token raises the scale the older codes move to it exactly, save those that
// fall below e4m3's normal range (2^-6 of the new scale), which round again.
//
// What bounds it: HBM, (2 * Hq + 4 * Hkv) * D * 2 bytes per token in bf16 (Hkv * D
// * 2 less for e4m3).  One CTA per (16-token block, KV head or two): the block's
// scale needs no other CTA, a thread owns 16 elements of one token of every head
// of the group, so its eight sines and cosines serve the K head and the G query
// heads, and every access is 16 bytes (8 for e4m3 codes of half pairs).  8 x 128
// and 32 query heads, prompts of 12.5 thousand tokens in bf16: 48.5 us, 6.3 TB/s; of
// 8.8 thousand in e4m3: 35.1-35.5 us, 5.6 TB/s, where the arithmetic (about 930
// instructions a warp and head, half of the issue slots) bounds it too; one token
// for each of 64 rows: 4.2 us in a graph, a chain of round trips (length, table
// entry, scales, then the stores).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr uint32_t kInfinity = 0x7f800000u;
constexpr int kQueries = 4;   // query heads whose loads a thread has in flight at once

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Two floats to two e4m3 codes (a in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Largest magnitude of 16 values, as bits: NaN is passed over; 0x7f800000 if one is infinite.
__device__ __forceinline__ uint32_t magnitude16(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
    return __float_as_uint(m);
}

// The same of the finite ones among them.
__device__ __forceinline__ uint32_t finite_magnitude16(const float (&x)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        if (u < kInfinity) m = max(m, u);
    }
    return m;
}

// Largest of all threads' values, over the CTA (one barrier; `part` is shared scratch).
template <int kWarpsT>
__device__ __forceinline__ void cta_max(uint32_t& a, uint32_t& b, uint32_t (&part)[2][kWarpsT]) {
    a = __reduce_max_sync(kFull, a);
    b = __reduce_max_sync(kFull, b);
    if (threadIdx.x % 32 == 0) {
        part[0][threadIdx.x / 32] = a;
        part[1][threadIdx.x / 32] = b;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarpsT; ++i) {
        a = max(a, part[0][i]);
        b = max(b, part[1][i]);
    }
}

// sin and cos of an angle of at most an eighth of a turn (pi / 4): their power
// series to the terms below 2^-25.
__device__ __forceinline__ void sincos_eighth(float a, float& s, float& c) {
    const float u = a * a;
    s = fmaf(u, 1.f / 362880, -1.f / 5040);
    s = fmaf(u, s, 1.f / 120);
    s = fmaf(u, s, -1.f / 6);
    s = fmaf(a * u, s, a);
    c = fmaf(u, -1.f / 3628800, 1.f / 40320);
    c = fmaf(u, c, -1.f / 720);
    c = fmaf(u, c, 1.f / 24);
    c = fmaf(u, c, -0.5f);
    c = fmaf(u, c, 1.f);
}

// The least power of two s in [2^-120, 2^120] with amax / s <= 448 = 0.875 * 2^9.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    // amax = 1.m * 2^e: 448 = 1.75 * 2^8, so s = 2^(e - 8), or 2^(e - 7) if 1.m > 1.75
    int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(-120, min(120, e));   // (zero and subnormal maxima end at -120)
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// What a row asks for, from its length and offsets alone (the same in every
// thread); `bad`: status bits of a row that cannot take its tokens.
struct RowWork {
    int tok0;      // its first token in k / v / q
    int n;         // new tokens
    int pos0;      // position of the first one
    uint32_t bad;
};

__device__ __forceinline__ RowWork row_work(const AppendTokensParams& p, int b) {
    RowWork w{b, 1, p.seq_lens[b], 0u};
    if (p.cu) {
        const int end = p.cu[b + 1];
        w.tok0 = p.cu[b];
        if (w.tok0 < 0 || end < w.tok0 || end > p.T) {   // offsets that do not describe T tokens
            w.bad = PKV_DEV_PLAN_MISMATCH;
            w.n = 0;
            return w;
        }
        w.n = end - w.tok0;
    }
    if (w.n > 0 && (w.pos0 < 0 || static_cast<int64_t>(w.pos0) + w.n > static_cast<int64_t>(p.max_pages) * p.page_size))
        w.bad = PKV_DEV_ROW_FULL;
    return w;
}

// The row's page that holds its 16-token block `blk`: blk / (blocks per page).
__device__ __forceinline__ int page_of(const AppendTokensParams& p, int blk) {
    return p.page_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(blk), p.page_magic)) : blk;
}

// The rest of the check, over the table entries of all of the row's new tokens,
// by the whole CTA (a barrier): a row is refused before any byte of it is written.
// One coalesced read up to D pages, then a loop, and every CTA of the row makes it:
// at 16-token pages and 8 KV heads n^2 / 16 bytes for n tokens, which shows from some
// 100 thousand on (e4m3, 32 query heads: 1.21 times the bytes' time at 65 thousand,
// 1.42 at 131 thousand).
__device__ __forceinline__ uint32_t row_pages_bad(const AppendTokensParams& p, int b, const RowWork& w) {
    uint32_t bad = w.bad;
    if (!bad && w.n > 0) {
        const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
        const int last = page_of(p, (w.pos0 + w.n - 1) / kBlockRows);
        for (int i = page_of(p, w.pos0 / kBlockRows) + static_cast<int>(threadIdx.x); i <= last; i += static_cast<int>(blockDim.x)) {
            const int page = row[i];
            if (page < 0)
                bad |= PKV_DEV_ROW_FULL;
            else if (page >= p.num_pages)
                bad |= PKV_DEV_PAGE_OOB;
        }
    }
    if (!__syncthreads_or(static_cast<int>(bad))) return 0u;
    return (__syncthreads_or(bad & PKV_DEV_ROW_FULL) ? PKV_DEV_ROW_FULL : 0u) |
           (__syncthreads_or(bad & PKV_DEV_PAGE_OOB) ? PKV_DEV_PAGE_OOB : 0u) |
           (__syncthreads_or(bad & PKV_DEV_PLAN_MISMATCH) ? PKV_DEV_PLAN_MISMATCH : 0u);
}

// A thread's 16 elements of one head of one token: two runs of eight, at
// elements e0 and e1 of the head.
struct Slice {
    uint4 a, b;
};

__device__ __forceinline__ Slice load_slice(const uint16_t* head, int e0, int e1) {
    Slice s;
    s.a = *reinterpret_cast<const uint4*>(head + e0);
    s.b = *reinterpret_cast<const uint4*>(head + e1);
    return s;
}

__device__ __forceinline__ void widen(const Slice& s, float (&x)[16]) {
    float a[8], b[8];
    unpack_bf16x8(s.a, a);
    unpack_bf16x8(s.b, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = a[i];
        x[8 + i] = b[i];
    }
}

// Turn a slice by the thread's eight angles (cos and sin already scaled).
// Half pairs: x runs through a, y through b.  Neighbouring pairs: (x, y) are
// (0, 1), (2, 3), ... of a, then of b.  A slice past the rotated elements is
// only widened.
template <bool kPairs>
__device__ __forceinline__ void turn(const Slice& s, bool rotate, const float (&c)[8], const float (&sn)[8],
                                     float (&x)[16]) {
    widen(s, x);
    if (!rotate) return;
    if constexpr (kPairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = fmaf(u, c[i], -w * sn[i]);
            x[2 * i + 1] = fmaf(w, c[i], u * sn[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[i], w = x[8 + i];
            x[i] = fmaf(u, c[i], -w * sn[i]);
            x[8 + i] = fmaf(w, c[i], u * sn[i]);
        }
    }
}

__device__ __forceinline__ void store_bf16(uint16_t* head, int e0, int e1, const float (&x)[16]) {
    *reinterpret_cast<uint4*>(head + e0) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    *reinterpret_cast<uint4*>(head + e1) =
        make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
}

// x / s and x * s rounded so that a second rounding, to fewer bits, gives what one
// rounding would: towards zero, with the last bit set where something was cut off.
__device__ __forceinline__ float sticky(float toward_zero, float rest) {
    return __uint_as_float(__float_as_uint(toward_zero) | (rest != 0.f ? 1u : 0u));
}

__device__ __forceinline__ float divide_odd(float x, float s) {
    const float q = __fdiv_rz(x, s);
    return sticky(q, fmaf(-q, s, x));
}

__device__ __forceinline__ float multiply_odd(float x, float s) {
    const float q = __fmul_rz(x, s);
    return sticky(q, fmaf(x, s, -q));
}

__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// Eight values to eight codes.  Scales that the append makes are powers of two, and x
// times their reciprocal is exact; a block filled by somebody else may hold its tokens
// at another scale.  NaN stays NaN; an infinite value becomes NaN too, not the largest
// code, where the block is known to hold one (x * 0 is NaN for it and +-0 otherwise).
__device__ __forceinline__ uint2 codes8(const float* x, float s, float inv, bool infinite) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    if (!power_of_two(s))
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = divide_odd(x[i], s);
    if (infinite)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], 0.f, y[i]);
    return make_uint2(pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16,
                      pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16);
}

// Move 16 codes from one scale to a larger one.
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float ratio) {
    const float2 lo = unpack_e4m3(w & 0xffffu), hi = unpack_e4m3(w >> 16);
    return pack_e4m3(multiply_odd(lo.x, ratio), multiply_odd(lo.y, ratio)) |
           pack_e4m3(multiply_odd(hi.x, ratio), multiply_odd(hi.y, ratio)) << 16;
}

__device__ __forceinline__ uint4 requantise16(const uint4& w, float ratio) {
    return make_uint4(requantise4(w.x, ratio), requantise4(w.y, ratio), requantise4(w.z, ratio), requantise4(w.w, ratio));
}

template <int D, bool Q8, bool kPairs>
__global__ void __launch_bounds__(D) append_tokens_kernel(const __grid_constant__ AppendTokensParams p) {
    constexpr int kTpt = D / 16;               // threads per token
    constexpr int kCta = kBlockRows * kTpt;    // = D
    __shared__ int s_row;
    __shared__ RowWork s_work;
    __shared__ uint32_t s_max[2][2][kCta / 32];
    __shared__ alignas(16) uint64_t s_step[PKV_ROTARY_MAX_DIM / 2];
    grid_dependency_wait();
    if (p.early) launch_dependents();

    for (int i = threadIdx.x; i < PKV_ROTARY_MAX_DIM / 2; i += kCta) s_step[i] = p.rot.step[i];   // (read after a barrier)
    const int piece = blockIdx.x, kvh0 = blockIdx.y * p.heads;   // this CTA's KV heads: kvh0 .. kvh0 + heads - 1
    // The row of this piece.  With offsets, row r owns the pieces from
    // floor(cu[r] / 16) + 2 r on: at least as many as 16-token blocks that
    // cu[r + 1] - cu[r] tokens can touch from any start inside a block.  The thread
    // that finds the row has its work in the same round trip.
    int b = piece, first = piece;
    RowWork w;
    if (p.cu) {
        if (threadIdx.x == 0) {
            s_row = p.B;
            s_work = RowWork{0, 0, 0, 0u};   // no row: the CTA still writes a length below
        }
        __syncthreads();
        int found = p.B;
        for (int r = threadIdx.x; r < p.B; r += kCta) {
            const RowWork its = row_work(p, r);
            const int64_t lo = p.cu[r] / kBlockRows + 2ll * r, hi = p.cu[r + 1] / kBlockRows + 2ll * (r + 1);
            if (lo <= piece && piece < hi && r < found) {   // (two rows can claim a piece only if offsets descend)
                found = r;
                w = its;
                atomicMin(&s_row, r);
            }
        }
        __syncthreads();
        b = s_row;
        if (found == b && b < p.B) s_work = w;
        __syncthreads();
        w = s_work;
        first = w.tok0 / kBlockRows + 2 * b;
    } else {
        w = row_work(p, b);
    }
    const int blk0 = (w.pos0 / kBlockRows + (piece - first)) * kBlockRows;   // first position of the 16-token block
    const int lo = max(blk0, w.pos0), hi = min(blk0 + kBlockRows, w.pos0 + w.n);
    const bool work = !w.bad && lo < hi;
    const int slot = static_cast<int>(threadIdx.x) / kTpt, j = static_cast<int>(threadIdx.x) % kTpt;
    const int pos = blk0 + slot;
    const bool live = work && pos >= lo && pos < hi;
    const int64_t tok = static_cast<int64_t>(w.tok0) + (pos - w.pos0);

    // the thread's elements of a head
    const int dim = p.rot.dim;
    const bool rotate = j < dim / 16;
    int e0, e1;
    if (rotate && !kPairs) {
        e0 = 8 * j;
        e1 = dim / 2 + 8 * j;
    } else {   // sixteen neighbours: pairs, or past the rotated elements
        e0 = 16 * j;
        e1 = e0 + 8;
    }

    // all loads that need no page are in flight before the row's pages are checked
    const int G = p.Hq / p.Hkv;
    Slice ks{}, vs{}, qs[kQueries] = {};
    auto load_head = [&](int kvh) {
        if (!live) return;
        ks = load_slice(p.k + tok * p.k_stride + kvh * D, e0, e1);
        vs = load_slice(p.v + tok * p.v_stride + kvh * D, e0, e1);
        if (p.q) {
            const uint16_t* qh = p.q + tok * p.q_stride + static_cast<int64_t>(kvh) * G * D;
#pragma unroll
            for (int g = 0; g < kQueries; ++g)
                if (g < G) qs[g] = load_slice(qh + g * D, e0, e1);
        }
    };
    load_head(kvh0);
    const uint32_t bad = row_pages_bad(p, min(b, p.B - 1), w);   // (no row: no work, nothing read)

    // the lengths after: one CTA per row, whichever piece it holds
    if (kvh0 == 0 && piece < p.B) {
        RowWork o = w;
        uint32_t o_bad = bad;
        if (p.cu) {
            o = row_work(p, piece);
            o_bad = row_pages_bad(p, piece, o);
        }
        if (threadIdx.x == 0) {
            p.new_lens[piece] = p.seq_lens[piece] + (o_bad ? 0 : o.n);
            if (o_bad) atomicOr(p.status, o_bad);
        }
    }
    if (bad || !work) return;
    const int blk = blk0 / kBlockRows, its_page = page_of(p, blk);
    const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + its_page];
    // token row of the block in the pool
    const size_t prow0 = static_cast<size_t>(page) * p.page_size + (blk0 - its_page * p.page_size);
    const bool held = lo > blk0;   // the block holds older tokens of the row

    float c[8], sn[8];
    if (live && rotate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t step = s_step[8 * j + i];
            const uint32_t at = static_cast<uint32_t>(pos);
            const uint32_t turns = __umulhi(static_cast<uint32_t>(step), at) + static_cast<uint32_t>(step >> 32) * at;
            const uint32_t quarter = (turns + 0x20000000u) >> 30;          // nearest quarter turn
            const int rest = static_cast<int>(turns - (quarter << 30));    // in [-2^29, 2^29)
            float s0, c0;
            sincos_eighth(static_cast<float>(rest) * 1.4629180792671596e-9f, s0, c0);   // * 2 pi / 2^32
            s0 *= p.rot.scale;
            c0 *= p.rot.scale;
            const bool odd = quarter & 1u;
            const float cc = odd ? s0 : c0, ss = odd ? c0 : s0;
            c[i] = (quarter == 1u || quarter == 2u) ? -cc : cc;
            sn[i] = (quarter & 2u) ? -ss : ss;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = sn[i] = 0.f;
    }

    for (int h = 0; h < p.heads; ++h) {
        const int kvh = kvh0 + h;
        const size_t head_off = ((prow0 + slot) * p.Hkv + kvh) * D;
        // what the block holds already
        [[maybe_unused]] const size_t sidx = prow0 / kBlockRows * p.Hkv + kvh;
        [[maybe_unused]] float k_old = 0.f, v_old = 0.f;
        [[maybe_unused]] uint4 k_held, v_held;
        if constexpr (Q8) {
            if (held) {
                k_old = p.k_scales[sidx];
                v_old = p.v_scales[sidx];
                if (pos < lo) {
                    k_held = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pages) + head_off + 16 * j);
                    v_held = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_pages) + head_off + 16 * j);
                }
            }
        }
        float x[16];
        turn<kPairs>(ks, rotate, c, sn, x);
        if constexpr (!Q8) {
            if (live) {
                store_bf16(static_cast<uint16_t*>(p.k_pages) + head_off, e0, e1, x);
                uint16_t* vh = static_cast<uint16_t*>(p.v_pages) + head_off;
                *reinterpret_cast<uint4*>(vh + e0) = vs.a;
                *reinterpret_cast<uint4*>(vh + e1) = vs.b;
            }
        } else {
            float y[16];
            widen(vs, y);
            uint32_t km = magnitude16(x), vm = magnitude16(y);   // (a slot without a new token holds zeros)
            cta_max(km, vm, s_max[h & 1]);   // and every thread has read the old scales and codes
            const bool infinite = km == kInfinity || vm == kInfinity;
            if (infinite) {
                km = finite_magnitude16(x);
                vm = finite_magnitude16(y);
                __syncthreads();   // s_max is read
                cta_max(km, vm, s_max[h & 1]);
            }
            const float k_new = fmaxf(block_scale(km), fabsf(k_old)), v_new = fmaxf(block_scale(vm), fabsf(v_old));
            uint8_t* kp = static_cast<uint8_t*>(p.k_pages) + head_off;
            uint8_t* vp = static_cast<uint8_t*>(p.v_pages) + head_off;
            if (live) {
                const float ki = 1.f / k_new, vi = 1.f / v_new;
                *reinterpret_cast<uint2*>(kp + e0) = codes8(x, k_new, ki, infinite);
                *reinterpret_cast<uint2*>(kp + e1) = codes8(x + 8, k_new, ki, infinite);
                *reinterpret_cast<uint2*>(vp + e0) = codes8(y, v_new, vi, infinite);
                *reinterpret_cast<uint2*>(vp + e1) = codes8(y + 8, v_new, vi, infinite);
            } else if (pos < lo) {   // an older token of the block
                if (k_new != k_old) *reinterpret_cast<uint4*>(kp + 16 * j) = requantise16(k_held, k_old / k_new);
                if (v_new != v_old) *reinterpret_cast<uint4*>(vp + 16 * j) = requantise16(v_held, v_old / v_new);
            }
            if (threadIdx.x == 0) {
                p.k_scales[sidx] = k_new;
                p.v_scales[sidx] = v_new;
            }
        }

        if (p.q && live) {
            const uint16_t* qh = p.q + tok * p.q_stride + static_cast<int64_t>(kvh) * G * D;
            uint16_t* oh = p.q_out + tok * p.q_out_stride + static_cast<int64_t>(kvh) * G * D;
            for (int g0 = 0; g0 < G; g0 += kQueries) {   // in place is fine: a thread writes only what it has read
#pragma unroll
                for (int g = 0; g < kQueries; ++g) {
                    if (g0 + g >= G) break;
                    if (g0 > 0) qs[g] = load_slice(qh + (g0 + g) * D, e0, e1);
                }
#pragma unroll
                for (int g = 0; g < kQueries; ++g) {
                    if (g0 + g >= G) break;
                    float z[16];
                    turn<kPairs>(qs[g], rotate, c, sn, z);
                    store_bf16(oh + (g0 + g) * D, e0, e1, z);
                }
            }
        }
        if (h + 1 < p.heads) load_head(kvh + 1);
    }
}

// From this many (block, KV head) units on a CTA takes two KV heads one after the
// other, which share its row look-up and its sines and cosines.  Below, one: the
// call is a chain of round trips.  Measured, one / two heads, one row, 8 KV heads,
// e4m3: 512 tokens 4.41 / 5.06 us, 1024 (528 units) 5.62 / 6.13, 2048 (1040) 12.6 /
// 12.2, 16384 69.1 / 64.6 us; bf16: 3.81 / 4.03, 5.19 / 5.65, 12.0 / 11.3, 66.9 /
// 66.1 us.  (Loading the second head's inputs during the first's arithmetic costs
// a fourth CTA per SM its registers: slower.)
constexpr int64_t kTwoHeadUnits = 1024;

template <int D, bool Q8, bool kPairs>
cudaError_t launch_t(AppendTokensParams p, cudaStream_t stream) {
    const int64_t pieces = p.cu ? static_cast<int64_t>(p.T) / kBlockRows + 2ll * p.B : p.B;
    const uint32_t bpp = static_cast<uint32_t>(p.page_size / kBlockRows);
    p.page_magic = bpp > 1 ? static_cast<uint32_t>((1ull << 32) / bpp + 1) : 0u;
    p.heads = p.Hkv % 2 == 0 && pieces * p.Hkv >= kTwoHeadUnits ? 2 : 1;
    // The next kernel's CTAs may move in early, while this grid leaves SMs free (one row
    // of 32768 appended and decoded: 20.0 us, without 21.6; 8 rows 28.5 / 28.9).  Moving
    // in as a larger grid's CTAs leave, the decode's longest tiles end up two to an SM: 56
    // rows of 1024-8192 95 us against 89.
    p.early = pieces * (p.Hkv / p.heads) <= p.num_sms ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pieces), static_cast<unsigned>(p.Hkv / p.heads));
    cfg.blockDim = dim3(D);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_tokens_kernel<D, Q8, kPairs>, p);
}

template <int D, bool Q8>
cudaError_t launch_d(const AppendTokensParams& p, cudaStream_t stream) {
    return p.rot.interleaved ? launch_t<D, Q8, true>(p, stream) : launch_t<D, Q8, false>(p, stream);
}

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensParams& p, cudaStream_t stream) {
    const bool q8 = p.k_scales != nullptr;
    switch (p.D) {
        case 64: return q8 ? launch_d<64, true>(p, stream) : launch_d<64, false>(p, stream);
        case 128: return q8 ? launch_d<128, true>(p, stream) : launch_d<128, false>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
