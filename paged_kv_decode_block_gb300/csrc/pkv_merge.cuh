// pkv_merge.cuh -- what every decode kernel does around its tiles: the tile of
// a queue entry, the neutral state of an empty row, and the exact LSE merges of
// the split partials.  The merges use the kernel's shared memory through its
// struct SM: scratch() / kScratchBytes (the idle stage buffers), merge_m /
// merge_inv / merge_nan_h, tile_slot, tile_base, abort and tr.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;   // CTA size of the decode kernels (the merges share work over it)

// Timeline stamp of thread 0 into the CTA's row (pkv_trace_enable); a uniform
// branch on a kernel parameter when tracing is off.
template <class SM>
__device__ __forceinline__ void trace_stamp(SM& sm, const AttnParams& p, int slot) {
    if (p.trace && threadIdx.x == 0) sm.tr[slot] = globaltimer_ns();
}

// ------------------------------------------------------------------ merges

// Write the neutral state (out = 0, lse = -inf) for every query head of row b.
__device__ void write_neutral_row(const AttnParams& p, int b, int tid, int nthreads) {
    for (int i = tid; i < p.Hq * p.D; i += nthreads) p.out[static_cast<size_t>(b) * p.Hq * p.D + i] = 0.f;
    for (int i = tid; i < p.Hq; i += nthreads) p.lse[static_cast<size_t>(b) * p.Hq + i] = -INFINITY;
}

// Exact LSE merge of the `ns` partial states of (b, kvh) into out / lse
// (M = max_s lse_s, w_s = 2^(lse_s - M) / sum_s 2^(lse_s - M), out = sum_s w_s o_s).
// Must be called by every thread of the CTA.  Partials come from other CTAs,
// so they are read through L2 (ld.cg).  `wsm` is shared scratch of
// kMergeCapFloats floats (the planner keeps ns * G within it).
template <int D, int G>
__device__ void merge_unit(const AttnParams& p, int b, int kvh, int ns, float* wsm, float* m_s, float* inv_s,
                           int* nan_s) {
    const int tid = threadIdx.x, nthreads = blockDim.x;
    const size_t base = static_cast<size_t>(p.row_start[b]) + static_cast<size_t>(kvh) * ns;
    if (tid == 0) *nan_s = 0;
    __syncthreads();
    for (int i = tid; i < ns * G; i += nthreads) {
        const float ls = __ldcg(p.ws_lse + base * G + i);
        if (isnan(ls)) *nan_s = 1;
        wsm[i] = ls;
    }
    __syncthreads();
    if (tid < G) {
        float M = -INFINITY;
        for (int s = 0; s < ns; ++s) M = fmaxf(M, wsm[s * G + tid]);
        float wsum = 0.f;
        if (M != -INFINITY)
            for (int s = 0; s < ns; ++s) wsum += exp2f(wsm[s * G + tid] - M);
        m_s[tid] = M;
        inv_s[tid] = M != -INFINITY ? 1.f / wsum : 0.f;
        const float lse2 = M != -INFINITY ? M + log2f(wsum) : -INFINITY;
        p.lse[static_cast<size_t>(b) * p.Hq + kvh * G + tid] = *nan_s ? NAN : lse2 * kLn2;
    }
    __syncthreads();
    for (int i = tid; i < ns * G; i += nthreads) {
        const int g = i % G;
        wsm[i] = m_s[g] != -INFINITY ? exp2f(wsm[i] - m_s[g]) * inv_s[g] : 0.f;
    }
    __syncthreads();
    const bool nan = *nan_s != 0;
    for (int i = tid; i < G * D / 4; i += nthreads) {
        const int g = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* src = p.ws_o + (base * G + g) * D + d;
#pragma unroll 8
        for (int s = 0; s < ns; ++s) {
            const float w = wsm[s * G + g];
            const float4 o = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(s) * G * D));
            acc.x = fmaf(w, o.x, acc.x);
            acc.y = fmaf(w, o.y, acc.y);
            acc.z = fmaf(w, o.z, acc.z);
            acc.w = fmaf(w, o.w, acc.w);
        }
        if (nan) acc = make_float4(NAN, NAN, NAN, NAN);
        *reinterpret_cast<float4*>(p.out + (static_cast<size_t>(b) * p.Hq + kvh * G + g) * D + d) = acc;
    }
    __syncthreads();
}

// Merge staging geometry: the weights, then the partials, in the idle stage
// buffers; ns <= kMaxSplits take the one-pass path.
template <int D, int G, class SM>
struct MergeCfg {
    static constexpr int kSplitBytes = G * D * 4;
    static constexpr int kWeightBytes = 2048;   // [64][G] floats at most
    static constexpr int kScratch = SM::kScratchBytes;
    static constexpr int kCap = (kScratch - kWeightBytes) / kSplitBytes;
    static constexpr int kMaxSplits = kCap < 64 ? kCap : 64;
    static_assert(64 * G * 4 <= kWeightBytes, "merge staging");
};

// The fused merge of the last-arriving CTA for up to MergeCfg::kMaxSplits
// splits.  The ns partial outputs of (b, kvh) are contiguous in the
// workspace; every thread copies its 16-byte pieces of them into the CTA's
// idle stage buffers with cp.async (the fastest way into one SM: per-thread
// loads are held back by the outstanding-request limit, and the bulk-copy
// engine measured slower).  The LSEs come in meanwhile, one warp per head
// holding splits lane and lane + 32; the max, sum and weights are shuffles.
// The weighted sum runs once everything has landed: T = kThreads / (G*D/4)
// lane groups share one float4 of the output (group `part` taking splits
// part, part + T, ...; a quarter warp reads 128 contiguous bytes), so all
// threads add, and the T part sums are added with a fixed butterfly: the
// result is the same on every launch.  Same arithmetic as merge_unit up to
// the order of the additions; all CTA threads call it.
template <int D, int G, class SM>
__device__ void merge_unit_onepass(SM& sm, const AttnParams& p, int b, int kvh, int ns, int base_slot) {
    using MC = MergeCfg<D, G, SM>;
    constexpr int kOut = G * D / 4;       // float4 outputs of (b, kvh)
    constexpr int T = kThreads / kOut;    // lane groups per output
    constexpr int W = 32 / T;             // outputs per warp
    static_assert(kThreads % kOut == 0 && T >= 1 && T <= 32 && (T & (T - 1)) == 0, "merge lane split");
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int out = warp * W + lane % W, part = lane / W;
    const int g_out = out / (D / 4), d = (out % (D / 4)) * 4;
    const size_t base = static_cast<size_t>(base_slot);
    float* w = reinterpret_cast<float*>(sm.scratch());   // [ns][G] weights
    float* obuf = reinterpret_cast<float*>(sm.scratch() + MC::kWeightBytes);   // [ns][G][D] partials

    const float ls_first = warp < G && lane < ns ? __ldcg(p.ws_lse + (base + lane) * G + warp) : -INFINITY;
    const float ls_first_hi = warp < G && lane + 32 < ns ? __ldcg(p.ws_lse + (base + lane + 32) * G + warp) : -INFINITY;
    {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.ws_o + base * G * D);
        const uint32_t dst = smem_addr(obuf);
        const int vecs = ns * (MC::kSplitBytes / 16);
        for (int i = tid; i < vecs; i += kThreads) cp_async16_plain(dst + i * 16, src + static_cast<size_t>(i) * 16);
    }
    for (int g = warp; g < G; g += kThreads / 32) {
        const float ls = g == warp ? ls_first : lane < ns ? __ldcg(p.ws_lse + (base + lane) * G + g) : -INFINITY;
        const float ls2 =
            g == warp ? ls_first_hi : lane + 32 < ns ? __ldcg(p.ws_lse + (base + lane + 32) * G + g) : -INFINITY;
        const bool nan = __any_sync(kFull, isnan(ls) || isnan(ls2));
        float M = fmaxf(ls, ls2);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
        const float e = M != -INFINITY && lane < ns ? exp2f(ls - M) : 0.f;
        const float e2 = M != -INFINITY && lane + 32 < ns ? exp2f(ls2 - M) : 0.f;
        float wsum = e + e2;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) wsum += __shfl_xor_sync(kFull, wsum, x);
        const float inv = M != -INFINITY ? 1.f / wsum : 0.f;
        if (lane < ns) w[lane * G + g] = e * inv;
        if (lane + 32 < ns) w[(lane + 32) * G + g] = e2 * inv;
        if (lane == 0) {
            sm.merge_nan_h[g] = nan ? 1 : 0;
            const float lse2 = M != -INFINITY ? M + log2f(wsum) : -INFINITY;
            p.lse[static_cast<size_t>(b) * p.Hq + kvh * G + g] = nan ? NAN : lse2 * kLn2;
        }
    }
    cp_async_commit_wait_all();
    __syncthreads();   // every thread's copies and the weights visible
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* ob = obuf + g_out * D + d;
#pragma unroll 2
    for (int s = part; s < ns; s += T) {
        const float ws = w[s * G + g_out];
        const float4 o = *reinterpret_cast<const float4*>(ob + s * G * D);
        acc.x = fmaf(ws, o.x, acc.x);
        acc.y = fmaf(ws, o.y, acc.y);
        acc.z = fmaf(ws, o.z, acc.z);
        acc.w = fmaf(ws, o.w, acc.w);
    }
#pragma unroll
    for (int x = W; x < 32; x <<= 1) {
        acc.x += __shfl_xor_sync(kFull, acc.x, x);
        acc.y += __shfl_xor_sync(kFull, acc.y, x);
        acc.z += __shfl_xor_sync(kFull, acc.z, x);
        acc.w += __shfl_xor_sync(kFull, acc.w, x);
    }
    if (part == 0)
        *reinterpret_cast<float4*>(p.out + (static_cast<size_t>(b) * p.Hq + kvh * G + g_out) * D + d) =
            sm.merge_nan_h[g_out] ? make_float4(NAN, NAN, NAN, NAN) : acc;
    // A later TMA into the stages is ordered after the copies above; every
    // caller that reuses the stages passes a CTA barrier before it does.
    fence_proxy_async_shared();
}

// The fused merge of the last-arriving CTA for more splits than one pass
// holds (MergeCfg::kMaxSplits).  The ns partial outputs of (b, kvh) are
// contiguous in the workspace: every thread copies its share of
// them into the CTA's idle stage buffers with 16-byte cp.async (all in flight
// at once, a chunk of splits at a time), while the LSEs come in with plain L2
// loads; the weighted sum then runs out of shared memory, one float4 of the
// output per thread with independent loads.  Same arithmetic as merge_unit;
// all CTA threads call it.
template <int D, int G, class SM>
__device__ void merge_unit_staged(SM& sm, const AttnParams& p, int b, int kvh, int ns, int base_slot) {
    constexpr int kScratch = SM::kScratchBytes;   // K and V stages
    constexpr int kSplitBytes = G * D * 4;
    constexpr int kOut = G * D / 4;                                            // float4 outputs of (b, kvh)
    constexpr int kPer = (kOut + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const size_t base = static_cast<size_t>(base_slot);
    uint8_t* scratch = sm.scratch();   // k and v stages are adjacent
    float* w = reinterpret_cast<float*>(scratch);                  // [ns][G] weights
    const int w_bytes = (ns * G * 4 + 1023) & ~1023;
    float* obuf = reinterpret_cast<float*>(scratch + w_bytes);     // [chunk][G][D] partials
    const int chunk = (kScratch - w_bytes) / kSplitBytes;

    auto issue = [&](int s0) {   // every thread: its 16-byte pieces of splits [s0, s0 + chunk)
        const int vecs = min(chunk, ns - s0) * (kSplitBytes / 16);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.ws_o + (base + s0) * G * D);
        const uint32_t dst = smem_addr(obuf);
        for (int i = tid; i < vecs; i += kThreads) cp_async16_plain(dst + i * 16, src + static_cast<size_t>(i) * 16);
    };
    const int warp = tid / 32, lane = tid % 32;
    issue(0);
    for (int i = tid; i < ns * G; i += kThreads) w[i] = __ldcg(p.ws_lse + base * G + i);
    __syncthreads();
    // per head: max and sum over the splits, one warp per head
    for (int g = warp; g < G; g += kThreads / 32) {
        float M = -INFINITY;
        bool nan = false;
        for (int s = lane; s < ns; s += 32) {
            nan |= isnan(w[s * G + g]);
            M = fmaxf(M, w[s * G + g]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
        nan = __any_sync(kFull, nan);
        float wsum = 0.f;
        if (M != -INFINITY)
            for (int s = lane; s < ns; s += 32) wsum += exp2f(w[s * G + g] - M);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) wsum += __shfl_xor_sync(kFull, wsum, x);
        if (lane == 0) {
            sm.merge_m[g] = M;
            sm.merge_inv[g] = M != -INFINITY ? 1.f / wsum : 0.f;
            sm.merge_nan_h[g] = nan ? 1 : 0;
            const float lse2 = M != -INFINITY ? M + log2f(wsum) : -INFINITY;
            p.lse[static_cast<size_t>(b) * p.Hq + kvh * G + g] = nan ? NAN : lse2 * kLn2;
        }
    }
    __syncthreads();
    for (int i = tid; i < ns * G; i += kThreads) {
        const int g = i % G;
        w[i] = sm.merge_m[g] != -INFINITY ? exp2f(w[i] - sm.merge_m[g]) * sm.merge_inv[g] : 0.f;
    }
    float4 acc[kPer];
#pragma unroll
    for (int r = 0; r < kPer; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < ns; s0 += chunk) {
        const int n = min(chunk, ns - s0);
        cp_async_commit_wait_all();
        __syncthreads();   // this chunk (and the weights) visible to every thread
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
            const int i = tid + r * kThreads;
            if (i < kOut) {
                const int g = i / (D / 4), d = (i % (D / 4)) * 4;
                const float* wg = w + s0 * G + g;
                const float* og = obuf + g * D + d;
#pragma unroll 8
                for (int s = 0; s < n; ++s) {
                    const float ws = wg[s * G];
                    const float4 o = *reinterpret_cast<const float4*>(og + s * G * D);
                    acc[r].x = fmaf(ws, o.x, acc[r].x);
                    acc[r].y = fmaf(ws, o.y, acc[r].y);
                    acc[r].z = fmaf(ws, o.z, acc[r].z);
                    acc[r].w = fmaf(ws, o.w, acc[r].w);
                }
            }
        }
        if (s0 + chunk < ns) {
            __syncthreads();   // chunk consumed before it is overwritten
            issue(s0 + chunk);
        }
    }
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int i = tid + r * kThreads;
        if (i < kOut) {
            const int g = i / (D / 4), d = (i % (D / 4)) * 4;
            *reinterpret_cast<float4*>(p.out + (static_cast<size_t>(b) * p.Hq + kvh * G + g) * D + d) =
                sm.merge_nan_h[g] ? make_float4(NAN, NAN, NAN, NAN) : acc[r];
        }
    }
    // A later TMA into these stages is ordered after the copies above; every
    // caller that reuses the stages passes a CTA barrier before it does.
    fence_proxy_async_shared();
}

// ------------------------------------------------------------------ tiles of the queue

// Tile of a queue entry: only the entry itself, so the producers can start
// streaming its planned pages at once (all of them are in the row's table).
__device__ __forceinline__ TileWork tile_from_item(const AttnParams& p, const pkv_work_item& it) {
    TileWork tw;
    tw.b = it.b;
    tw.kvh = it.kvh;
    tw.split = it.split;
    tw.page_begin = it.page_begin;
    tw.page_end = it.page_end;
    tw.t0 = it.page_begin * p.page_size;
    tw.t_stream = it.page_end * p.page_size;
    tw.t1 = tw.t_stream;
    tw.slot = 0;
    tw.finalize = 0;
    tw.splits = 0;
    tw.poisoned = 0;
    tw.lazy = 1;
    return tw;
}

// The rest of a queue tile: the row's length clips the token range, and the
// plan is checked against it (a mismatch poisons the tile and flags it).
__device__ __forceinline__ void tile_finish(const AttnParams& p, TileWork& tw) {
    const int n = p.seq_lens[tw.b];
    const int pages = (n + p.page_size - 1) / p.page_size;
    tw.splits = p.row_splits[tw.b];
    const int want_end = min((tw.split + 1) * p.chunk_pages, pages);
    tw.poisoned = (tw.page_begin != tw.split * p.chunk_pages || tw.page_end != want_end) ? 1 : 0;
    if (tw.poisoned && threadIdx.x == 0) atomicOr(&p.ctr->status, static_cast<uint32_t>(PKV_DEV_PLAN_MISMATCH));
    tw.t1 = tw.poisoned ? tw.t0 : min(tw.t_stream, n);
    tw.finalize = tw.splits == 1;
    tw.slot = p.row_start[tw.b] + tw.kvh * tw.splits + tw.split;
    tw.lazy = 0;
}

// After a split tile has written its partial: the last split of (b, kvh) to
// arrive merges all of them (all CTA threads call this).
template <int D, int G, class SM>
__device__ void merge_if_last(SM& sm, const AttnParams& p, int b, int kvh, int ns) {
    // The CTA's partial is written; after the barrier, thread 0's fence makes those
    // writes visible device-wide before its arrival is counted (release), and the
    // arrival's acquire orders the other splits' writes before our reads.  The
    // counter's reset needs no fence: the next launch reads it only after this grid
    // has completed.  (The caller has just passed a barrier too; dropping this one
    // measured slower.)
    __syncthreads();
    if (threadIdx.x == 0) {
        const int u = b * p.Hkv + kvh;
        fence_acq_rel_gpu();
        const uint32_t prev = atom_add_acquire_gpu(&p.arrive[u], 1u);
        const int last = prev == static_cast<uint32_t>(ns - 1);
        if (last) p.arrive[u] = 0;   // ready for the next launch
        sm.tile_slot[1] = last;
        if (p.trace) sm.tr[kTrArrived] = globaltimer_ns();
    }
    __syncthreads();
    if (sm.tile_slot[1]) {
        // the stage buffers are idle here and serve as the merge's scratch
        static_assert(SM::kScratchBytes >= kMergeCapFloats * 4 + 2 * G * D * 4,
                      "merge scratch");
        if (ns <= MergeCfg<D, G, SM>::kMaxSplits)
            merge_unit_onepass<D, G>(sm, p, b, kvh, ns, sm.tile_base);
        else
            merge_unit_staged<D, G>(sm, p, b, kvh, ns, sm.tile_base);
        trace_stamp(sm, p, kTrMergeEnd);
    }
}

// The merge shared by all ns splits of (b, kvh), for a launch whose CTAs are
// all resident at once (cooperative launch of one wave).  Each split publishes
// its partial, waits until all ns have arrived, then merges its own 1/ns share
// of the G*D/4 float4 outputs, lanes over the splits, so each CTA reads only
// its share's columns of every partial (plus the LSEs) instead of one CTA
// reading all of them.  Every split departs once after the
// wait; the last to depart rewinds both counters for the next launch.  Same
// exact LSE rule as merge_unit (all CTA threads call this).
template <int D, int G, class SM>
__device__ void merge_all_splits(SM& sm, const AttnParams& p, int b, int kvh, int split, int ns) {
    __syncthreads();
    const int u = b * p.Hkv + kvh;
    uint32_t* arrive = p.arrive + u;
    uint32_t* depart = p.arrive + static_cast<size_t>(p.B) * p.Hkv + u;
    uint32_t departed = 0;   // thread 0: departures before this one (read after the merge)
    if (threadIdx.x == 0) {
        fence_acq_rel_gpu();   // release: the partial written above, before the arrival
        atomicAdd(arrive, 1u);
        const bool ok = wait_count(arrive, static_cast<uint32_t>(ns), &p.ctr->status, &sm.abort);
        departed = atomicAdd(depart, 1u);
        sm.tile_slot[1] = ok;
        if (p.trace) sm.tr[kTrArrived] = globaltimer_ns();
    }
    __syncthreads();
    const bool ok = sm.tile_slot[1] != 0;
    // This split's share: float4 outputs [i0, i1).  L lanes (a power of two, at
    // most 32, at least ns when ns <= 32) merge one output over the splits, so
    // a warp covers 32 / L outputs per pass and the whole share usually takes
    // one pass: every load of the share is in flight at once.
    constexpr int kItems = G * D / 4;
    const int per = (kItems + ns - 1) / ns;
    const int i0 = split * per, i1 = min(kItems, i0 + per);
    int L = 1;
    while (L < ns && L < 32) L <<= 1;
    const int groups = 32 / L;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane % L, grp = lane / L;
    const size_t base = static_cast<size_t>(sm.tile_base);
    for (int pass = i0; pass < i1; pass += (kThreads / 32) * groups) {   // uniform over the CTA
        const int i = pass + warp * groups + grp;
        const bool live = i < i1;
        const int g = live ? i / (D / 4) : 0, d = live ? (i % (D / 4)) * 4 : 0;
        float m = -INFINITY, l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        int nan = 0;
        if (live) {
            for (int s = sub; s < ns; s += L) {   // the lane's splits, merged online
                const float ls = __ldcg(p.ws_lse + (base + s) * G + g);
                const float4 o = __ldcg(reinterpret_cast<const float4*>(p.ws_o + ((base + s) * G + g) * D + d));
                nan |= isnan(ls) ? 1 : 0;
                if (ls > m) {
                    const float c = exp2f(m - ls);   // m = -inf: 0
                    l *= c;
                    a.x *= c;
                    a.y *= c;
                    a.z *= c;
                    a.w *= c;
                    m = ls;
                }
                if (ls != -INFINITY) {
                    const float e = exp2f(ls - m);
                    l += e;
                    a.x = fmaf(e, o.x, a.x);
                    a.y = fmaf(e, o.y, a.y);
                    a.z = fmaf(e, o.z, a.z);
                    a.w = fmaf(e, o.w, a.w);
                }
            }
        }
        // combine the L lanes of the group (xor partners stay inside it)
        float M = m;
        for (int x = L / 2; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
        const float sc = m != -INFINITY ? exp2f(m - M) : 0.f;
        l *= sc;
        a.x *= sc;
        a.y *= sc;
        a.z *= sc;
        a.w *= sc;
        for (int x = L / 2; x > 0; x >>= 1) {
            l += __shfl_xor_sync(kFull, l, x);
            a.x += __shfl_xor_sync(kFull, a.x, x);
            a.y += __shfl_xor_sync(kFull, a.y, x);
            a.z += __shfl_xor_sync(kFull, a.z, x);
            a.w += __shfl_xor_sync(kFull, a.w, x);
            nan |= __shfl_xor_sync(kFull, nan, x);
        }
        if (live && sub == 0) {
            float4 o;
            float lse2;
            if (nan || !ok) {
                o = make_float4(NAN, NAN, NAN, NAN);
                lse2 = NAN;
            } else if (M == -INFINITY) {
                o = make_float4(0.f, 0.f, 0.f, 0.f);
                lse2 = -INFINITY;
            } else {
                const float inv = 1.f / l;
                o = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                lse2 = M + log2f(l);
            }
            const int h = kvh * G + g;
            *reinterpret_cast<float4*>(p.out + (static_cast<size_t>(b) * p.Hq + h) * D + d) = o;
            if (d == 0) p.lse[static_cast<size_t>(b) * p.Hq + h] = lse2 * kLn2;
        }
    }
    if (threadIdx.x == 0 && departed == static_cast<uint32_t>(ns - 1)) {
        *arrive = 0;   // every split has seen the full count: ready for the next launch
        *depart = 0;
    }
}

}  // namespace
}  // namespace pkv
