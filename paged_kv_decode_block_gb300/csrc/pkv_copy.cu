// pkv_copy.cu -- pages of a cache copied to other pages, in all of its pools at once
// (pkv_copy_pages).
//
// Pure bytes: each is read once and written once, HBM bounds it.  What a fork or a
// compaction copies is many short stretches (a tail page of a few KB, a block's
// scales of 32 bytes) in many pools, so all of them go into one launch: the list of
// copies and the pools travel as the kernel's parameter (no upload, no memory that a
// later call could overwrite).  A block takes one work item at a time: 32 KB of one
// page, of which the vectors behind the copied tokens cost nothing, or, where pages
// are smaller, that much of the pool's line of (copy, vector of the page).
// 1237 pages of 64 tokens in 8 layers of an 8-bit cache (2.6 GB moved) take 398 us, 6.5
// TB/s; by the line, with less in flight, 428.  64 tails in 64 pools take 25 us on the GPU,
// most of it the launch's parameter and one round of loads and stores; the call on the
// host, which checks and writes the lists, 38-44 (from 33 copies on it marks pages
// in an array of a byte for each page of the pool, so the pool's size counts too).
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                  // vectors of a thread in flight
constexpr int kItem = kThreads * kEach;   // vectors of a work item

__device__ __forceinline__ uint32_t vectors_of(const CopyPool& pool, int32_t tokens) {
    return (tokens + pool.unit_tokens - 1) / pool.unit_tokens * pool.unit_vecs;
}

// A stretch of one page.
template <class V>
__device__ __forceinline__ void copy_stretch(const CopyPool& pool, const pkv_page_copy& cp, uint32_t first) {
    const uint32_t n = vectors_of(pool, cp.tokens);
    const V* from = static_cast<const V*>(pool.data) + static_cast<size_t>(cp.src) * pool.page_vecs;
    V* to = static_cast<V*>(pool.data) + static_cast<size_t>(cp.dst) * pool.page_vecs;
    V v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t k = first + i * kThreads + threadIdx.x;
        if (k < n) v[i] = from[k];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t k = first + i * kThreads + threadIdx.x;
        if (k < n) to[k] = v[i];
    }
}

// A stretch of a pool's line.
template <class V>
__device__ __forceinline__ void copy_line(const CopyPool& pool, const pkv_page_copy* copies, uint32_t first, uint32_t total) {
    V v[kEach];
    V* to[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t at = first + i * kThreads + threadIdx.x;
        to[i] = nullptr;
        if (at >= total) continue;
        const uint32_t c = at / pool.page_vecs, k = at - c * pool.page_vecs;
        const pkv_page_copy cp = copies[c];
        if (k >= vectors_of(pool, cp.tokens)) continue;
        V* base = static_cast<V*>(pool.data);
        to[i] = base + static_cast<size_t>(cp.dst) * pool.page_vecs + k;
        v[i] = base[static_cast<size_t>(cp.src) * pool.page_vecs + k];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (to[i]) *to[i] = v[i];
}

template <class Params>
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ Params p) {
    grid_dependency_wait();
    launch_dependents();
    for (uint32_t item = blockIdx.x; item < p.items; item += gridDim.x) {
        int lo = 0, hi = p.num_pools - 1;   // the pool of this item: the last that begins at or before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (p.pools[mid].first_item <= item)
                lo = mid;
            else
                hi = mid - 1;
        }
        const CopyPool& pool = p.pools[lo];
        const uint32_t at = item - pool.first_item;
        if (pool.stretches) {
            const uint32_t c = at / pool.stretches, first = (at - c * pool.stretches) * kItem;
            if (pool.wide)
                copy_stretch<uint4>(pool, p.copies[c], first);
            else
                copy_stretch<uint32_t>(pool, p.copies[c], first);
        } else if (pool.wide) {
            copy_line<uint4>(pool, p.copies, at * kItem, p.num_copies * pool.page_vecs);
        } else {
            copy_line<uint32_t>(pool, p.copies, at * kItem, p.num_copies * pool.page_vecs);
        }
    }
}

// The parameter of a launch: few copies and pools, or as many as a parameter holds.
template <int kCopies, int kPools>
struct CopyParams {
    CopyPool pools[kPools];
    pkv_page_copy copies[kCopies];
    uint32_t items;
    int32_t num_pools, num_copies;
};

template <int kCopies, int kPools>
cudaError_t launch(const CopyPool* pools, int num_pools, const pkv_page_copy* copies, int num_copies, int num_sms,
                   cudaStream_t stream) {
    using Params = CopyParams<kCopies, kPools>;
    static_assert(sizeof(Params) <= 32764, "a kernel's parameters");
    Params p;
    p.num_pools = num_pools;
    p.num_copies = num_copies;
    uint32_t items = 0;
    for (int i = 0; i < num_pools; ++i) {
        p.pools[i] = pools[i];
        p.pools[i].first_item = items;
        // pages of at least half an item are taken one by one
        p.pools[i].stretches = pools[i].page_vecs >= kItem / 2 ? (pools[i].page_vecs + kItem - 1) / kItem : 0;
        items += p.pools[i].stretches ? num_copies * p.pools[i].stretches
                                      : (static_cast<uint32_t>(num_copies) * pools[i].page_vecs + kItem - 1) / kItem;
    }
    p.items = items;
    for (int i = 0; i < num_copies; ++i) p.copies[i] = copies[i];
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(items < static_cast<uint32_t>(num_sms) * 8 ? items : num_sms * 8);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_kernel<Params>, p);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPool* pools, int num_pools, const pkv_page_copy* copies, int num_copies,
                              int num_sms, cudaStream_t stream) {
    for (int at = 0; at < num_pools; at += kCopyMaxPools) {
        const int np = num_pools - at < kCopyMaxPools ? num_pools - at : kCopyMaxPools;
        uint32_t widest = 1;
        for (int i = 0; i < np; ++i) widest = pools[at + i].page_vecs > widest ? pools[at + i].page_vecs : widest;
        // copies of a launch: within a parameter, and vectors and items within 32 bits
        const uint32_t room = 0x7fffffffu / kCopyMaxPools / widest;
        const int most = room < static_cast<uint32_t>(kCopyMaxCopies) ? (room ? static_cast<int>(room) : 1) : kCopyMaxCopies;
        for (int c = 0; c < num_copies; c += most) {
            const int nc = num_copies - c < most ? num_copies - c : most;
            const cudaError_t e = np <= 64 && nc <= 64 ? launch<64, 64>(pools + at, np, copies + c, nc, num_sms, stream)
                                                       : launch<kCopyMaxCopies, kCopyMaxPools>(pools + at, np, copies + c, nc, num_sms, stream);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace pkv
