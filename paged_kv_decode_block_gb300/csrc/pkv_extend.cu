// pkv_extend.cu -- causal attention of each row's new tokens over its pages
// (pkv_extend), also over the 8-bit cache (pkv_extend_q8).
//
// For new token i of row b (position ctx + i, ctx = len - n) and query head h:
//     s_t = <q, k_t> / sqrt(D), t <= ctx + i;   out = sum_t softmax(s)_t v_t
// computed block by block with a running reference m and sum l:
//     p_t = 2^(c s_t - m),  l += sum p_t,  O += P V;  out = O / l,  lse = ln2 (m + log2 l)
// with c = log2(e) / sqrt(D).  m follows the running maximum only when that has
// grown by more than 8 (p stays below 2^8, which fp32 sums and bf16 weights hold
// as well as 1): most blocks then leave O where it is, in tensor memory.
//
// Shape: the G query heads of a KV head are packed with the tokens into rows, so
// that K and V are read once for all of them.  A tile is 256 rows in two groups
// of 128; one KV block of 128 tokens serves both.  One CTA per SM, specialised
// warps: one loads (TMA), two issue tcgen05.mma, two warpgroups do the softmax with
// a row per thread, and one cleans V where masks end (bf16), or one loads V's codes
// and four widen them to f16 (8-bit).  Scores and outputs stay in tensor
// memory: S0, S1, O0, O1 of 128 columns each; P replaces S, in place, as the
// second product's first operand.  While one group is at its softmax the tensor
// core works for the other.
//
// Bound: a KV head's token is 4 D bytes (8-bit: 2 D) and 4 D operations for each row
// of scores, so above about 280 rows (140) that read the same tokens it is the tensor
// core, 2048 cycles a block at D = 128, and below them HBM.  Measured, 32 query and 8
// KV heads, D = 128, bf16:
//   2048 tokens after 30720          703-783 us   1.37-1.51 PFLOP/s, about 3000 cycles a
//                                                 block: the gap between one group's products
//                                                 and the other's, and the boxes of 16 tokens
//   8 prompts of 128-4096            216 us       0.93 PFLOP/s: a tile of few blocks costs 17
//                                                 thousand cycles besides (its masked blocks,
//                                                 outputs, code that is not in the cache)
//   5 tokens each after 512-32768    55 us        4.6 TB/s: 6 us until the stream runs, 6 us
//                                                 to join the parts
// and e4m3:
//   4 tokens each, 56 rows of 1024-8192   216 us  softmax and widening, a warp's latencies
//   8 rows, chunks of 512                 419 us  the same: 0.87 PFLOP/s
#include "pkv_extend_schedule.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kPieceRing = 4;
constexpr float kMoveAt = 8.0f;    // log2 by which the maximum outgrows the reference

template <int D, bool Q8>
struct Cfg {
    static constexpr int kHalves = D / 64;                    // 128-byte rows per head
    static constexpr int kGroup = kHalves * 1024;             // 8 tokens of a block: [half][8 tokens][128 bytes]
    static constexpr int kTile = kExtBlock * D * 2;           // bytes of a K or V block in bf16
    static constexpr int kCode = kExtBlock * D;               // ... in e4m3
    static constexpr int kQ = kExtRows * D * 2;
    // K and V take turns in one ring (bf16); or K's codes, V's codes and V in f16 have a ring each (8-bit)
    static constexpr int kStages = Q8 ? (D == 128 ? 2 : 4) : (D == 128 ? 5 : 10);
    static constexpr int kKeys = Q8 ? (D == 128 ? 3 : 8) : 0;
    static constexpr int kCodes = Q8 ? (D == 128 ? 3 : 4) : 0;
    static constexpr int kThreads = Q8 ? 512 : 384;
    // [0, 8) softmax; 8-bit: [8, 12) widening; then one warp for loads, two for products, one for values
    static constexpr int kLoad = Q8 ? 12 : 8;
    static constexpr int kMma = kLoad + 1;
    static constexpr int kValues = kLoad + 3;
    static constexpr int kReaders = Q8 ? 15 : 11;             // warps that read the piece ring
    static constexpr int kKeysAt = kQ + kStages * kTile, kCodesAt = kKeysAt + kKeys * kCode;
    static constexpr size_t kBytes = static_cast<size_t>(kCodesAt) + kCodes * kCode;
    // Blocks whose scales are held.  Those of block b + kKeys are written once both groups' scores of block b are
    // there; the softmax then still reads block b's, but is done with those of b - 1.
    static constexpr int kScales = Q8 ? kKeys + 1 : 0;
};

struct alignas(16) Piece {
    int32_t tok0, ntok;     // the tile's tokens in q / out (ntok 0: no more pieces)
    int32_t kvh, b;
    int32_t limit0;         // tokens that the first one sees
    int32_t lo, hi;         // KV blocks
    int32_t slot;           // workspace slot, or -1: the whole tile
    int32_t len;            // the row's tokens
    int32_t bad;            // no products: NaN
    int32_t pad[2];
};
struct Found {              // about a piece, while it is worked on
    volatile int32_t poison;      // a page of it does not exist
    volatile int32_t nonfinite;   // V held infinities or NaN in a block with masked places
};

struct Ctl {
    uint64_t full[10], empty[10], fixed[10];       // blocks in bf16, and V blocks cleaned
    uint64_t key_full[8], key_empty[8];            // blocks of K in e4m3
    uint64_t code_full[4], code_empty[4];          // ... of V
    uint64_t q_split[2];                           // the groups' queries in two e4m3 parts
    uint64_t q_read[2];                            // (D = 64) all of a group's queries are in registers
    uint64_t scale_full[9];
    uint64_t q_full, q_empty, drain;
    uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], pair_full, turn[2];
    // of shared rows: (8-bit, at first) what the first group has scaled the query's parts by; the second group's
    // reference and sum
    union {
        float2 pair_ml[128];
        int64_t scan[20];   // (the schedule, before there are pieces)
    };
    float pair_u[128];      // (8-bit) the second group's reference of O
    uint64_t piece_full[kPieceRing], piece_empty[kPieceRing];
    Piece piece[kPieceRing];
    Found found[kPieceRing];
    ExtRow row;                                    // the row that the CTA's part begins in, its first unit, its index
    int64_t row_unit;
    int32_t row0;
    volatile int abort, late;                      // a wait ran out; one at the end did too
    uint32_t tmem;
    int32_t keys_issued, values_issued;            // blocks whose loads have begun
    int32_t q_loads;
    float scales[1][24];                           // [kScales]: 8 of K, 8 of V, and log2 of their magnitudes
    __device__ __forceinline__ float* scales_of(uint32_t i) { return scales[0] + i * 24; }
};

// Waits for a phase, for at most kWaitLimitNs: then every wait of the CTA gives up, and the kernel's end sets the
// status.  Without a call, which a register split does not allow, and short, as there are many.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    uint32_t start = 0;
    for (uint32_t tries = 1; !mbar_try_wait(bar, parity); ++tries) {
        if (tries % 64) continue;   // (reading the clock would make the wait late)
        if (*abort) return false;
        uint32_t now;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
        now |= 1;
        if (start == 0) start = now;
        if (now - start > static_cast<uint32_t>(kWaitLimitNs)) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// (for all lanes of a warp alike)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(kFull, wait_for(bar, parity, abort));
}

__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t at) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 8-token groups from `group` on of one head: [group][half][8 tokens][64 elements]
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int group, int head, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(head), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void stg256(void* to, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

struct Rows {
    const ExtendParams& p;
    int tt;
    __device__ __forceinline__ ExtRow operator()(int b) const {
        const int32_t lo = p.cu ? p.cu[b] : b, hi = p.cu ? p.cu[b + 1] : b + 1;
        return ext_row(lo, hi, p.seq_lens[b], p.T, static_cast<int64_t>(p.max_pages) * p.page_size, tt);
    }
};

// Exclusive prefix of v over the block's threads; the total in ctl->scan[16].
template <int NT>
__device__ __forceinline__ int64_t block_scan(Ctl* c, int64_t v, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) c->scan[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        const int64_t s = c->scan[i];
        before += i < warp ? s : 0;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// ------------------------------------------------------------------ loads
//
// One warp walks the CTA's part, tells the others its pieces, and loads queries, keys
// and (bf16) values.  It is busy for 100 cycles with each box of a page (16 tokens at
// least), 16 boxes a block.  In the 8-bit cache, whose blocks are half the bytes, that
// was what a block waited for, so a second warp loads the values there (drafts over
// 56 rows of 1024-8192 246 -> 207 us); in bf16 a second warp makes no more room in the
// ring and the two hold one another up (2048 tokens after 30720 723 against 775 us).

// Where a lane finds its boxes of a block: the page of 16 tokens, and its own box's tokens.
struct Boxes {
    const int32_t* row;   // the row's table
    int32_t hi, len, page_size, num_pages, tokens, x, from;
    bool mine;
    __device__ __forceinline__ Boxes(const ExtendParams& p)
        : page_size(p.page_size), num_pages(p.num_pages), tokens(p.box_tokens) {
        const int lane = threadIdx.x & 31, n = kExtBlock / tokens;
        x = lane % n;
        from = x * (tokens / 16);   // the lane that knows its page
        mine = lane < n;
    }
    // the page of this lane's 16 tokens of block j, or -2 past the row's end
    __device__ __forceinline__ int entry(int j) const {
        const uint32_t t = static_cast<uint32_t>(j) * kExtBlock + (threadIdx.x & 7) * 16;
        return j < hi && t < static_cast<uint32_t>(len) ? row[t / static_cast<uint32_t>(page_size)] : -2;
    }
    __device__ __forceinline__ bool ok(int page) const { return page >= 0 && page < num_pages; }
    // the pool's token that this lane's box begins with, or -1: nothing to load
    __device__ __forceinline__ int token(int j, int page) const {
        const int box_page = __shfl_sync(kFull, page, from);
        const uint32_t t = j * kExtBlock + x * tokens;
        return mine && ok(box_page) ? box_page * page_size + static_cast<int>(t % static_cast<uint32_t>(page_size)) : -1;
    }
};

// Loads this lane's box of a block of K or V (`bytes` a box) into `to`, completing on `bar`.
template <bool Q8>
__device__ __forceinline__ void load_block(uint8_t* to, const Boxes& bx, int tok, int bytes, const CUtensorMap* map, int head,
                                           uint64_t* bar, uint64_t policy) {
    const int n = __popc(__ballot_sync(kFull, tok >= 0));
    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(bar, n * bytes);
    __syncwarp();
    if (tok >= 0) {
        if (Q8)
            tma_load_3d(to + bx.x * bytes, map, 0, head, tok, bar, policy);
        else
            tma_load_5d(to + bx.x * bytes, map, tok / 8, head, bar, policy);
    }
}

template <int D, bool Q8>
__device__ __forceinline__ void load(const ExtendParams& p, Ctl* c, uint8_t* smem, const CUtensorMap* qmap,
                                     const CUtensorMap* kmap, const CUtensorMap* vmap, ExtWalk& w, const Rows& rows, uint64_t policy) {
    using C = Cfg<D, Q8>;
    const int lane = threadIdx.x & 31;
    constexpr int kBlock = Q8 ? C::kCode : C::kTile;
    constexpr uint32_t kRing = Q8 ? C::kKeys : C::kStages;
    uint64_t* const full = Q8 ? c->key_full : c->full;
    uint64_t* const empty = Q8 ? c->key_empty : c->empty;
    Boxes bx(p);
    const int bytes = kBlock / (kExtBlock / bx.tokens);
    const int per = kExtRows / 2 / p.G;                             // tokens of a group
    uint32_t blocks = 0, q_loads = 0;
    for (uint32_t pc = 0;; ++pc) {
        ExtPiece e{};
        const bool more = w.next(e, rows);
        const int slot = pc % kPieceRing;
        if (pc >= kPieceRing && !wait_warp(&c->piece_empty[slot], (pc / kPieceRing - 1) & 1, &c->abort)) return;
        Piece& pi = c->piece[slot];
        const ExtRow& r = e.r;
        const int ntok = more ? min(w.tt, r.n - e.tile * w.tt) : 0;
        if (lane == 0) {
            pi.tok0 = r.tok0 + e.tile * w.tt;
            pi.ntok = ntok;
            pi.kvh = e.kvh;
            pi.b = e.b;
            pi.limit0 = r.len - r.n + e.tile * w.tt + 1;
            pi.lo = more ? e.lo : 0;
            pi.hi = more ? e.hi : 0;
            pi.slot = !more || (e.lo == 0 && e.hi == e.blocks) ? -1 : 2 * w.cta + (e.lo == 0 ? 1 : 0);
            pi.bad = more ? r.bad : 0;
            pi.len = more ? r.len : 0;
            c->found[slot].poison = 0;
            c->found[slot].nonfinite = 0;
            if (more && r.bad) atomicOr(p.status, static_cast<uint32_t>(PKV_DEV_PLAN_MISMATCH));
            if (more && e.parts) p.splits[w.cta] = ExtSplit{pi.tok0, ntok, e.kvh, e.parts};
            mbar_arrive(&c->piece_full[slot]);
        }
        __syncwarp();
        if (!more) return;
        if (r.bad) continue;

        bx.row = p.block_table + static_cast<size_t>(e.b) * p.max_pages;
        bx.hi = e.hi;
        bx.len = r.len;
        auto scale = [&](int j, int page) {   // lanes 0..7: K's, 8..15: V's
            if (!Q8 || lane >= 16 || !bx.ok(page)) return 0.0f;
            const uint32_t blk = (j * kExtBlock + (lane & 7) * 16) % static_cast<uint32_t>(p.page_size) / kBlockRows;
            const float x = (lane < 8 ? p.k_scales : p.v_scales)[(static_cast<size_t>(page) * (p.page_size / kBlockRows) + blk) * p.Hkv + e.kvh];
            return lane < 8 || fabsf(x) < INFINITY ? x : __uint_as_float(0x7fffffffu);   // (an infinite scale of V: NaN)
        };
        // pages are asked for two blocks ahead and scales one, so that no block waits for one load behind the other
        int next = bx.entry(e.lo), next2 = bx.entry(e.lo + 1);
        float next_scale = scale(e.lo, next);
        for (int j = e.lo; j < e.hi; ++j, ++blocks) {
            const int page = next;
            const float sc = next_scale;
            next = next2;
            next2 = bx.entry(j + 2);
            next_scale = scale(j + 1, next);
            if (__any_sync(kFull, page != -2 && !bx.ok(page)) && lane == 0) {
                atomicOr(p.status, static_cast<uint32_t>(PKV_DEV_PAGE_OOB));
                c->found[slot].poison = 1;
            }
            const int tok = bx.token(j, page);
            const uint32_t at = Q8 ? blocks : 2 * blocks, st = at % kRing;
            if (at >= kRing && !wait_warp(&empty[st], (at / kRing - 1) & 1, &c->abort)) return;
            if constexpr (Q8) {
                if (lane < 16) c->scales_of(blocks % C::kScales)[lane] = sc;
                if (lane >= 8 && lane < 16) c->scales_of(blocks % C::kScales)[8 + lane] = log2f(fabsf(sc));
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->scale_full[blocks % C::kScales]);
            }
            if (lane == 0) c->keys_issued = blocks + 1;
            load_block<Q8>(smem + (Q8 ? C::kKeysAt : C::kQ) + st * kBlock, bx, tok, bytes, kmap, e.kvh, &full[st], policy);
            if (j == e.lo) {   // the queries, behind the first keys: their place is free later
                if (q_loads > 0 && !wait_warp(&c->q_empty, (q_loads - 1) & 1, &c->abort)) return;
                const int groups = ntok > per ? 2 : 1;
                if (lane == 0) {
                    c->q_loads = q_loads + 1;
                    mbar_arrive_expect_tx(&c->q_full, groups * (C::kQ / 2));
                    for (int g = 0; g < groups; ++g)
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_3d(smem + g * (C::kQ / 2) + h * 16384, qmap, h * 64, e.kvh * p.G,
                                        r.tok0 + e.tile * w.tt + g * per, &c->q_full, policy);
                }
                __syncwarp();
                ++q_loads;
            }
            if (!Q8) {
                const uint32_t vt = (at + 1) % kRing;
                if (at + 1 >= kRing && !wait_warp(&empty[vt], ((at + 1) / kRing - 1) & 1, &c->abort)) return;
                if (lane == 0) c->values_issued = blocks + 1;
                load_block<Q8>(smem + C::kQ + vt * kBlock, bx, tok, bytes, vmap, e.kvh, &full[vt], policy);
            }
        }
    }
}

// The first block with places that some row of the tile does not see.
__device__ __forceinline__ int first_masked(const Piece& pi) { return pi.limit0 / kExtBlock; }

// V of a block with masked places (bf16).  A weight of 0 does not hide an infinity or
// NaN in a product, so V is cleaned before it is used: slots behind the row's end
// (which may hold anything) become 0; so do infinities and NaN of tokens that some
// rows see and others don't, which the rows that see them get back at the end (true
// is returned if there are any).  Rows of the block from `seen` on are not seen by
// all, those from `valid` on lie behind the end.
template <int D>
__device__ __forceinline__ bool clean_values(uint32_t tile, int seen, int valid) {
    using C = Cfg<D, false>;
    const int lane = threadIdx.x & 31;
    constexpr int kPer = C::kHalves * 8;   // 16-byte pieces of a token
    auto at = [&](int i) { return tile + i / (8 * kPer) * C::kGroup + i / 8 % C::kHalves * 1024 + i / kPer % 8 * 128 + i % 8 * 16; };
    uint32_t any = 0;
#pragma unroll 8
    for (int i = seen * kPer + lane; i < valid * kPer; i += 32) {
        uint32_t v[4];
        lds128(v, at(i));
#pragma unroll
        for (int k = 0; k < 4; ++k) any |= (v[k] & 0x7f807f80u) + 0x00800080u;
    }
    const bool odd = __any_sync(kFull, (any & 0x80008000u) != 0);
    if (odd) {
        for (int i = seen * kPer + lane; i < valid * kPer; i += 32) {
            uint32_t v[4];
            lds128(v, at(i));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((v[k] & 0x7f80u) == 0x7f80u) v[k] &= 0xffff0000u;
                if ((v[k] & 0x7f800000u) == 0x7f800000u) v[k] &= 0x0000ffffu;
            }
            sts128(at(i), v[0], v[1], v[2], v[3]);
        }
    }
    for (int i = valid * kPer + lane; i < kExtBlock * kPer; i += 32) sts128(at(i), 0, 0, 0, 0);
    return odd;
}

// bf16: the warp that cleans V in blocks with masked places.
template <int D>
__device__ __forceinline__ void clean(const ExtendParams& p, Ctl* c, uint8_t* smem) {
    using C = Cfg<D, false>;
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    for (uint32_t pc = 0;; ++pc) {
        const int slot = pc % kPieceRing;
        if (!wait_warp(&c->piece_full[slot], (pc / kPieceRing) & 1, &c->abort)) return;
        const Piece pi = c->piece[slot];
        const int hi = pi.bad || pi.ntok == 0 ? pi.lo : pi.hi, masked = first_masked(pi);
        for (int j = pi.lo; j < hi; ++j, n += 2) {
            // (every block is waited for, in order, and its place given back: a parity tells a phase from the next one only,
            // so the ring must not go round without this warp)
            const uint32_t kt = n % C::kStages, vn = n + 1, st = vn % C::kStages;
            if (!wait_warp(&c->full[kt], (n / C::kStages) & 1, &c->abort)) return;
            if (lane == 0) mbar_arrive(&c->empty[kt]);
            if (!wait_warp(&c->full[st], (vn / C::kStages) & 1, &c->abort)) return;
            bool odd = false;
            if (j >= masked) {
                const int first = j * kExtBlock;
                odd = clean_values<D>(smem_addr(smem) + C::kQ + st * C::kTile, max(pi.limit0 - first, 0), min(pi.len - first, kExtBlock));
                fence_proxy_async_shared();
                __syncwarp();
            }
            if (lane == 0) {
                if (odd) c->found[slot].nonfinite = 1;
                if (j >= masked) mbar_arrive(&c->fixed[st]);
                mbar_arrive(&c->empty[st]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->piece_empty[slot]);
        if (pi.ntok == 0) return;
    }
}

// 8-bit: the warp that loads V's codes.
template <int D>
__device__ __forceinline__ void load_values(const ExtendParams& p, Ctl* c, uint8_t* smem, const CUtensorMap* vmap, uint64_t policy) {
    using C = Cfg<D, true>;
    const int lane = threadIdx.x & 31;
    Boxes bx(p);
    const int bytes = C::kCode / (kExtBlock / bx.tokens);
    uint32_t n = 0;
    for (uint32_t pc = 0;; ++pc) {
        const int slot = pc % kPieceRing;
        if (!wait_warp(&c->piece_full[slot], (pc / kPieceRing) & 1, &c->abort)) return;
        const Piece pi = c->piece[slot];
        bx.row = p.block_table + static_cast<size_t>(pi.b) * p.max_pages;
        bx.hi = pi.bad || pi.ntok == 0 ? pi.lo : pi.hi;
        bx.len = pi.len;
        int next = bx.entry(pi.lo), next2 = bx.entry(pi.lo + 1);
        for (int j = pi.lo; j < bx.hi; ++j, ++n) {
            const int tok = bx.token(j, next);
            next = next2;
            next2 = bx.entry(j + 2);
            const uint32_t st = n % C::kCodes;
            if (n >= C::kCodes && !wait_warp(&c->code_empty[st], (n / C::kCodes - 1) & 1, &c->abort)) return;
            if (lane == 0) c->values_issued = n + 1;
            load_block<true>(smem + C::kCodesAt + st * C::kCode, bx, tok, bytes, vmap, pi.kvh, &c->code_full[st], policy);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->piece_empty[slot]);
        if (pi.ntok == 0) return;
    }
}

// ------------------------------------------------------------------ matrix products

// How group g shares in a piece of nb blocks.  Two groups of rows take every block
// up to the last that their own tokens see.  A tile whose rows all fit the first
// group is shared by blocks instead: the first group takes the even ones, the second
// the odd ones of the same rows, and their states are joined at the end, so that a
// short chunk's chain of product, softmax, product runs twice side by side.
struct Share {
    int nb;      // the piece's blocks
    int count;   // this group's
    bool pair;
    int g;
    __device__ __forceinline__ int block(int i) const { return pair ? 2 * i + g : i; }
    __device__ __forceinline__ bool mine(int j) const { return pair ? (j & 1) == g : j < count; }
    __device__ __forceinline__ bool last(int j) const { return pair ? j + 2 >= nb : j + 1 == count; }
};
__device__ __forceinline__ Share share_of(const Piece& pi, int g, int per) {
    Share s;
    s.g = g;
    s.nb = pi.bad || pi.ntok == 0 ? 0 : pi.hi - pi.lo;
    s.pair = s.nb > 1 && pi.ntok <= per;
    const int last = min(pi.ntok, (g + 1) * per) - 1;
    if (s.pair)
        s.count = (s.nb + 1 - g) / 2;
    else
        s.count = s.nb == 0 || last < g * per ? 0 : max(0, min(pi.hi, static_cast<int>(ext_blocks(pi.limit0 + last))) - pi.lo);
    return s;
}

// One thread for each group: the products are asynchronous, and a thread's waits
// hide behind the other's products.  PV(j) goes before QK(j + 1), which overwrites
// its weights.  Where both groups have rows the threads take turns, a block each:
// left alone their products mix, both groups' scores come at the same time, and the
// tensor core rests while both are at their softmax.  Both threads give every block
// back, used or not.
template <int D, bool Q8>
__device__ __forceinline__ void multiply(const ExtendParams& p, Ctl* c, uint8_t* smem, const int g) {
    using C = Cfg<D, Q8>;
    const int per = kExtRows / 2 / p.G;
    constexpr uint32_t kIdQk = Q8 ? umma_idesc_e4m3(kExtBlock) : umma_idesc(kExtBlock, false), kIdPv = umma_idesc(D, true, Q8);
    const uint32_t tS = c->tmem + g * 128, tO = tS + 256, base = smem_addr(smem);
    // descriptors count in 16 bytes: what is added to them never carries out of the address.  The parts of Q and the
    // codes of K are rows of D bytes.
    const uint64_t q_first = Q8 ? umma_desc_bytes<D>(base) : umma_desc(base, 16, 1024),
                   k_desc = Q8 ? umma_desc_bytes<D>(base + C::kKeysAt) : umma_desc(base + C::kQ, 16, C::kGroup),
                   v_desc = umma_desc(base + C::kQ, 1024, C::kGroup);
    uint32_t fixed_phase = 0, q_loads = 0, done = 0, outs = 0, turns = 0, splits = 0;
    struct Place {   // in a ring: the next block's, and its parity
        uint32_t st = 0, phase = 0;
        __device__ __forceinline__ void advance(uint32_t ring) {
            if (++st == ring) st = 0, phase ^= 1;
        }
    } both, keys;
    Place &v = both, &k = Q8 ? keys : both;
    constexpr uint32_t kKeyRing = Q8 ? C::kKeys : C::kStages;
    uint64_t* const key_full = Q8 ? c->key_full : c->full;
    uint64_t* const key_empty = Q8 ? c->key_empty : c->empty;

    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, &c->abort); };
    // (unrolled, with the descriptors' steps as constants: a product takes 64 cycles, and a loop no fewer to issue one;
    // 2048 tokens after 6144 182 us against 230)
    auto qk = [&](uint64_t q_desc, uint32_t at, bool turn) {   // S = Q K^T
        constexpr int kSteps = D / 16;   // bf16: 16 elements each; e4m3: 32, of both parts of Q
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            // (the other thread wakes while the last two products go out)
            if (k == kSteps - 2 && turn) mbar_arrive(&c->turn[1 - g]);
            if constexpr (Q8) {
                const int part = k / (kSteps / 2), step = k % (kSteps / 2);
                umma_ss_e4m3(tS, q_desc + part * (C::kQ / 4 / 16) + step * 2, k_desc + at * (C::kCode / 16) + step * 2, kIdQk, k > 0);
            } else {
                umma_ss(tS, q_desc + (k / 4) * (16384 / 16) + (k % 4) * 2,
                        k_desc + at * (C::kTile / 16) + (k / 4) * (1024 / 16) + (k % 4) * 2, kIdQk, k > 0);
            }
        }
        umma_commit(&c->s_full[g]);
    };
    auto pv = [&](uint32_t at, bool add) {   // O (+)= P V
#pragma unroll
        for (int k = 0; k < kExtBlock / 16; ++k)
            umma_ts(tO, tS + k * 8, v_desc + at * (C::kTile / 16) + k * (2 * C::kGroup / 16), kIdPv, add || k > 0);
    };
    for (uint32_t pc = 0;; ++pc) {
        const int slot = pc % kPieceRing;
        if (!wait(&c->piece_full[slot], (pc / kPieceRing) & 1)) return;
        const Piece pi = c->piece[slot];
        const Share sh = share_of(pi, g, per);
        const int nb = sh.nb, ntok = pi.ntok;
        const int masked = Q8 ? 1 << 30 : first_masked(pi) - pi.lo;
        mbar_arrive(&c->piece_empty[slot]);
        if (ntok == 0) return;
        if (nb == 0) continue;
        const uint64_t q_desc = q_first + (sh.pair ? 0 : g * (C::kQ / 2 / 16));

        const uint32_t q_phase = q_loads++ & 1;
        if (!wait(&c->q_full, q_phase)) return;
        if (Q8 && (g == 0 || sh.pair)) {   // (the loads of a piece's queries follow the products of the last one's)
            if (!wait(&c->q_split[0], q_phase)) return;
        } else if (Q8 && ntok > per) {
            if (!wait(&c->q_split[1], splits++ & 1)) return;
        }
        const bool turn = !sh.pair && ntok > per;   // (both threads find the same)
        bool add = false;
        for (int j = -1; j < nb; ++j) {   // PV of block j, QK of the next
            uint32_t vs = 0;
            if (j >= 0) {
                vs = v.st;
                if (j >= masked) {
                    if (!wait(&c->fixed[vs], (fixed_phase >> vs) & 1)) return;
                    fixed_phase ^= 1u << vs;
                } else if (!wait(&c->full[vs], v.phase)) {
                    return;
                }
                v.advance(C::kStages);
            }
            // (the next keys are there, as a rule, and are asked for while there is time)
            if (j + 1 < nb && !wait(&key_full[k.st], k.phase)) return;
            const bool mine = j >= 0 && sh.mine(j);
            if (mine) {
                if (!add && outs > 0 && !wait(&c->o_empty[g], (outs - 1) & 1)) return;
                if (!wait(&c->p_full[g], done++ & 1)) return;
            }
            if (turn && (g == 1 || turns > 0) && !wait(&c->turn[g], (g == 1 ? turns : turns - 1) & 1)) return;
            tc_fence_after();
            if (mine) {
                pv(vs, add);
                add = true;
                if (sh.last(j)) {
                    umma_commit(&c->o_full[g]);
                    ++outs;
                }
            }
            if (j + 1 < nb && sh.mine(j + 1))
                qk(q_desc, k.st, turn);
            else if (turn)
                mbar_arrive(&c->turn[1 - g]);
            turns += turn;
            if (j >= 0) umma_commit(&c->empty[vs]);
            if (j + 1 < nb) {
                umma_commit(&key_empty[k.st]);
                if (j + 2 == nb) umma_commit(&c->q_empty);
                k.advance(kKeyRing);
            }
        }
    }
}

// ------------------------------------------------------------------ e4m3 to f16

// V's codes become f16, exactly and by one instruction for two; their scales join the
// weights in fp32.  (K's go into the product as they are.)  In blocks with masked
// places NaN codes become 0, as infinities and NaN do in clean_values.
template <int D>
__device__ __forceinline__ void widen(const ExtendParams& p, Ctl* c, uint8_t* smem) {
    using C = Cfg<D, true>;
    const int tid = threadIdx.x & 127, lane = tid & 31;
    constexpr int kPerRow = D / 16;                       // threads of a token
    const int chunk = tid % kPerRow, half = chunk / 4;
    const uint32_t swap = half & 1;                       // the two halves' stores take other banks
    const uint32_t base = smem_addr(smem);
    uint32_t n = 0;
    for (uint32_t pc = 0;; ++pc) {
        const int slot = pc % kPieceRing;
        if (!wait_warp(&c->piece_full[slot], (pc / kPieceRing) & 1, &c->abort)) return;
        const Piece pi = c->piece[slot];
        const int ntok = pi.ntok, lo = pi.lo, hi = pi.bad || ntok == 0 ? pi.lo : pi.hi, masked = first_masked(pi);
        const int len = pi.len;
        for (int j = lo; j < hi; ++j, ++n) {
            const uint32_t cs = n % C::kCodes, st = n % C::kStages;
            if (!wait_warp(&c->code_full[cs], (n / C::kCodes) & 1, &c->abort)) return;
            if (n >= C::kStages && !wait_warp(&c->empty[st], (n / C::kStages - 1) & 1, &c->abort)) return;
            const uint32_t src = base + C::kCodesAt + cs * C::kCode + tid * 16;
            const uint32_t dst = base + C::kQ + st * C::kTile + half * 1024;
            const bool clean = j >= masked;
            const int seen = max(pi.limit0 - j * kExtBlock, 0), valid = len - j * kExtBlock;
            bool odd = false;
            // (a short loop: loads ahead of their use, or two pieces at once, make the code longer, and these warps' and the
            // softmax's together no longer fit the instruction cache: drafts over 56 rows 226 and 230 us against 215)
#pragma unroll 1
            for (int i = 0; i < kPerRow; ++i) {
                uint32_t v[4];
                lds128(v, src + i * 2048);
                if (i + 1 == kPerRow) {   // read: the next codes may come
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c->code_empty[cs]);
                }
                const int row = tid / kPerRow + i * (128 / kPerRow);
                if (clean && row >= seen) {   // rows that not all of the tile's rows see, and what lies behind the row's end
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t nan = ((v[k] & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u) >> 7;
                        odd |= nan != 0 && row < valid;
                        v[k] = row < valid ? v[k] & ~(nan * 0xffu) : 0;
                    }
                }
                // the half that goes first, first
                const uint32_t w[4] = {swap ? v[2] : v[0], swap ? v[3] : v[1], swap ? v[0] : v[2], swap ? v[1] : v[3]};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[2 * k] = e4m3x2_f16x2(static_cast<uint16_t>(w[k]));
                    o[2 * k + 1] = e4m3x2_f16x2(static_cast<uint16_t>(w[k] >> 16));
                }
                const uint32_t first = (chunk % 4) * 2 + swap, at = dst + row / 8 * C::kGroup + row % 8 * 128;
                const uint32_t a0 = at + ((first ^ (row & 7)) << 4);
                sts128(a0, o[0], o[1], o[2], o[3]);
                sts128(a0 ^ 16, o[4], o[5], o[6], o[7]);
            }
            if (clean && __any_sync(kFull, odd) && lane == 0) c->found[slot].nonfinite = 1;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->full[st]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->piece_empty[slot]);
        if (ntok == 0) return;
    }
}

// ------------------------------------------------------------------ queries for e4m3 products

// A row's query, bf16, becomes the sum of two e4m3 numbers in place, times a power of
// two that brings its largest element to [2^7, 2^8): 4 bits of significand and the 4
// that are left, whose last place is e4m3's least step of 2^-9 or more for elements from
// 2^-2 on: those down to 2^-9 of the largest are exact, those below off by at most
// half a step, 2^-17 of the largest.  Two e4m3 products cost what one of bf16 does, and
// the cache's keys go into them untouched; widening K as well as V is twice the work for
// warps that a block waits for already.  `scale` is what the scores are to be multiplied
// by; NaN if an element is not finite.  False: a wait ran out.
template <int D, class Read>
__device__ __forceinline__ bool split_query(uint32_t at, int row, float& scale, const Read& all_read) {
    uint32_t q[D / 2];   // pairs
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        uint32_t v[4];
        lds128(v, at + i / 8 * 16384 + row * 128 + ((i % 8 ^ (row & 7)) << 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) q[4 * i + k] = v[k];
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < D / 2; ++i) most = max(most, max(q[i] & 0x7fff0000u, q[i] << 16 & 0x7fff0000u));
    const uint32_t e = max(most >> 23, 8u);   // exponent of the largest
    const float by = __uint_as_float((261 - e) << 23);
    if (D == 64 && !all_read()) return false;   // rows of 64 bytes lie in other rows' places
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h2[2], l2[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t w = q[8 * i + 2 * k + u];
                const float x = __uint_as_float(w << 16) * by, y = __uint_as_float(w & 0xffff0000u) * by;
                h2[u] = e4m3x2(x, y);
                const F2 b = e4m3x2_f32(static_cast<uint16_t>(h2[u]));
                l2[u] = e4m3x2(x - b.x, y - b.y);
            }
            hi[k] = h2[0] | h2[1] << 16;
            lo[k] = l2[0] | l2[1] << 16;
        }
        // (D = 64: a row is 64 bytes, whose four pieces change places with pairs of rows)
        const uint32_t to = D == 128 ? at + row * 128 + ((i ^ (row & 7)) << 4) : at + row * 64 + ((i ^ (row >> 1 & 3)) << 4);
        sts128(to, hi[0], hi[1], hi[2], hi[3]);
        sts128(to + 128 * D, lo[0], lo[1], lo[2], lo[3]);
    }
    scale = most >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float((e - 7) << 23);
    return true;
}

// ------------------------------------------------------------------ softmax and outputs

// Where a row's results go: out / lse, or the state in a workspace slot.
struct RowOut {
    uint16_t* out;     // null: a workspace slot
    float* lse;
    float4* ws;
    float2* ml;
};
__device__ __forceinline__ RowOut row_out(const ExtendParams& p, const Piece& pi, int row, int shift, int D) {
    RowOut o{};
    if (pi.slot < 0) {
        const int64_t tok = pi.tok0 + (row >> shift);
        const int head = pi.kvh * p.G + (row & (p.G - 1));
        o.out = p.out + tok * p.out_stride + static_cast<int64_t>(head) * D;
        o.lse = p.lse ? p.lse + tok * p.Hq + head : nullptr;
    } else {
        o.ws = reinterpret_cast<float4*>(p.ws_o) + static_cast<size_t>(pi.slot) * (D / 4) * kExtRows + row;
        o.ml = p.ws_ml + static_cast<size_t>(pi.slot) * kExtRows + row;
    }
    return o;
}
// What clean_values took out of V and this row sees, tokens [t0, t1), is added to what
// the row has written: an infinity or NaN of its own value.  Rare, so V is read from
// the pages again.
template <int D, bool Q8>
__device__ __noinline__ void add_nonfinite(const ExtendParams& p, const int32_t* row, int kvh, int t0, int t1, RowOut o) {
    for (int t = t0; t < t1; ++t) {
        const int page = row[t / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;
        const size_t at = ((static_cast<size_t>(page) * p.page_size + t % p.page_size) * p.Hkv + kvh) * D;
        for (int d = 0; d < D; ++d) {
            float v;
            if (Q8) {
                const uint8_t code = static_cast<const uint8_t*>(p.v_pages)[at + d];
                v = (code & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.0f;
            } else {
                v = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.v_pages)[at + d]) << 16);
            }
            if (fabsf(v) <= 3.4e38f) continue;
            if (o.out) {
                const float x = __uint_as_float(static_cast<uint32_t>(o.out[d]) << 16) + v;
                o.out[d] = static_cast<uint16_t>(bf16x2(x, 0.0f));
            } else {
                reinterpret_cast<float*>(o.ws + static_cast<size_t>(d / 4) * kExtRows)[d % 4] += v;
            }
        }
    }
}
__device__ __forceinline__ void write_nan(const RowOut& o, int D) {
    if (o.out) {
        for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(o.out + d) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (o.lse) *o.lse = __uint_as_float(0x7fffffffu);
    } else {
        *o.ml = make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu));
    }
}

// The row's output times f, where it lies.  (The block's product has not begun, and the
// one before is done, as this block's scores came after it.)
template <int D>
__device__ __forceinline__ void rescale(uint32_t tO, float f) {
#pragma unroll 1
    for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        tmem_ld32(o, tO + k);
        tmem_wait_ld();
        tmem_loaded32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st32(tO + k, o);
    }
}

// Scores above the running reference m by more than 2^8 move it: the sum and the
// output follow, for the whole warp.  Rows that do not exist (not `live`) hold the
// queries of other rows of the call, or what another CTA is writing over them: they
// have no say in it.
template <int D>
__device__ __forceinline__ void follow_maximum(float top, bool live, bool first, uint32_t tO, float& m, float& l) {
    if (first) {
        m = top;
    } else if (__any_sync(kFull, live && top > m + kMoveAt)) {
        const float to = fmaxf(m, top);
        const float f = to == -INFINITY ? 1.0f : ex2(m - to);
        l *= f;
        m = to;
        rescale<D>(tO, f);
    }
}

// Scores of a block that the row does not see become -inf, where they lie.
__device__ __forceinline__ void mask_scores(uint32_t tS, int seen) {
    // what every row of the warp sees, and what some row does: a later row sees more
    const int all = __shfl_sync(kFull, seen, 0), most = __shfl_sync(kFull, seen, 31);
#pragma unroll 1
    for (int k = 0; k < kExtBlock; k += 32) {
        if (k + 32 <= all) continue;
        uint32_t s[32];
        if (k >= most) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = 0xff800000u;
        } else {
            tmem_ld32(s, tS + k);
            tmem_wait_ld();
            tmem_loaded32(s);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = i < seen - k ? s[i] : 0xff800000u;
        }
        tmem_st32(tS + k, s);
    }
    tmem_wait_st();
}

// Scores of keys with a scale below 0 change their sign, where they lie (16 columns a scale).
__device__ __forceinline__ void turn_scores(uint32_t tS, const float* scales) {
#pragma unroll 1
    for (int k = 0; k < kExtBlock; k += 32) {
        uint32_t s[32];
        tmem_ld32(s, tS + k);
        tmem_wait_ld();
        tmem_loaded32(s);
        const uint32_t a = __float_as_uint(scales[k / 16]) & 0x80000000u, b = __float_as_uint(scales[k / 16 + 1]) & 0x80000000u;
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] ^= i < 16 ? a : b;
        tmem_st32(tS + k, s);
    }
    tmem_wait_st();
}

// One block of a row's scores to weights: maximum, 2^(c s - m), sum; weights in
// bf16 over the scores.  All 128 scores stay in registers between the two passes.
template <int D>
__device__ __forceinline__ void softmax_block(uint32_t tS, uint32_t tO, float cs, bool live, bool first, float& m, float& l) {
    uint32_t s[128];
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_ld32(s + 32 * k, tS + 32 * k);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_loaded32(s + 32 * k);
    float mx[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 4]));
#pragma unroll
    for (int k = 8; k < 128; k += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], __uint_as_float(s[k + i]), __uint_as_float(s[k + 4 + i]));
    follow_maximum<D>(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs, live, first, tO, m, l);
    const float ref = m == -INFINITY ? 0.0f : -m;
    const uint64_t ref2 = pack2(ref, ref), cs2 = pack2(cs, cs);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 128; k += 32) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const F2 e = unpack2(fma2(pack2(__uint_as_float(s[k + i]), __uint_as_float(s[k + i + 1])), cs2, ref2));
            const float a = ex2(e.x), b = ex2(e.y);
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(a, b));
            w[i / 2] = bf16x2(a, b);
        }
        tmem_st16(tS + k / 2, w);
    }
    const F2 a = unpack2(add2(sum[0], sum[1]));
    l += a.x + a.y;
}

// What a score of codes is multiplied by: the magnitude of K's scale (its sign is in the score) times the row's
// factor.  Not 0, or a score of -inf in a place that is not seen would not stay one; a score is below 2^24, so that
// fp32's least normal number makes as little of it.  A scale that is no number stays none.
__device__ __forceinline__ float key_factor(float scale, float cs) { return max_nan(fabsf(scale) * cs, 0x1p-126f); }
// What a weight is multiplied by: V's scale times by^2.  No product is larger than 2^14, so where the factor is out of
// range the weights that meet it are below 2^-113 and may count for less; but 0 times infinity must not come of it.
__device__ __forceinline__ float value_factor(float scale, float by) {
    return min_nan(max_nan(scale * by * by, -0x1.fffffep127f), 0x1.fffffep127f);
}

// The same over the 8-bit cache: 16 scores share a scale of K, their weights one of
// V.  `scales` has K's 8 (whose signs have gone into the scores) and V's 8; those of
// blocks that the row does not see at all may be anything.
// What goes into the product with V, 2^(c s - m) times V's scale, is rounded to f16
// (11 bits where bf16 has 8: with scales that are no powers of two even the heaviest
// weight is rounded) and has a reference u of its own in log2, since the heaviest token
// may lie in a block of small scale: the largest product of the row is kept from 2^6 to
// 2^14, f16 holds the others to 2^-11 of themselves or 2^-31 of it, and O counts in 2^u.
// (Loops, and the scores read twice: the widening warps leave neither the registers
// nor the room for instructions to do otherwise.  64 columns at a time take 4 to 8 %
// longer; 16 make drafts 4 % faster and chunks of 512 4 % slower.)
template <int D>
__device__ __forceinline__ void softmax_block_q8(uint32_t tS, uint32_t tO, float cs, const float* scales, int seen, bool live,
                                                 bool first, float& m, float& l, float& u) {
    float top = -INFINITY, topv = -INFINITY;
    uint32_t s[32];
#pragma unroll 1
    for (int k = 0; k < 128; k += 32) {
        tmem_ld32(s, tS + k);
        tmem_wait_ld();
        tmem_loaded32(s);
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            const float* y = reinterpret_cast<const float*>(s + i);
            float a = max3(y[0], y[1], y[2]), b = max3(y[3], y[4], y[5]);
            a = max3(a, y[6], y[7]), b = max3(b, y[8], y[9]);
            a = max3(a, y[10], y[11]), b = max3(b, y[12], y[13]);
            a = fmaxf(max3(a, y[14], y[15]), b);
            const float t = a * (k + i < seen ? fabsf(scales[(k + i) / 16]) * cs : 1.0f);   // (finite times 0 at worst)
            top = fmaxf(top, t);
            topv = fmaxf(topv, t + scales[16 + (k + i) / 16]);
        }
    }
    topv -= 6.0f;
    if (first) {
        m = top;
        u = topv;
    } else {
        if (top > m + kMoveAt) {
            l *= ex2(m - top);
            m = top;
        }
        if (__any_sync(kFull, live && topv > u + kMoveAt)) {   // (see follow_maximum)
            const float to = fmaxf(u, topv);
            rescale<D>(tO, to == -INFINITY ? 1.0f : ex2(u - to));
            u = to;
        }
    }
    const float ref = m == -INFINITY ? 0.0f : -m, move = u == -INFINITY ? 0.0f : -ref - u;
    const uint64_t ref2 = pack2(ref, ref);
    // 2^move in two steps, as it may be out of range where the scales are far from 1; beyond 2^252 no product makes a
    // difference in the output, which is at most 2^(23 - move)
    const float by = ex2(fminf(0.5f * move, 126.0f));
    uint64_t sum[2] = {0, 0};
#pragma unroll 1
    for (int k = 0; k < 128; k += 32) {
        tmem_ld32(s, tS + k);
        tmem_wait_ld();
        tmem_loaded32(s);
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            const float ks = k + h < seen ? key_factor(scales[(k + h) / 16], cs) : 1.0f;
            const float vs = k + h < seen ? value_factor(scales[8 + (k + h) / 16], by) : 0.0f;
            const uint64_t ks2 = pack2(ks, ks), vs2 = pack2(vs, vs);
#pragma unroll
            for (int i = h; i < h + 16; i += 2) {
                const F2 e = unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), ks2, ref2));
                const uint64_t y = pack2(ex2(e.x), ex2(e.y));
                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], y);
                const F2 z = unpack2(mul2(y, vs2));
                s[i / 2] = f16x2(z.x, z.y);
            }
        }
        tmem_st16(tS + k / 2, s);
    }
    const F2 a = unpack2(add2(sum[0], sum[1]));
    l += a.x + a.y;
}

template <int D, bool Q8>
__device__ __forceinline__ bool attend(const ExtendParams& p, Ctl* c, uint8_t* smem) {
    using C = Cfg<D, Q8>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = warp >> 2, row = threadIdx.x & 127;
    const int shift = 31 - __clz(p.G), per = kExtRows / 2 >> shift;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // this warp's 32 lanes of tensor memory
    const uint32_t tS = c->tmem + lanes + g * 128, tO = c->tmem + lanes + 256 + g * 128;
    uint32_t done = 0, outs = 0, blocks = 0, pairs = 0, q_loads = 0, splits = 0;
    if (!wait_warp(&c->piece_full[0], 0, &c->abort)) return false;
    Piece next = c->piece[0];   // (read ahead: shared memory is slow beside the products' operands)
    for (uint32_t pc = 0;; ++pc) {
        const int slot = pc % kPieceRing;
        const Piece pi = next;
        if (pi.ntok == 0) return true;
        const Share sh = share_of(pi, g, per);
        const int nb = sh.count, lo = pi.lo;
        const int base_row = sh.pair ? 0 : g * 128;
        const bool live = base_row + row < pi.ntok << shift;                // this thread's row exists
        const bool warp_live = base_row + (row & ~31) < pi.ntok << shift;   // some row of the warp does
        // tokens that the row sees (rows that do not exist: no more than there are, which keeps them within 31 bits)
        const int limit = static_cast<int>(min(static_cast<uint32_t>(pi.limit0) + ((base_row + row) >> shift), static_cast<uint32_t>(pi.len)));
        const int masked = first_masked(pi);
        float m = -INFINITY, l = 0.0f, u = -INFINITY, cs = p.scale_log2;
        if (Q8 && sh.nb > 0) {   // (every piece's load is waited for, and the next one follows every warp: a parity tells a
                                 // phase from the next one only, and in a piece of one block the second group may have no rows)
            const uint32_t phase = q_loads++ & 1;
            if (!wait_warp(&c->q_full, phase, &c->abort)) return false;
            if (lane == 0) mbar_arrive(&c->q_empty);
            if (sh.pair && g == 1) {
                if (!wait_warp(&c->q_split[0], phase, &c->abort)) return false;
                cs *= c->pair_ml[row].x;
            } else if (pi.ntok > g * per) {
                if (D == 64 || warp_live) {
                    // (a barrier of the hardware has no limit: warps that give up would leave the others there)
                    auto all_read = [&] {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c->q_read[g]);
                        return wait_warp(&c->q_read[g], splits++ & 1, &c->abort);
                    };
                    float scale;
                    if (!split_query<D>(smem_addr(smem) + g * (C::kQ / 2), row, scale, all_read)) return false;
                    if (sh.pair) c->pair_ml[row].x = scale;
                    cs *= scale;
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->q_split[g]);
            }
        }
        for (int j = 0; j < nb; ++j) {
            if (!wait_warp(&c->s_full[g], done & 1, &c->abort)) return false;
            ++done;
            tc_fence_after();
            if (warp_live) {
                const int at = lo + sh.block(j);
                const int seen = limit - at * kExtBlock;   // columns of the block that the row sees
                const bool cut = at >= masked;
                const float* scales = nullptr;
                if constexpr (Q8) {
                    const uint32_t b = blocks + sh.block(j);
                    if (!wait_warp(&c->scale_full[b % C::kScales], (b / C::kScales) & 1, &c->abort)) return false;
                    scales = c->scales_of(b % C::kScales);
                }
                if (Q8 && __any_sync(kFull, scales[lane & 7] < 0.0f)) turn_scores(tS, scales);
                if (cut) mask_scores(tS, seen);
                if constexpr (Q8)
                    softmax_block_q8<D>(tS, tO, cs, scales, cut ? seen : kExtBlock, live, j == 0, m, l, u);
                else
                    softmax_block<D>(tS, tO, cs, live, j == 0, m, l);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->p_full[g]);
        }
        blocks += sh.nb;

        const int after = (pc + 1) % kPieceRing;
        if (!wait_warp(&c->piece_full[after], ((pc + 1) / kPieceRing) & 1, &c->abort)) return false;
        next = c->piece[after];

        // outputs
        if (nb > 0) {
            if (!wait_warp(&c->o_full[g], outs & 1, &c->abort)) return false;
            ++outs;
            tc_fence_after();
        }
        float f0 = 1.0f, f1 = 0.0f;   // the two groups' parts of shared rows
        // 8-bit: O counts in 2^u where the sum counts in 2^m; in two steps, as 2^(u - m) may be far off
        auto step = [](float u, float m) { return u == -INFINITY || m == -INFINITY ? 1.0f : ex2(0.5f * (u - m)); };
        float h0 = Q8 ? step(u, m) : 1.0f, h1 = 1.0f;
        if (sh.pair) {
            if (g == 1) {
                c->pair_ml[row] = make_float2(m, l);
                if (Q8) c->pair_u[row] = u;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&c->pair_full);
                    mbar_arrive(&c->piece_empty[slot]);
                }
                continue;
            }
            if (!wait_warp(&c->pair_full, pairs & 1, &c->abort)) return false;
            ++pairs;
            tc_fence_after();
            const float2 other = c->pair_ml[row];
            if (Q8) h1 = step(c->pair_u[row], other.x);
            const float to = fmaxf(m, other.x), ref = to == -INFINITY ? 0.0f : to;
            f0 = ex2(m - ref);
            f1 = ex2(other.x - ref);
            l = l * f0 + other.y * f1;
            m = to;
        }
        const bool poison = pi.bad || c->found[slot].poison;
        if (warp_live) {
            const RowOut o = row_out(p, pi, base_row + row, shift, D);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // (all scores -inf: out 0, lse -inf)
            if (poison) {
                if (live) write_nan(o, D);
            } else if (nb == 0) {
                if (live) *o.ml = make_float2(-INFINITY, 0.0f);   // (only a part of a tile can have nothing to see)
            } else {
                // (a loop: this is run once a tile, and its instructions come from afar)
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t x[32];
                    tmem_ld32(x, tO + k);
                    if (sh.pair) {
                        uint32_t y[32];
                        tmem_ld32(y, tO + 128 + k);
                        tmem_wait_ld();
                        tmem_loaded32(x);
                        tmem_loaded32(y);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = Q8 ? __float_as_uint(__uint_as_float(x[i]) * h0 * (h0 * f0) + __uint_as_float(y[i]) * h1 * (h1 * f1))
                                      : __float_as_uint(__uint_as_float(x[i]) * f0 + __uint_as_float(y[i]) * f1);
                    } else {
                        tmem_wait_ld();
                        tmem_loaded32(x);
                        if (Q8) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * h0 * h0);
                        }
                    }
                    if (live && o.out) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = bf16x2(__uint_as_float(x[2 * i]) * inv, __uint_as_float(x[2 * i + 1]) * inv);
                        if (p.out_wide) {   // whole sectors
                            stg256(o.out + k, x);
                            stg256(o.out + k + 16, x + 8);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<uint4*>(o.out + k + 2 * i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                        }
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            o.ws[static_cast<size_t>((k + i) / 4) * kExtRows] =
                                make_float4(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
                    }
                    __syncwarp();
                }
                if (c->found[slot].nonfinite && live)
                    add_nonfinite<D, Q8>(p, p.block_table + static_cast<size_t>(pi.b) * p.max_pages, pi.kvh,
                                         max(lo, masked) * kExtBlock,
                                         static_cast<int>(min(static_cast<uint32_t>(limit), static_cast<uint32_t>(pi.hi) * kExtBlock)), o);
                if (live && o.out && o.lse) *o.lse = kLn2 * (m + log2f(l));
                if (live && !o.out) *o.ml = make_float2(m, l);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (nb > 0) mbar_arrive(&c->o_empty[g]);
            if (sh.pair) mbar_arrive(&c->o_empty[1]);
            mbar_arrive(&c->piece_empty[slot]);
        }
    }
}

// A wait has run out: everything that this CTA was to write is NaN.
template <int D>
__device__ __noinline__ void poison(const ExtendParams& p, Ctl* c, const ExtParts& parts, const Rows& rows) {
    const int cta = blockIdx.x, tid = threadIdx.x;
    ExtWalk w;
    w.begin(parts, cta, p.B, p.Hkv, rows.tt, c->row0, c->row, c->row_unit);
    ExtPiece e{};
    while (w.next(e, rows)) {
        Piece pi{};
        pi.tok0 = e.r.tok0 + e.tile * w.tt;
        pi.kvh = e.kvh;
        pi.slot = e.lo == 0 && e.hi == e.blocks ? -1 : 2 * cta + (e.lo == 0 ? 1 : 0);
        const int ntok = min(w.tt, e.r.n - e.tile * w.tt);
        if (tid < ntok * p.G) write_nan(row_out(p, pi, tid, 31 - __clz(p.G), D), D);
        if (tid == 0 && e.parts) p.splits[cta] = ExtSplit{pi.tok0, ntok, e.kvh, e.parts};
    }
}

// ------------------------------------------------------------------ the kernel

template <int D, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::kThreads, 1)
extend_kernel(const __grid_constant__ ExtendParams p, const __grid_constant__ CUtensorMap qmap,
              const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D, Q8>;
    extern __shared__ __align__(1024) uint8_t smem[];   // (the swizzle counts from 1024-byte boundaries)
    Ctl* c = reinterpret_cast<Ctl*>(smem + C::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&c->full[i], Q8 ? 4 : 1);
            mbar_init(&c->empty[i], Q8 ? 2 : 3);   // the products' two threads and (bf16) the warp that cleans
            mbar_init(&c->fixed[i], 1);
        }
        for (int i = 0; i < C::kKeys; ++i) {
            mbar_init(&c->key_full[i], 1);
            mbar_init(&c->key_empty[i], 2);
        }
        for (int i = 0; i < C::kCodes; ++i) {
            mbar_init(&c->code_full[i], 1);
            mbar_init(&c->code_empty[i], 4);
        }
        for (int i = 0; i < C::kScales; ++i) mbar_init(&c->scale_full[i], 1);
        mbar_init(&c->q_full, 1);
        mbar_init(&c->q_empty, Q8 ? 2 + 8 : 2);   // the products' two threads and (8-bit) the softmax warps
        mbar_init(&c->drain, 2);
        mbar_init(&c->pair_full, 4);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&c->s_full[g], 1);
            mbar_init(&c->p_full[g], 4);
            mbar_init(&c->o_full[g], 1);
            mbar_init(&c->o_empty[g], 4);
            mbar_init(&c->turn[g], 1);
            mbar_init(&c->q_split[g], 4);
            mbar_init(&c->q_read[g], 4);
        }
        for (int i = 0; i < kPieceRing; ++i) {
            mbar_init(&c->piece_full[i], 1);
            mbar_init(&c->piece_empty[i], C::kReaders);
        }
        c->abort = 0;
        c->late = 0;
        c->keys_issued = c->values_issued = 0;
        c->q_loads = 0;
        fence_mbar_init();
    }
    if (warp == C::kMma) tmem_alloc(&c->tmem, 512);
    if (warp == C::kLoad && lane < 3) prefetch_map(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
    grid_dependency_wait();
    launch_dependents();

    // the CTA's part of the work
    const Rows rows{p, kExtRows / p.G};
    const int cta = blockIdx.x;
    int64_t W = 0, first = -1, run = 0;
    ExtParts parts{};
    // units of all rows, then (with more rows than threads in another pass) the row that holds the part's first
    const int chunks = (p.B + C::kThreads - 1) / C::kThreads;
    for (int i = 0; i < 2 * chunks; ++i) {
        const bool find = i >= chunks;
        const int b = (find ? i - chunks : i) * C::kThreads + tid;
        ExtRow r{};
        if (b < p.B) {
            r = rows(b);
            if (cta == 0 && p.cu && !find && (p.cu[b] < 0 || p.cu[b + 1] < p.cu[b] || p.cu[b + 1] > p.T))
                atomicOr(p.status, static_cast<uint32_t>(PKV_DEV_PLAN_MISMATCH));
        }
        const int64_t units = r.units * p.Hkv;
        int64_t total;
        const int64_t before = run + block_scan<C::kThreads>(c, units, &total);
        run += total;
        if (!find && i + 1 == chunks) {
            W = run;
            if (W == 0) break;
            parts = ext_parts(W, gridDim.x);
            if (cta >= parts.parts) break;
            first = parts.begin(cta);
            run = 0;
        }
        if ((find || chunks == 1) && first >= before && first < before + units) c->row = r, c->row0 = b, c->row_unit = before;
        if (chunks == 1) break;
    }
    const bool work = first >= 0;
    if (tid == 0) p.splits[cta] = ExtSplit{0, 0, 0, 0};
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (work) {
        if (warp < 8) {
            if constexpr (Q8)
                asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
            else
                asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
            if (!attend<D, Q8>(p, c, smem)) {
                poison<D>(p, c, parts, rows);
            }
        } else if (Q8 && warp < 12) {
            if constexpr (Q8) {
                asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
                widen<D>(p, c, smem);
            }
        } else {
            if constexpr (Q8)
                asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
            else
                asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
            uint64_t policy;
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
            if (warp == C::kLoad) {
                ExtWalk w;
                w.begin(parts, cta, p.B, p.Hkv, rows.tt, c->row0, c->row, c->row_unit);
                load<D, Q8>(p, c, smem, &qmap, &kmap, &vmap, w, rows, policy);
            } else if (warp == C::kValues) {
                if constexpr (Q8)
                    load_values<D>(p, c, smem, &vmap, policy);
                else
                    clean<D>(p, c, smem);
            } else if (warp == C::kMma || warp == C::kMma + 1) {
                if (lane == 0) multiply<D, Q8>(p, c, smem, warp - C::kMma);
                __syncwarp();
            }
        }
    }
    __syncthreads();
    if (c->abort && warp == C::kMma + 1 && lane == 0) umma_commit(&c->drain);
    if (c->abort && warp == C::kMma) {   // products and copies in flight land before the memory goes
        if (lane == 0) {
            atomicOr(p.status, static_cast<uint32_t>(PKV_DEV_TIMEOUT));
            umma_commit(&c->drain);
            wait_for(&c->drain, 0, &c->late);
            constexpr uint32_t kRing = Q8 ? C::kKeys : C::kStages, kValueRing = Q8 ? C::kCodes : C::kStages;
            for (uint32_t i = max(c->keys_issued - 10, 0); i < c->keys_issued; ++i) {   // (as many as any ring holds)
                const uint32_t at = Q8 ? i : 2 * i;
                if (at + kRing >= (Q8 ? c->keys_issued : 2 * c->keys_issued))
                    wait_for(Q8 ? &c->key_full[at % kRing] : &c->full[at % kRing], (at / kRing) & 1, &c->late);
            }
            for (uint32_t i = max(c->values_issued - 10, 0); i < c->values_issued; ++i) {
                const uint32_t at = Q8 ? i : 2 * i + 1;
                if (at + kValueRing >= (Q8 ? c->values_issued : 2 * c->values_issued))
                    wait_for(Q8 ? &c->code_full[at % kValueRing] : &c->full[at % kValueRing], (at / kValueRing) & 1, &c->late);
            }
            if (c->q_loads) wait_for(&c->q_full, (c->q_loads - 1) & 1, &c->late);
        }
        __syncwarp();
    }
    if (warp == C::kMma) tmem_free(c->tmem, 512);
}

// ------------------------------------------------------------------ shared tiles joined

// The parts of a tile that several CTAs shared, weighted by 2^(m - max m).  One
// block per CTA that began such a tile and 32 of its rows; lanes are rows (the
// layout in which the states were left).  What it waits for is memory: the
// references and sums of all parts come in one round (warps take parts), then the
// states, of which a warp takes an eighth of the columns with 16 loads in flight (5
// drafted tokens over 8 rows, 150 parts: 5.8 us; with one part behind the other 9.5).
template <int D>
__global__ void __launch_bounds__(256) extend_merge_kernel(const __grid_constant__ ExtendParams p) {
    extern __shared__ float weights[];   // [part][32 rows]; -1: saw nothing, its state was not written
    __shared__ float part_of[2][8][32];
    grid_dependency_wait();
    const ExtSplit sp = p.splits[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + lane;
    if (static_cast<int>(blockIdx.y) * 32 >= sp.ntok * p.G) return;   // (the block as a whole: rows behind the last are done for nothing)
    auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)); };
    float m = -INFINITY;
    bool nan = false;
#pragma unroll 4
    for (int i = warp; i < sp.parts; i += 8) {
        const float2 s = p.ws_ml[slot(i) * kExtRows + row];
        m = fmaxf(m, s.x);
        nan |= s.x != s.x;
    }
    part_of[0][warp][lane] = nan ? __uint_as_float(0x7fffffffu) : m;
    __syncthreads();
    nan = false;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float x = part_of[0][w][lane];
        m = fmaxf(m, x);
        nan |= x != x;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
#pragma unroll 4
    for (int i = warp; i < sp.parts; i += 8) {
        const float2 s = p.ws_ml[slot(i) * kExtRows + row];
        const float f = ex2(s.x - ref);
        weights[i * 32 + lane] = s.y == 0.0f ? -1.0f : f;
        l += s.y * f;
    }
    part_of[1][warp][lane] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += part_of[1][w][lane];
    constexpr int kCols = D / 4 / 8;   // columns (of four) of a warp
    float4 o[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[k] = make_float4(0, 0, 0, 0);
    constexpr int kAtOnce = 16 / kCols;   // (16 loads of a thread in flight; a state that was not written is read too, and left out)
    for (int i0 = 0; i0 < sp.parts; i0 += kAtOnce) {
        float4 x[kAtOnce][kCols];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float4* from = reinterpret_cast<const float4*>(p.ws_o) +
                                 (slot(min(i0 + i, sp.parts - 1)) * (D / 4) + warp * kCols) * kExtRows + row;
#pragma unroll
            for (int k = 0; k < kCols; ++k) x[i][k] = from[static_cast<size_t>(k) * kExtRows];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (i0 + i >= sp.parts) break;
            const float f = weights[(i0 + i) * 32 + lane];
            if (f == -1.0f) continue;
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                o[k].x += x[i][k].x * f, o[k].y += x[i][k].y * f, o[k].z += x[i][k].z * f, o[k].w += x[i][k].w * f;
        }
    }
    if (row >= sp.ntok * p.G) return;
    float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (nan) inv = l = __uint_as_float(0x7fffffffu);
    const int shift = 31 - __clz(p.G);
    const int64_t tok = sp.tok0 + (row >> shift);
    const int head = sp.kvh * p.G + (row & (p.G - 1));
    uint16_t* out = p.out + tok * p.out_stride + static_cast<int64_t>(head) * D + warp * kCols * 4;
#pragma unroll
    for (int k = 0; k < kCols; k += 2)
        *reinterpret_cast<uint4*>(out + 4 * k) = make_uint4(bf16x2(o[k].x * inv, o[k].y * inv), bf16x2(o[k].z * inv, o[k].w * inv),
                                                            bf16x2(o[k + 1].x * inv, o[k + 1].y * inv), bf16x2(o[k + 1].z * inv, o[k + 1].w * inv));
    if (warp == 0 && p.lse) p.lse[tok * p.Hq + head] = kLn2 * (m + log2f(l));
}

template <int D, bool Q8>
cudaError_t launch(const ExtendParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   int ctas, cudaStream_t stream) {
    constexpr size_t kSmem = Cfg<D, Q8>::kBytes + sizeof(Ctl) + Cfg<D, Q8>::kScales * 24 * sizeof(float);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    // (on every call, as a device reset drops it)
    cudaError_t e = cudaFuncSetAttribute(extend_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(Cfg<D, Q8>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, extend_kernel<D, Q8>, p, qmap, kmap, vmap);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ctas, kExtRows / 32);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = static_cast<size_t>(ctas) * 32 * sizeof(float);   // (19 KB: a tile has at most a part on each SM)
    return cudaLaunchKernelEx(&cfg, extend_merge_kernel<D>, p);
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, int ctas, cudaStream_t stream) {
    const bool q8 = p.k_scales != nullptr;
    if (p.D == 128) return q8 ? launch<128, true>(p, qmap, kmap, vmap, ctas, stream) : launch<128, false>(p, qmap, kmap, vmap, ctas, stream);
    return q8 ? launch<64, true>(p, qmap, kmap, vmap, ctas, stream) : launch<64, false>(p, qmap, kmap, vmap, ctas, stream);
}

}  // namespace pkv
