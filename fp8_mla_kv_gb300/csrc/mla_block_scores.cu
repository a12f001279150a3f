// mla_block_scores: how much each token's heads want each complete block before the token's own,
//   score[t, b] = sum over heads h of softmax over b of (sm_scale q[t, h] . K_b),
// K_b the mean keys of mla_block_keys.
//
// A product of two matrices with a softmax over its rows and a sum over its rows' heads, on tcgen05: a tile is 128
// (token, head) rows of one sequence, its columns are the sequence's blocks, 256 of them in fp32 in tensor memory, where
// they stay until the rows' sums are known: nothing is multiplied twice or goes through memory. Up to
// eight CTAs (a cluster) take a tile's columns in parts and exchange the rows' maxima and sums through
// their shared memory; beyond 2,048 blocks a CTA has several rounds of 256 and multiplies twice.
// A warp's 32 rows are whole tokens where a token has at most 32 heads (lanes left over stay empty), so that the sum
// over heads is one warp's; two or four warps share a token with more.
//
// Roles: warps 0-7 softmax (TMEM lanes 32 (w % 4) .., every other 16 columns), 8-11 copy keys, 12 q, 13 issues the
// products. q comes by TMA in boxes of 32 rows x 64 dims, one for each lane quarter; keys, which lie wherever the block table
// says, by 16 bytes a thread and time (cp.async): TMA's gather of four rows took 41,000 cycles for what boxes take 15,000.
// Both in 128-byte-swizzled tiles of 128 rows through a ring each, for each 64 dims one of q and up to two of keys.
//
// 4,096 tokens of 16 heads with up to 255 blocks: 37.1 us; 32 tokens of 128 heads with up to 1,024: 15.4 us. In both a CTA
// takes 24,000 to 30,000 cycles, one after the other: 5,000 until the first operands are asked for, 10,000 to 16,000 of products
// (the first: what an SM gets from L2, 96 KB a step of 64 dims for its two CTAs in 1,700 cycles; the second: memory, as each step asks
// for 128 bytes of every row; one product of 256 columns a step instead of two of 128: 38.3 us), 9,000 to 11,000 of softmax, exchange and sums, and the first case has 512 tiles for 304 places.
// Keys by TMA gather 135 us, copies that fence each tile 97, four softmax warps 80; q and keys prefetched into L2 by
// rows: no faster.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include <cuda.h>

#include "mla_seq.cuh"

namespace {

using namespace mla;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSoftWarps = 8, kLoadWarps = 4, kLoadWarp = kSoftWarps, kQWarp = kLoadWarp + kLoadWarps, kMmaWarp = kQWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kRows = 128;                                 // M
constexpr int kCols = 256;                                 // columns a round: tensor memory of a CTA
constexpr int kTileKeys = 128;                             // keys per ring tile
constexpr int kTileBytes = 128 * 128;
constexpr int kSlots = 6;                                  // of both rings: two CTAs an SM
constexpr int kMostKeySlots = 4, kMostQSlots = 3;
constexpr int kMaxCluster = 8;

constexpr int kOffRing = 0;
constexpr int kStep = 16;                                  // columns that a softmax warp takes at a time
constexpr int kOffTurn = kOffRing + (kSlots - 1) * kTileBytes;     // per softmax warp kStep columns x 32 rows: where the last slot is
static_assert(kSoftWarps * kStep * 32 * 4 <= kTileBytes, "the turned scores have the place of a tile");
constexpr int kOffJoin = kOffRing + kSlots * kTileBytes;   // per lane quarter and column: parts of a token's sum
constexpr int kOffMax = kOffJoin + 4 * kCols * 4;          // per half of the softmax warps and row: maximum and sum, read by the cluster
constexpr int kOffSeen = kOffMax + 2 * kRows * 8;          // per token: blocks that it sees
constexpr int kOffOff = kOffSeen + kRows * 4;              // per kStep columns and row: the maximum that its exponentials go by
constexpr int kOffBars = kOffOff + (kCols / kStep) * kRows * 4;
constexpr int kNumBars = 2 * kMostKeySlots + 2 * kMostQSlots + 3;
constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) & ~15;
constexpr int kSmem = kOffMisc + 16;
static_assert(2 * (kSmem + 2048) <= 228 * 1024, "two CTAs an SM, each with 1 KB of find_unit's and 1 KB of the system's");

struct ScoreArgs {
    Batch b;
    const __nv_bfloat16* keys;
    float* scores;
    int H, d_qk, num_keys;
    int tile_tokens;                                       // tokens a tile
    int least;                                             // columns that a CTA takes at least
    int cluster;
    float scale_log2;
};

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16: fp32 D, BF16 A and B, both K-major, M = 128, N.
__device__ __forceinline__ uint32_t idesc(uint32_t n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((kRows >> 4) << 24);
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)) : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 lanes x 32 bits, 16 columns: thread t gets lane t, columns c .. c + 15.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    // (the registers pass through, so that no use of them is scheduled before the wait)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Where a role is in a ring: the slot and how often it has come round (the parity of a wait).
struct Turn {
    int slot = 0;
    uint32_t parity = 0u;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// Dims x .. x + 63 of rows y .. y + 31.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
// 16 bytes to shared memory, zeros where there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Arrives at the barrier when all of this thread's copies so far have landed. (The order to the products, which read
// through another proxy, is made by the thread that waits: a fence here would wait for the copies behind, too.)
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 peer_float2(uint32_t saddr, int rank) {
    uint32_t at;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void put_shared(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" :: "r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ float get_shared(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 get_shared4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
// One thread of the warp; ptxas knows that it is one.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A bounded wait that also ends as soon as another role has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag != 0) return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag));
}

// kSixteen: two tokens a warp, as whose rows the sums run without a look at the heads; kFew: fewer than 32 heads; kMany: 32 and more.
enum Heads { kSixteen, kFew, kMany };

template <int kHeads>
__global__ void __launch_bounds__(kThreads, 2)
block_scores_kernel(const __grid_constant__ CUtensorMap q_map, const ScoreArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    float* const turn = reinterpret_cast<float*>(smem + kOffTurn);
    float* const join = reinterpret_cast<float*>(smem + kOffJoin);
    float2* const max_s = reinterpret_cast<float2*>(smem + kOffMax);             // [2][kRows]
    int* const seen_s = reinterpret_cast<int*>(smem + kOffSeen);
    float* const off_s = reinterpret_cast<float*>(smem + kOffOff);              // [kCols / kStep][kRows]
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + kOffBars);        // [kMostKeySlots] a tile copied
    uint64_t* const empty = full + kMostKeySlots;                               // [kMostKeySlots] its products are done
    uint64_t* const qfull = empty + kMostKeySlots;                              // [kMostQSlots] the same for q
    uint64_t* const qempty = qfull + kMostQSlots;
    uint64_t* const dfull = qempty + kMostQSlots;                               // a round's products are done
    uint64_t* const dfree = dfull + 1;                                          // and have been read
    uint64_t* const fin = dfree + 1;                                            // all products are done
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    // (while the first loads are on their way; find_unit's barriers are these writes' too)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMostKeySlots; ++i) {
            mbar_init(&full[i], 32 * kLoadWarps);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMostQSlots; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], 1);
        }
        mbar_init(dfull, 1);
        mbar_init(dfree, kSoftWarps);
        mbar_init(fin, 1);
        *abort_flag = (smem_u32(smem) & 1023u) != 0u;      // (the operands' layout would be off: no result)
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    if (blockIdx.x == 0) check_lengths(a.b);
    const int rank = a.cluster > 1 ? static_cast<int>(blockIdx.x) % a.cluster : 0;
    const int2 u = find_unit<kThreads>(a.b.n_seq, static_cast<int>(blockIdx.x) / a.cluster, [&](int s) {
        return parts_of(sequence_of(a.b, s).n, a.tile_tokens);
    });
    tc_after();
    const uint32_t tmem = *tmem_slot;
    auto give_back = [&]() {
        if (warp == kMmaWarp)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kCols) : "memory");
    };
    if (u.x < 0) return give_back();                       // (all CTAs of a cluster have the same tile)
    const Sequence q = sequence_of(a.b, u.x);
    const int first = u.y * a.tile_tokens, n_tokens = min(a.tile_tokens, q.n - first);
    const int last = position_of(a.b, q, first + n_tokens - 1);
    const int blocks = last < 0 ? 0 : last / a.b.page_size;            // the tile's columns
    if (blocks == 0) return give_back();
    // This CTA's: [c0, c0 + cols)
    const int share = (parts_of(blocks, a.cluster) + 15) & ~15;
    const int per = max(a.least, share), c0 = static_cast<int>(min(static_cast<int64_t>(blocks), static_cast<int64_t>(rank) * per));
    const int cols = min(per, blocks - c0);
    if (cols == 0) return give_back();                     // (its peers know: they neither wait for it nor read its maxima)
    const int peers = parts_of(blocks, per);               // CTAs of the cluster with columns
    const int rounds = (cols + kCols - 1) / kCols, passes = rounds > 1 ? 2 : 1;
    const int n_dims = a.d_qk / 64;
    // The rings hold two steps of 64 dims with two tiles of keys each, or three with one. With one round the copies are over when the
    // scores are turned; with more, the last slot is kept free for that.
    const int key_slots = cols > kTileKeys && rounds == 1 ? 4 : 3, q_slots = rounds == 1 ? kSlots - key_slots : 2;
    const int q_off = kOffRing + key_slots * kTileBytes;

    bool ok = *abort_flag == 0;

    // Row r of the tile: lane r % 32 of warp r / 32. Tokens of at most 32 heads stand side by side in a warp.
    const int H = kHeads == kSixteen ? 16 : a.H;
    const int heads_warps = kHeads != kMany || H <= 32 ? 1 : H <= 64 ? 2 : 4;      // warps of a token
    const int per_warp = kHeads != kMany ? 32 / H : 1;                 // tokens of a warp
    auto row_of = [&](int r, int& token, int& head) {                  // false: an empty lane
        const int w = r >> 5, l = r & 31;
        if (heads_warps == 1) {
            token = w * per_warp + l / H;
            head = l % H;
            return l < per_warp * H && token < n_tokens;
        }
        token = w / heads_warps;
        head = (w % heads_warps) * 32 + l;
        return head < H && token < n_tokens;
    };

    if (warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps) {
        // ---- keys: thread = 16-byte unit x of 64 dims, rows y + 16 i of each tile ----
        const int id = threadIdx.x - 32 * kLoadWarp, x = id & 7, y = id >> 3;
        const int32_t* bt = a.b.block_table + static_cast<int64_t>(u.x) * a.b.max_pages + c0;
        const uint32_t ring = smem_u32(smem) + kOffRing + 128 * y + ((x ^ (y & 7)) << 4);      // (16 i leaves y & 7)
        Turn at;
        at.parity = 1u;                                    // (a slot's first wait is over at once)
        for (int pass = 0; pass < passes; ++pass) {
            for (int r = 0; r < rounds && ok; ++r) {
                const int n = min(kCols, cols - r * kCols);
                const __nv_bfloat16* src[2][8];
                uint32_t there = 0u;
                bool odd = false;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = kTileKeys * t + y + 16 * i;
                        const int32_t page = c < n ? __ldg(bt + r * kCols + c) : -1;
                        odd = odd || page >= a.num_keys;
                        const bool has = page >= 0 && page < a.num_keys;
                        there |= (has ? 1u : 0u) << (8 * t + i);
                        src[t][i] = a.keys + static_cast<int64_t>(has ? page : 0) * a.d_qk + 8 * x;
                    }
                if (odd) atomicOr(a.b.err, MLA_ERR_PAGE_RANGE);
#pragma unroll 1
                for (int k = 0; k < n_dims && ok; ++k) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int rows = (n - kTileKeys * t + 15) & ~15;       // as many as the product takes
                        if (rows <= 0) break;
                        ok = ok && warp_wait(&empty[at.slot], at.parity, abort_flag);
                        if (ok) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (y + 16 * i < rows)
                                    copy16(ring + at.slot * kTileBytes + 2048 * i, src[t][i] + 64 * k, ((there >> (8 * t + i)) & 1u) != 0u);
                            copies_arrive(&full[at.slot]);
                        }
                        at.next(key_slots);
                    }
                }
            }
            if (pass == 0 && a.cluster > 1) cluster_sync();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");   // (a call that failed may have some on their way)
    } else if (warp == kQWarp) {
        // ---- q: lane l < 4 the box of lane quarter l ----
        int q_row = 0;
        if (lane < 4)
            q_row = heads_warps == 1 ? (q.start + first + lane * per_warp) * H
                                     : (q.start + first + lane / heads_warps) * H + 32 * (lane % heads_warps);
        q_row = min(q_row, a.b.T * H - 1);               // (a box of none of the tile's tokens)
        Turn at;
        at.parity = 1u;
        int issued = 0;
        for (int pass = 0; pass < passes; ++pass) {
            for (int r = 0; r < rounds && ok; ++r)
                for (int k = 0; k < n_dims && ok; ++k, ++issued) {
                    ok = warp_wait(&qempty[at.slot], at.parity, abort_flag);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&qfull[at.slot], kTileBytes);
                    __syncwarp();
                    if (lane < 4)
                        copy_box(smem + q_off + at.slot * kTileBytes + lane * (kTileBytes / 4), &q_map, 64 * k, q_row, &qfull[at.slot]);
                    at.next(q_slots);
                }
            if (pass == 0 && a.cluster > 1) cluster_sync();
        }
        // Copies in flight land before the CTA ends.
        if (!ok)
            for (int i = max(0, issued - q_slots); i < issued; ++i)
                (void)mbar_wait_bounded(&qfull[i % q_slots], static_cast<uint32_t>((i / q_slots) & 1));
    } else if (warp == kMmaWarp) {
        // ---- products, one elected thread ----
        Turn at, q_at;                                     // (the elected thread is the same each time)
        const uint32_t d_ring = smem_u32(smem) + kOffRing, d_q = smem_u32(smem) + q_off;
        for (int pass = 0; pass < passes; ++pass) {
            if (elect_one()) {
                for (int r = 0; r < rounds && ok; ++r) {
                    const int n = min(kCols, cols - r * kCols), tiles = n > kTileKeys ? 2 : 1;
                    const int round = pass * rounds + r;
                    if (round > 0) ok = wait_or_abort(dfree, static_cast<uint32_t>((round - 1) & 1), abort_flag);
                    tc_after();
                    const uint32_t id0 = idesc((min(kTileKeys, n) + 15) & ~15), id1 = idesc((n - kTileKeys + 15) & ~15);
                    for (int k = 0; k < n_dims && ok; ++k) {
                        ok = wait_or_abort(&qfull[q_at.slot], q_at.parity, abort_flag);
                        const uint64_t dq = sw128_desc(d_q + q_at.slot * kTileBytes);
                        for (int t = 0; t < tiles && ok; ++t) {
                            ok = wait_or_abort(&full[at.slot], at.parity, abort_flag);
                            if (!ok) break;
                            fence_proxy_async_smem();
                            tc_after();
                            const uint64_t dk = sw128_desc(d_ring + at.slot * kTileBytes);
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                umma(tmem + kTileKeys * t, dq + static_cast<uint64_t>(2 * s), dk + static_cast<uint64_t>(2 * s),
                                     t == 0 ? id0 : id1, k > 0 || s > 0);
                            umma_commit(&empty[at.slot]);
                            at.next(key_slots);
                        }
                        if (ok) umma_commit(&qempty[q_at.slot]);
                        q_at.next(q_slots);
                    }
                    if (ok) umma_commit(dfull);
                }
                if (pass + 1 == passes) {                  // before tensor memory is freed
                    umma_commit(fin);
                    (void)mbar_wait_bounded(fin, 0);
                }
            }
            __syncwarp();
            if (pass == 0 && a.cluster > 1) cluster_sync();
        }
    } else {
        // ---- softmax: thread = row, of its quarter's columns every other kStep ----
        const int quarter = warp & 3, half = warp >> 2;
        const int row = 32 * quarter + lane;
        int token, head;
        const bool lives = row_of(row, token, head);
        const int pos = lives ? position_of(a.b, q, first + token) : -1;
        const int seen = (pos < 0 ? 0 : pos / a.b.page_size) - c0;         // columns of this CTA that the row sees
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const int32_t* bt = a.b.block_table + static_cast<int64_t>(u.x) * a.b.max_pages + c0;
        if (lives && head == 0) seen_s[token] = seen + c0;                 // (by both halves: the same)
        float m = -INFINITY, l = 0.0f;
        // Which of a round's columns have a key: lane j gets the bits of columns 32 j ..
        auto keyed_columns = [&](int r) {
            int32_t page[kCols / 32];
#pragma unroll
            for (int j = 0; j < kCols / 32; ++j) {
                const int c = r * kCols + 32 * j + lane;
                page[j] = c < cols ? __ldg(bt + c) : -1;
            }
            uint32_t mine = 0u;
#pragma unroll
            for (int j = 0; j < kCols / 32; ++j) {
                const uint32_t word = __ballot_sync(0xffffffffu, page[j] >= 0 && page[j] < a.num_keys);
                if (lane == j) mine = word;
            }
            return mine;
        };
        uint32_t keyed = 0u;
        // The bits of the kStep columns j.
        auto keyed_step = [&](int j) { return (__shfl_sync(0xffffffffu, keyed, j >> 1) >> (kStep * (j & 1))) & 0xffffu; };
        // Scores of the row in log2 units, -inf where it sees no block.
        auto load = [&](int r, int j, float (&x)[kStep]) {
            uint32_t v[kStep];
            tmem_ld16(lanes + kStep * j, v);
            const int left = seen - (r * kCols + kStep * j);
            const uint32_t word = keyed_step(j);
            const uint32_t sees = left >= kStep ? word : left <= 0 ? 0u : word & ((1u << left) - 1u);
#pragma unroll
            for (int c = 0; c < kStep; ++c) x[c] = __uint_as_float(v[c]) * a.scale_log2;
            if (!__all_sync(0xffffffffu, sees == 0xffffu)) {
#pragma unroll
                for (int c = 0; c < kStep; ++c) x[c] = ((sees >> c) & 1u) != 0u ? x[c] : -INFINITY;
            }
        };
        for (int r = 0; r < rounds; ++r) {
            keyed = keyed_columns(r);
            ok = warp_wait(dfull, static_cast<uint32_t>(r & 1), abort_flag);
            ok = !bar_sync_or(1, 32 * kSoftWarps, !ok);        // one answer for all of these warps
            if (!ok) break;
            tc_after();
            const int steps = (min(kCols, cols - r * kCols) + kStep - 1) / kStep;
#pragma unroll 1
            for (int j = half; j < steps; j += 2) {
                float x[kStep];
                load(r, j, x);
                float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kStep; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                const float off = now == -INFINITY ? 0.0f : now;
                l *= ex2_approx(m - off);                  // (nothing so far: l is 0)
                m = now;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                uint32_t v[kStep];
#pragma unroll
                for (int c = 0; c < kStep; ++c) {
                    const float p = ex2_approx(x[c] - off);
                    sum[c & 3] += p;
                    v[c] = __float_as_uint(p);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (rounds == 1) {
                    tmem_st16(lanes + kStep * j, v);
                    off_s[j * kRows + row] = m;
                }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dfree);
        }
        // Maxima and sums of both halves, of all CTAs
        max_s[half * kRows + row] = make_float2(m, l);
        float all_m = -INFINITY, all_l = 0.0f;
        auto add = [&](float2 v) {
            const float now = fmaxf(all_m, v.x), to = now == -INFINITY ? 0.0f : now;
            all_l = all_l * ex2_approx(all_m - to) + v.y * ex2_approx(v.x - to);       // (0 x 0 where there is nothing)
            all_m = now;
        };
        float2* const all_s = reinterpret_cast<float2*>(turn);
        if (a.cluster > 1) {
            cluster_sync();
            const uint32_t at = smem_u32(&max_s[half * kRows + row]);
            for (int k = 0; k < peers; ++k) add(peer_float2(at, k));
            all_s[half * kRows + row] = make_float2(all_m, all_l);             // (a half's, of all CTAs)
            all_m = -INFINITY;
            all_l = 0.0f;
        }
        bar_sync_or(1, 32 * kSoftWarps, false);
        const float2* const both = a.cluster > 1 ? all_s : max_s;
        add(both[row]);
        add(both[kRows + row]);
        if (a.cluster > 1) bar_sync_or(1, 32 * kSoftWarps, false);             // (the scores are turned there)
        // p = exp2(x - off) x f; with one round exp2(x - a maximum so far) is in tensor memory
        const float off = all_m == -INFINITY ? 0.0f : all_m;
        const float f = lives ? 1.0f / (all_l == 0.0f ? 1.0f : all_l) : 0.0f;
        // Row r of column c at 16-byte unit r / 4 ^ c % 8 of the column: neither a column's rows nor eight columns' units
        // meet a bank twice.
        const uint32_t mine = smem_u32(turn) + warp * kStep * 128;     // (a multiple of 1,024: bits 4 .. 6 are the unit's)
        // What the lane sums and stores: column lane % kStep, and of the warp's tokens every other one, or half of the rows of one.
        const int col = lane & (kStep - 1), part = lane / kStep;
        const uint32_t put = mine + 4 * lane, get = mine + 128 * col + ((col & 7) << 4);
        const int my_token = kHeads != kMany ? quarter * per_warp + part : quarter / heads_warps;     // (16 heads, or 32 and more)
        const int my_end = my_token < n_tokens ? min(seen_s[my_token], c0 + cols) - (c0 + col) : 0;
        float* const my_scores = a.scores + (static_cast<int64_t>(q.start) + first + my_token) * a.b.max_pages + c0 + col;
        for (int r = 0; r < rounds && ok; ++r) {
            if (rounds > 1) {
                keyed = keyed_columns(r);
                ok = warp_wait(dfull, static_cast<uint32_t>((rounds + r) & 1), abort_flag);
                ok = !bar_sync_or(1, 32 * kSoftWarps, !ok);
                if (!ok) break;
                tc_after();
            }
            const int steps = (min(kCols, cols - r * kCols) + kStep - 1) / kStep;
#pragma unroll 1
            for (int j = half; j < steps; j += 2) {
                if (rounds == 1) {
                    uint32_t v[kStep];
                    tmem_ld16(lanes + kStep * j, v);
                    const float g = ex2_approx(off_s[j * kRows + row] - off) * f;      // (0 where nothing was seen so far)
#pragma unroll
                    for (int c = 0; c < kStep; ++c)
                        put_shared((put ^ ((c & 7) << 4)) + 128 * c, lives ? __uint_as_float(v[c]) * g : 0.0f);
                } else {
                    float x[kStep];
                    load(r, j, x);
#pragma unroll
                    for (int c = 0; c < kStep; ++c)
                        put_shared((put ^ ((c & 7) << 4)) + 128 * c, lives ? ex2_approx(x[c] - off) * f : 0.0f);
                }
                __syncwarp();
                const int at = r * kCols + kStep * j;          // column at + col of this CTA's
                const bool has = ((keyed_step(j) >> col) & 1u) != 0u;
                auto sum16 = [&](int r) {                      // rows r .. r + 15
                    const uint32_t from = get ^ (r << 2);
                    const float4 v0 = get_shared4(from), v1 = get_shared4(from ^ 16), v2 = get_shared4(from ^ 32), v3 = get_shared4(from ^ 48);
                    return (((v0.x + v0.y) + (v0.z + v0.w)) + ((v1.x + v1.y) + (v1.z + v1.w))) +
                           (((v2.x + v2.y) + (v2.z + v2.w)) + ((v3.x + v3.y) + (v3.z + v3.w)));
                };
                if (kHeads == kSixteen) {
                    const float sum = sum16(16 * part);
                    if (at < my_end) my_scores[at] = has ? sum : -INFINITY;
                } else if (kHeads == kFew) {
                    for (int k = part; k < per_warp; k += 2) {
                        const int tok = quarter * per_warp + k;
                        if (tok >= n_tokens) break;
                        float sum = 0.0f;
                        for (int h = k * H; h < (k + 1) * H; ++h) sum += get_shared((get ^ ((h >> 2) << 4)) + 4 * (h & 3));
                        const int c = c0 + at + col;
                        if (c < min(seen_s[tok], c0 + cols))
                            a.scores[(static_cast<int64_t>(q.start) + first + tok) * a.b.max_pages + c] = has ? sum : -INFINITY;
                    }
                } else {
                    // a warp's part of one token's heads; lanes past the last head hold 0
                    float sum = sum16(16 * part);
                    sum += __shfl_xor_sync(0xffffffffu, sum, kStep);
                    if (heads_warps > 1) {
                        if (part == 0) join[kCols * quarter + kStep * j + col] = sum;
                    } else if (part == 0 && at < my_end) {
                        my_scores[at] = has ? sum : -INFINITY;
                    }
                }
                __syncwarp();
            }
            if (kHeads == kMany && heads_warps > 1) {      // thread = column
                bar_sync_or(1, 32 * kSoftWarps, false);
                const int at = r * kCols + 32 * warp + lane;
                const bool has = ((__shfl_sync(0xffffffffu, keyed, warp) >> lane) & 1u) != 0u;
                for (int k = 0; k < 4 / heads_warps && k < n_tokens; ++k) {
                    float sum = 0.0f;
                    for (int w = k * heads_warps; w < (k + 1) * heads_warps; ++w) sum += join[kCols * w + 32 * warp + lane];
                    if (c0 + at < min(seen_s[k], c0 + cols))
                        a.scores[(static_cast<int64_t>(q.start) + first + k) * a.b.max_pages + c0 + at] = has ? sum : -INFINITY;
                }
            }
            if (rounds > 1) {
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dfree);
            }
        }
    }
    tc_before();
    __syncthreads();
    if (*abort_flag != 0 && threadIdx.x == 0) atomicOr(a.b.err, MLA_ERR_PIPELINE_TIMEOUT);
    tc_after();
    give_back();
    if (a.cluster > 1) cluster_sync();                     // (the others have read this CTA's maxima)
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// TMA's maps are made by the driver, whose entry point is looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::once_flag once;
    static EncodeTiled fn = nullptr;
    std::call_once(once, []() {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}

// BF16 [rows, dims], copied 64 dims x 32 rows at a time.
bool make_map(CUtensorMap* map, const void* data, int64_t rows, int dims) {
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t size[2] = {static_cast<cuuint64_t>(dims), static_cast<cuuint64_t>(rows)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(dims) * 2};
    const cuuint32_t box[2] = {64, 32}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(data), size, stride, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" int mla_block_scores(const void* q_bf16, int T, int H, int d_qk, const void* keys_bf16, int num_keys,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int n_seq,
                                int max_pages, int page_size, float sm_scale, float* scores, void* stream) {
    Batch b = {q_start, kv_len, block_table, n_seq, max_pages, page_size, T, nullptr};
    if (num_keys < 0 || !std::isfinite(sm_scale)) return MLA_EINVAL;
    if ((d_qk != kLatent && d_qk != kLatent + kRope) || H < 1 || H > 128) return MLA_EUNSUPPORTED;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0 || max_pages == 0) return rc;
    if (static_cast<int64_t>(T) * H > INT_MAX / 4) return MLA_EUNSUPPORTED;
    if (q_bf16 == nullptr || scores == nullptr || (keys_bf16 == nullptr && num_keys > 0) || off(q_bf16, 16) ||
        off(keys_bf16, 16) || off(scores, 4))
        return MLA_EINVAL;
    void (*const kernel)(const CUtensorMap, const ScoreArgs) =
        H == 16 ? block_scores_kernel<kSixteen> : H < 32 ? block_scores_kernel<kFew> : block_scores_kernel<kMany>;
    b.err = mla_host::device_error_word();
    const int sms = mla_host::sm_count();
    if (b.err == nullptr || sms <= 0 || !mla_host::max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmem))
        return MLA_ECUDA;
    ScoreArgs a = {b, static_cast<const __nv_bfloat16*>(keys_bf16), scores, H, d_qk, num_keys, 1, kCols, 1, sm_scale * kLog2e};
    a.tile_tokens = H <= 32 ? 4 * (32 / H) : H <= 64 ? 2 : 1;
    // (a tile has a token at least, and only a sequence's last one has fewer than tile_tokens)
    const int64_t tiles = std::min<int64_t>(T, static_cast<int64_t>(T) / a.tile_tokens + n_seq);
    // CTAs per tile: as many as hold three quarters of the table's blocks at once (tables are seldom full), and where
    // that leaves SMs without work, as many as have kLeast columns each.
    constexpr int kLeast = 64;
    while (a.cluster < kMaxCluster && a.cluster * kCols < max_pages - max_pages / 4) a.cluster *= 2;
    while (a.cluster < kMaxCluster && tiles * a.cluster < sms && a.cluster * kLeast < max_pages) a.cluster *= 2;
    if (tiles * a.cluster < 2 * sms) a.least = kLeast;
    if (tiles * a.cluster > INT_MAX) a.cluster = 1;
    alignas(64) CUtensorMap q_map;
    if (!make_map(&q_map, q_bf16, static_cast<int64_t>(T) * H, d_qk)) return MLA_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, q_map, a) == cudaSuccess && cudaGetLastError() == cudaSuccess ? MLA_OK
                                                                                                              : MLA_ECUDA;
}
