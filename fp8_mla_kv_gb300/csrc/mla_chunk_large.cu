// mla_chunk_attention, the kernel for many query rows: tiles of 64 (token, head) rows on
// tcgen05, where the tensor cores are what costs.
//
// Everything is turned: positions are the rows of the MMAs (M = 128 of them a block) and
// query rows the columns (N = 64), so that O^T of 512 dims x 64 rows fills half of the
// tensor memory and one CTA holds a whole tile, and so that what belongs to a position
// (its four tile scales, whether it is present) is one thread's, a register instead of
// a value broadcast from shared memory for every score: folding the partials of an
// untransposed S that way took 1,536 of the SM's shared-memory cycles per 64 positions.
//
// Per block of 128 positions:
//   QK   five products (the latent tiles, K = 128, and RoPE, 64): A = the positions' bytes as
//        the cache holds them, E4M3 (RoPE: BF16), put into tensor memory by the converting
//        warps without a look at them, B = q in shared memory. An E4M3 A wants an 8-bit B, so
//        q is two of them: an E4M3 part and the rest as E5M2, each row brought to [2^7, 2^8)
//        by a power of two first. A value of at least 2^-6 there is the sum of its parts exactly
//        (8 bits of BF16, 4 in the first part, and the rest is at most 8 units of the last bit:
//        E5M2 has all of those); a smaller one is off by at most 2^-14, 2^-21 of the row's largest.
//        Each tile's partial goes to an S slot of its own; the softmax warps fold them with the fp32
//        tile scales as they come. (A K rounded to f16 with its scale in it needs one
//        accumulator but moves a score near 20 by 3.5e-3. f16 codes and f16 q, exact too, need
//        the conversion before QK: it then waits for the tile's last PV, and took 3,817 us instead of
//        3,390 on the chunk below.)
//   P    thread = position x 32 query rows. The exp2 offset of a row is an earlier maximum:
//        it moves only when a score is more than kRescaleSlack above it, which one
//        vote per block shows; only then maxima over the positions are taken.
//   PV   O^T_t += V_t^T P^T: V = code x scale / sigma as f16 in shared memory (sigma_t: a
//        scale near the largest of tile t so far), read MN-major; P as f16, MN-major
//        too. Roundings: P, scale / sigma and their product, half a step of 2^-11 each.
// The order of the dims within QK is the one in which a thread that loaded 16 bytes of a
// row can store them to tensor memory; q is laid out to match.
//
// Roles: warps 0-7 softmax (lane quarter w % 4, query rows 32 (w / 4) ..), 8-15 turn cache
// rows into operands (straight from global memory, a block's rows in registers until PV has
// left their place; each warp 16 positions), 16 issues QK, 17 and 18 walk the block table ahead
// of them (slots, scales, sigma, prefetches into L2), 19 issues PV.
//
// 4,096 new tokens of 16 heads behind 12,288 positions: 2,960 us, 690 TFLOP/s, 0.36 of the
// measured dense bf16 rate. What bounds it: L1 and shared memory are busy 72 % of the time (V is written
// there once and read by PV, q and P by the MMAs, the rows come through it), the issue slots
// 53 %, the tensor pipe 31 %; and a block is a chain of about a dozen hand-offs between the roles,
// 120 cycles each, which keeps these from overlapping further. 24 sequences of two tokens of 128 heads
// and up to 16,384 positions: 247 us, of which starting and ending a piece take about 12 us each of three.
#include <cfloat>
#include <climits>
#include <cmath>

#include "mla_chunk.cuh"

namespace {

using namespace mla;
using namespace mla_chunk;

constexpr int kN = kLargeBlock;              // positions per block (M of the MMAs)
constexpr int kRows = kLargeRows;            // query rows per tile (N of the MMAs)
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kMetaWarp = kMmaWarp + 1, kMetaWarps = 2;
constexpr int kPvWarp = kMetaWarp + kMetaWarps;
constexpr int kThreads = 20 * 32;            // five warpgroups
// Registers per thread: launched as kLaunchRegs each and dealt out again.
constexpr int kLaunchRegs = 96;
constexpr int kSoftRegs = 104;
template <bool kRopeOn> constexpr int kConvRegs = kRopeOn ? 112 : 104;   // (104 with RoPE: 2,969 instead of 2,939 us)
template <bool kRopeOn> constexpr int kAuxRegs = kRopeOn ? 48 : 64;      // (48 without: 84 instead of 79 us, spills)
static_assert(2 * kSoftRegs + 2 * kConvRegs<true> + kAuxRegs<true> <= 5 * kLaunchRegs &&
              2 * kSoftRegs + 2 * kConvRegs<false> + kAuxRegs<false> <= 5 * kLaunchRegs, "registers");
constexpr int kCols = kRows / 2;             // query rows per softmax warp
constexpr int kMeta = 2;                     // blocks the meta warp may be ahead
// The exp2 offset puts the largest score at kTop (log2 units) and moves when one is kRescaleSlack above
// that: p <= 2^15, and f16's smallest p is 2^-28 of the largest (a million positions below half of that are
// together less than the rounding of the output). A move costs most of a block: 24 sequences of
// two tokens at 128 heads take 297, 279 and 273 us with kTop 7, 4 and 0.
constexpr float kTop = 4.0f, kRescaleSlack = 11.0f;
constexpr float kSigmaSlack = 64.0f;         // scale / sigma <= 2^6: code x scale / sigma < 2^15 in f16
constexpr float kLn2 = 0.6931471805599453f;

// Shared memory (the base is 1024-byte aligned). Operand tiles are rows of 64 16-bit
// values (128 B) in 8-row groups of 1 KB, 16-byte unit u of row r at unit u ^ (r & 7);
// wider tiles are sequences of such 64-column chunks.
constexpr int kQChunk = kRows * 128;                       // 8 KB
constexpr int kOffQ = 0;                                   // a chunk per latent tile and part of q, and RoPE
constexpr int kVChunk = kN * 128;                          // 16 KB
constexpr int kOffV = kOffQ + 9 * kQChunk;                 // 4 tiles of 128 positions x 128 dims
constexpr int kOffP = kOffV + 8 * kVChunk;                 // 128 positions x 64 query rows
constexpr int kOffMeta = kOffP + kN * 128;
struct __align__(16) Meta {
    float sc[4][kN];                         // tile scales; 0 where absent
    uint16_t rs[4][kN];                      // scale / sigma, f16
    int32_t slot[kN];                        // -1 where absent (a cache that fits a GPU has less than 2^31 rows)
    float f[4];                              // what O^T of each tile has to be multiplied by (sigma moved)
    float sigma[4];
    uint8_t state[kN];                       // 0 absent, 1 present, 2 a scale that is not finite
};
constexpr int kOffRow = kOffMeta + kMeta * static_cast<int>(sizeof(Meta));
struct __align__(16) RowData {               // per query row
    float neg_m[kRows];                      // exp2 offset (log2 units), negated
    float alpha[kRows];                      // what O^T and l are multiplied by when it moves; at the end 1 / l
    float shift[kRows];                      // undoes q's power of two
    int lim[kRows];                          // positions it attends, counted from the piece's first
    int unseen[kRows];                       // attends something, but nothing so far
    float wmax[4][kRows];                    // by lane quarter: maxima; at the end sums of p
    float smax[kMetaWarps][4];               // largest scales, where a sigma moves
    int any_unseen[2], pad[2];
};
constexpr int kOffBars = kOffRow + static_cast<int>(sizeof(RowData));
constexpr int kNumBars = 32;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kSmemTotal = kOffMisc + 16;
static_assert(kSmemTotal <= 232448, "shared memory");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColA = 4 * kRows, kColS = kColA + 128; // O^T tiles, four A slots of 32, two S slots of 64
constexpr int kASlots = 4;

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16 instruction descriptor: fp32 D, A and B format (0 f16, 1 bf16), majors, M, N.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t fmt, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// kind::f8f6f4: the same fields; formats 0 E4M3, 1 E5M2.
constexpr uint32_t kIdQK = idesc_f16(0, false, false, kN, kRows);     // S^T = K_t . (the E4M3 part of q_t)^T
constexpr uint32_t kIdQK2 = kIdQK | (1u << 10);                       // + K_t . (its E5M2 part)^T
constexpr uint32_t kIdQR = idesc_f16(1, false, false, kN, kRows);     // RoPE (bf16)
constexpr uint32_t kIdPV = idesc_f16(0, true, true, kTile, kRows);    // O^T_t += V_t^T . P^T

__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)) : "memory");
}
__device__ __forceinline__ void umma_ts8(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)) : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Waits for this warp's tcgen05.ld; the registers pass through, so that no use of them
// is scheduled before it.
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 bits, 32 columns: thread t gets lane t, columns c .. c + 31.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
           "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
           "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t* r, uint32_t* q) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]), "+r"(q[4]), "+r"(q[5]), "+r"(q[6]), "+r"(q[7]),
                   "+r"(q[8]), "+r"(q[9]), "+r"(q[10]), "+r"(q[11]), "+r"(q[12]), "+r"(q[13]), "+r"(q[14]), "+r"(q[15])
                 :: "memory");
}
// 16 lanes x 256 bits, 4 times (32 columns): thread t gives lanes t / 4 and t / 4 + 8, columns
// 8j + 2 (t % 4) + {0, 1} from r[4j], r[4j+1] (lane t / 4) and r[4j+2], r[4j+3].
__device__ __forceinline__ void tmem_st_16x256_x4(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int kRegs>
__device__ __forceinline__ void deal_registers() {
    if (kRegs > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegs));
    if (kRegs < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegs));
}

// Byte offset of 16-byte unit u of row r in a swizzled tile of `rows` rows.
__device__ __forceinline__ uint32_t swz(int rows, int r, int u) {
    return static_cast<uint32_t>((u >> 3) * rows * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// A bounded wait that also ends as soon as another role has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    // (the clock's upper bits are enough, in a register)
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    const int t0 = static_cast<int>(clock64() >> 16);
#pragma unroll 1
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (static_cast<int>(clock64() >> 16) - t0 > static_cast<int>(kWaitCycles >> 16)) {
            *abort_flag = 1;
            return false;
        }
    }
}
// The same by a whole warp, with one answer for it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

// Whether a cache row holds a value that is not finite: a NaN code, or a RoPE value that is
// NaN or infinite (the scales have been looked at). One is added to the field of all the
// exponent (and, of a code, mantissa) bits: a carry into the bit above.
template <bool kRopeOn>
__device__ __noinline__ bool row_is_odd(const uint8_t* row) {
    uint32_t odd = 0u;
#pragma unroll 4
    for (int i = 0; i < kLatent / 4; ++i) odd |= ((__ldg(reinterpret_cast<const uint32_t*>(row) + i) & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    if (kRopeOn)
#pragma unroll 4
        for (int i = 0; i < kRope / 2; ++i)
            odd |= ((__ldg(reinterpret_cast<const uint32_t*>(row + kTailOff) + i) & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    return odd != 0u;
}

// Those of the tiles (bits 0 .. 3) of a cache row whose codes are all zeros.
__device__ __forceinline__ uint32_t zero_tiles(const uint8_t* row, uint32_t tiles) {
#pragma unroll 1
    for (int i = 0; i < kLatent / 16; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(row) + i);
        if (((w.x | w.y | w.z | w.w) & 0x7f7f7f7fu) != 0u) tiles &= ~(1u << (i >> 3));
    }
    return tiles;
}

// A row's 16 bytes, zeros where the row is absent (slot < 0): a predicate, not a branch.
__device__ __forceinline__ uint4 ld_row(const uint8_t* cache, int slot, uint32_t row_bytes, uint32_t off) {
    const uint8_t* p = cache + static_cast<uint64_t>(static_cast<uint32_t>(slot)) * row_bytes + off;
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ge.s32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w) : "l"(p), "r"(slot));
    return r;
}

__device__ __forceinline__ uint32_t word4(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void clear4(uint4& v, int i) { (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = 0u; }

// One thread of the warp; ptxas knows that it is one, so the MMAs' operands need no loop
// over the active threads.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

template <bool kRopeOn>
__global__ void __launch_bounds__(kThreads, 1)
mla_chunk_large_kernel(const ChunkArgs args) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Meta* meta = reinterpret_cast<Meta*>(smem + kOffMeta);
    RowData& rd = *reinterpret_cast<RowData*>(smem + kOffRow);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
    uint64_t* afull = bars;            // [4] A slot written (8 converting warps)
    uint64_t* afree = bars + 4;        // [4] its QK is done (commit)
    uint64_t* sfull = bars + 8;        // [2] S slot written (commit)
    uint64_t* sfree = bars + 10;       // [2] S slot read (8 softmax warps)
    uint64_t* vfull = bars + 12;       // [4] V tile written (8 converting warps)
    uint64_t* vfree = bars + 16;       // [4] its PV is done (commit)
    uint64_t* pfull = bars + 20;       // P written, O^T corrected (8 softmax warps)
    uint64_t* pvdone = bars + 21;      // PV of a block done (commit)
    uint64_t* mfull = bars + 22;       // [2] meta stage written (2 meta warps)
    uint64_t* mfree = bars + 24;       // [2] meta stage read (8 softmax, 8 converting warps)
    uint64_t* fin = bars + 27;         // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const Piece pc = find_piece(args, static_cast<int>(blockIdx.x), lane);
    if (pc.seq < 0) return;
    if ((smem_u32(smem) & 1023u) != 0u) {      // the operand layout's phase would be off: no result
        if (threadIdx.x == 0) atomicOr(args.err, MLA_ERR_PIPELINE_TIMEOUT);
        return;
    }
    const int n_keys = pc.k1 - pc.k0;
    const int nblk = (n_keys + kN - 1) / kN;
    const int n_rows = min(kRows, pc.rows - pc.row0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kASlots; ++i) {
            mbar_init(&afull[i], kConvWarps);
            mbar_init(&afree[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], kSoftWarps);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&vfull[i], kConvWarps);
            mbar_init(&vfree[i], 1);
        }
        mbar_init(pfull, kSoftWarps);
        mbar_init(pvdone, 1);
        for (int i = 0; i < kMeta; ++i) {
            mbar_init(&mfull[i], kMetaWarps);
            mbar_init(&mfree[i], kSoftWarps + kConvWarps);
        }
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x < kRows) {
        const int r = threadIdx.x, lim = r < n_rows ? row_limit(args, pc, pc.row0 + r) - pc.k0 : 0;
        rd.lim[r] = lim;
        rd.unseen[r] = lim > 0;
        rd.neg_m[r] = 0.0f;
    }
    // ---- q of the tile's rows as operand tiles: a warp per row, lane l the 16-byte units
    // l and l + 32 of the latent and, l < 8, unit l of RoPE; the next row's on their way ----
    uint4 ahead[3];
    auto load_q = [&](int r) {
        ahead[0] = ahead[1] = ahead[2] = make_uint4(0u, 0u, 0u, 0u);
        if (r < n_rows) {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(args.q + (pc.grow0 + pc.row0 + r) * args.d_qk);
            ahead[0] = ld_nc_v4(src + 16 * lane);
            ahead[1] = ld_nc_v4(src + 512 + 16 * lane);
            if (kRopeOn && lane < 8) ahead[2] = ld_nc_v4(src + 1024 + 16 * lane);
        }
    };
    load_q(warp);
#pragma unroll 1
    for (int r = warp; r < kRows; r += kThreads / 32) {
        const uint4 v[3] = {ahead[0], ahead[1], ahead[2]};
        load_q(r + kThreads / 32);
        // The row's largest value (as bits: |bf16| are ordered like integers) and the power of two that
        // brings it into [2^7, 2^8); undone on the scores.
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
        }
        const int mx = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int k = mx >= 0x7f80 ? 0 : max((mx >> 7) - 134, -126);
        const __nv_bfloat162 down = __float2bfloat162_rn(__int_as_float((127 - k) << 23));
        if (lane == 0) rd.shift[r] = __int_as_float((127 + k) << 23);
        // Each value as an E4M3 part and the rest as an E5M2 one. Operand place of the dims: 4-byte word
        // m of the 32 bytes that a converting thread holds of a row (16 c .. of each half) goes to tensor-memory
        // column 8 (m / 2) + 2 c + m % 2, so the 8 dims of a unit stay together.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 x = __float22half2_rn(__bfloat1622float2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), down)));
                hi[j] = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
                const __half2 y(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi[j]), __NV_E4M3));
                lo[j] = __nv_cvt_halfraw2_to_fp8x2(__hsub2(x, y), __NV_SATFINITE, __NV_E5M2);
            }
            const int u = lane + 32 * i, ut = u & 15;
            const int at = 4 * (16 * (ut >> 3) + 8 * (ut & 1) + 2 * ((ut >> 1) & 3));      // bytes
            uint8_t* q = smem + kOffQ + 2 * (u >> 4) * kQChunk + swz(kRows, r, at >> 4) + (at & 8);
            *reinterpret_cast<uint2*>(q) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(q + kQChunk) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        if (kRopeOn && lane < 8) {
            const uint32_t w[4] = {v[2].x, v[2].y, v[2].z, v[2].w};
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), down);
                h[j] = *reinterpret_cast<const uint32_t*>(&x);
            }
            const int at = 16 * (2 * (lane >> 2)) + 4 * (lane & 3);
            uint8_t* q = smem + kOffQ + 8 * kQChunk;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pos = at + 16 * j;
                *reinterpret_cast<uint2*>(q + swz(kRows, r, pos >> 3) + ((pos & 4) << 1)) = make_uint2(h[2 * j], h[2 * j + 1]);
            }
        }
    }
    fence_proxy_async_smem();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int kGroups = kRopeOn ? 5 : 4;          // S partials per block: [RoPE,] tiles 0 .. 3

    if (warp < kSoftWarps) {
        deal_registers<kSoftRegs>();
        // ---- softmax: thread = position 32 quarter + lane, query rows c0 .. c0 + 31 ----
        const int quarter = warp & 3, half = warp >> 2;
        const int key = 32 * quarter + lane;
        const int c0 = kCols * half;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        // what is uniform over this half's query rows
        const int my_lim = rd.lim[c0 + lane];
        const int lim_min = __reduce_min_sync(0xffffffffu, my_lim);
        bool unseen = true;                            // some row has seen nothing yet: take maxima
        float l = 0.0f;                                // sum of p of query row c0 + lane, over the warp's positions
        float sig[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        bool ok = true;
        int g = 0;
        for (int b = 0; b < nblk && ok; ++b) {
            const Meta& mt = meta[b % kMeta];
            // A wait that ran out only skips work up to the vote, which all four warps take.
            ok = warp_wait(&mfull[b % kMeta], static_cast<uint32_t>((b / kMeta) & 1), abort_flag);
            int state = mt.state[key];
            uint64_t s[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) s[j] = 0ull;
            // (loops over the groups and tiles are not unrolled anywhere: the roles' code, taken
            // together, has to stay in the instruction cache)
#pragma unroll 1
            for (int t = 4 - kGroups; t < 4; ++t, ++g) {
                const int slot = g & 1;
                ok = ok && warp_wait(&sfull[slot], static_cast<uint32_t>((g >> 1) & 1), abort_flag);
                if (!ok) break;
                tc_after();
                uint32_t v[16], w[16];
                tmem_ld16(lane_base + kColS + kRows * slot + c0, v);
                tmem_ld16(lane_base + kColS + kRows * slot + c0 + 16, w);
                const uint32_t f = __float_as_uint(t < 0 ? args.sm_scale_log2 : mt.sc[t][key] * args.sm_scale_log2);
                const uint64_t ff = two(f, f);
                tc_wait_ld16(v, w);
                tc_before();
                warp_arrive(&sfree[slot]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j] = fma2(two(v[2 * j], v[2 * j + 1]), ff, s[j]);
                    s[j + 8] = fma2(two(w[2 * j], w[2 * j + 1]), ff, s[j + 8]);
                }
            }
            // A value of the position's row that is not finite shows in its score with any finite query
            // row (0 * it is not 0), so with the first. (Looked into after the vote.)
            const bool odd = !(fabsf(lo_of(s[0])) <= FLT_MAX);
            float d[kCols];
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&rd.shift[c0 + c]);
                const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&rd.neg_m[c0 + c]);
                s[c / 2] = fma2(s[c / 2], x.x, m.x);
                s[c / 2 + 1] = fma2(s[c / 2 + 1], x.y, m.y);
                d[c] = lo_of(s[c / 2]);
                d[c + 1] = hi_of(s[c / 2]);
                d[c + 2] = lo_of(s[c / 2 + 1]);
                d[c + 3] = hi_of(s[c / 2 + 1]);
            }
            if (__builtin_expect(__any_sync(0xffffffffu, state != 1) || kN * (b + 1) > lim_min, 0)) {
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    if (state == 2) d[c] = __int_as_float(0x7FC00000);
                    if (state == 0 || kN * b + key >= rd.lim[c0 + c]) d[c] = -INFINITY;
                }
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kCols; c += 4)
                tops[(c >> 2) & 3] = fmaxf(fmaxf(tops[(c >> 2) & 3], fmaxf(d[c], d[c + 1])), fmaxf(d[c + 2], d[c + 3]));
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            // P of the block before has been read, and O^T is complete up to it.
            if (b > 0) {
                ok = ok && warp_wait(pvdone, static_cast<uint32_t>((b - 1) & 1), abort_flag);
                tc_after();
            }
            const bool moved = bar_sync_or(1 + half, 128, unseen || top > kTop + kRescaleSlack || odd || !ok);
            const float f0 = mt.f[0], f1 = mt.f[1], f2 = mt.f[2], f3 = mt.f[3];
            const bool sigma_moved = b > 0 && (f0 != 1.0f || f1 != 1.0f || f2 != 1.0f || f3 != 1.0f);
            if (__builtin_expect(moved, 0)) {
                // Rare after the first block: maxima over the positions, new offsets for the rows
                // whose scores ran ahead, l and O^T rescaled.
                if (bar_sync_or(1 + half, 128, !ok)) {
                    ok = false;
                    break;
                }
                if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
                    // A query row that attends such a row gets NaN; one for which it is masked must not
                    // meet 0 * NaN in PV, so its V becomes 0.
                    const int slot = mt.slot[key];
                    if (slot >= 0 && odd && row_is_odd<kRopeOn>(args.cache + slot * args.row_bytes)) {
                        state = 2;
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if (kN * b + key < rd.lim[c0 + c]) d[c] = __int_as_float(0x7FC00000);
                    }
#pragma unroll 1
                    for (int t = 0; t < 4; ++t) {
                        ok = ok && warp_wait(&vfull[t], static_cast<uint32_t>(b & 1), abort_flag);
                        if (state == 2)
#pragma unroll 1
                            for (int u = 0; u < 16; ++u)
                                *reinterpret_cast<uint4*>(smem + kOffV + 2 * t * kVChunk + swz(kN, key, u)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                // Maxima over the warp's positions, as the sums below: lane x ends with row x.
                float v[kCols / 2];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const bool up = (lane & 16) != 0;
                    const float keep = up ? d[c + 16] : d[c], give = up ? d[c] : d[c + 16];
                    v[c] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 16));
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) {
                    const bool up = (lane & x) != 0;
#pragma unroll
                    for (int c = 0; c < x; ++c) {
                        const float keep = up ? v[c + x] : v[c], give = up ? v[c] : v[c + x];
                        v[c] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, x));
                    }
                }
                rd.wmax[quarter][c0 + lane] = v[0];
                if (bar_sync_or(1 + half, 128, !ok)) {
                    ok = false;
                    break;
                }
                if (quarter == 0) {
                    const int c = c0 + lane;
                    const float up = fmaxf(fmaxf(rd.wmax[0][c], rd.wmax[1][c]), fmaxf(rd.wmax[2][c], rd.wmax[3][c])) - kTop;
                    const bool first = rd.unseen[c] != 0 && up > -INFINITY;
                    const bool move = first || up > kRescaleSlack;
                    rd.alpha[c] = move ? (first ? 0.0f : ex2_approx(-up)) : 1.0f;
                    if (first) rd.unseen[c] = 0;
                    rd.wmax[0][c] = move ? up : 0.0f;      // by how much the offset moves
                    if (move) rd.neg_m[c] -= up;
                    const bool left = __any_sync(0xffffffffu, rd.unseen[c] != 0);
                    if (lane == 0) rd.any_unseen[half] = left;
                }
                bar_sync_or(1 + half, 128, false);
                unseen = rd.any_unseen[half] != 0;
#pragma unroll
                for (int c = 0; c < kCols; c += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(&rd.wmax[0][c0 + c]);
                    d[c] -= m.x;
                    d[c + 1] -= m.y;
                    d[c + 2] -= m.z;
                    d[c + 3] -= m.w;
                }
                l *= rd.alpha[c0 + lane];
            }
            if (__builtin_expect(b > 0 && (moved || sigma_moved), 0)) {
#pragma unroll 1
                for (int t = 0; t < 4; ++t) {
                    uint32_t o[kCols];
                    tmem_ld32(lane_base + kRows * t + c0, o);
                    tc_wait_ld(o);
                    const float f = t == 0 ? f0 : t == 1 ? f1 : t == 2 ? f2 : f3;
                    if (f != 1.0f) {
#pragma unroll
                        for (int c = 0; c < kCols; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                    }
                    if (moved) {
#pragma unroll
                        for (int c = 0; c < kCols; c += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(&rd.alpha[c0 + c]);
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * a.x);
                            o[c + 1] = __float_as_uint(__uint_as_float(o[c + 1]) * a.y);
                            o[c + 2] = __float_as_uint(__uint_as_float(o[c + 2]) * a.z);
                            o[c + 3] = __float_as_uint(__uint_as_float(o[c + 3]) * a.w);
                        }
                    }
                    tmem_st32(lane_base + kRows * t + c0, o);
                }
                tc_wait_st();
            }
            uint8_t* prow = smem + kOffP + key * 128;
#pragma unroll
            for (int u = 0; u < kCols / 8; ++u) {
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 8; ++k) d[8 * u + k] = ex2_approx(d[8 * u + k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(d[8 * u + 2 * k], d[8 * u + 2 * k + 1]);
                *reinterpret_cast<uint4*>(prow + (((4 * half + u) ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) sig[t] = mt.sigma[t];
            fence_proxy_async_smem();
            tc_before();
            warp_arrive(pfull);
            warp_arrive(&mfree[b % kMeta]);
            // The sums of P over the warp's positions, while PV runs: at each step half of the rows go
            // to the lane across, so lane x ends with row x.
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) {
                const bool up = (lane & x) != 0;
#pragma unroll
                for (int c = 0; c < x; ++c) {
                    const float keep = up ? d[c + x] : d[c], give = up ? d[c] : d[c + x];
                    d[c] = keep + __shfl_xor_sync(0xffffffffu, give, x);
                }
            }
            l += d[0];
        }
        // ---- epilogue: l over the positions, then O^T * sigma / l ----
        if (ok && nblk > 0) {
            ok = warp_wait(pvdone, static_cast<uint32_t>((nblk - 1) & 1), abort_flag);
            tc_after();
        }
        if (!bar_sync_or(1 + half, 128, !ok)) {
            rd.wmax[quarter][c0 + lane] = l;
            bar_sync_or(1 + half, 128, false);
            if (quarter == 0) {
                const int c = c0 + lane;
                const float sum = (rd.wmax[0][c] + rd.wmax[1][c]) + (rd.wmax[2][c] + rd.wmax[3][c]);
                // 0: nothing attended; NaN: an attended row holds a value that is not finite
                const float kNaN = __int_as_float(0x7FC00000);
                rd.alpha[c] = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : kNaN);
                const float lse = sum > 0.0f ? (log2f(sum) - rd.neg_m[c]) * kLn2 : (sum == 0.0f ? -INFINITY : kNaN);
                if (c < n_rows) {
                    if (pc.part < 0) args.lse[pc.grow0 + pc.row0 + c] = lse;
                    else args.part_lse[static_cast<int64_t>(pc.part) * kRows + c] = lse;
                }
            }
            bar_sync_or(1 + half, 128, false);
            const int left = n_rows - c0;              // query rows of this half that there are
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
                uint32_t o[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) o[c] = 0u;
                if (nblk > 0) {
                    tmem_ld32(lane_base + kRows * t + c0, o);
                    tc_wait_ld(o);
                }
                const float f = t == 0 ? sig[0] : t == 1 ? sig[1] : t == 2 ? sig[2] : sig[3];
                const int dim = kTile * t + key;           // here the lane is a dim
                if (pc.part < 0) {
                    __nv_bfloat16* to = args.out + (pc.grow0 + pc.row0 + c0) * kLatent + dim;
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c < left) to[c * kLatent] = __float2bfloat16_rn(__uint_as_float(o[c]) * (f * rd.alpha[c0 + c]));
                } else {
                    float* to = args.part_o + (static_cast<int64_t>(pc.part) * kRows + c0) * kLatent + dim;
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c < left) to[c * kLatent] = __uint_as_float(o[c]) * (f * rd.alpha[c0 + c]);
                }
            }
            tc_before();
        }
    } else if (warp < kMmaWarp) {
        deal_registers<kConvRegs<kRopeOn>>();
        // ---- conversion: lane (rows r0 and r0 + 8, 16-byte pieces c of each 64) ----
        const int quarter = warp & 3, hh = (warp - kSoftWarps) >> 2;
        const int c = lane & 3;
        const int r0 = 32 * quarter + 16 * hh + (lane >> 2);
        const uint32_t a_base = tmem + (static_cast<uint32_t>(32 * quarter + 16 * hh) << 16) + kColA;
        const uint32_t row_bytes = static_cast<uint32_t>(args.row_bytes);
        int slot[2];
        uint4 v[4][2][2];                              // a block's codes; v[3] holds RoPE's values first
        bool ok = true;
        int g = 0;
        auto rows_of = [&](int b) {
            ok = ok && warp_wait(&mfull[b % kMeta], static_cast<uint32_t>((b / kMeta) & 1), abort_flag);
            if (!ok) return;
            slot[0] = meta[b % kMeta].slot[r0];
            slot[1] = meta[b % kMeta].slot[r0 + 8];
        };
        auto load = [&](uint4 (&x)[2][2], uint32_t off) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[e][0] = ld_row(args.cache, slot[e], row_bytes, off + 16 * c);
                x[e][1] = ld_row(args.cache, slot[e], row_bytes, off + 16 * c + 64);
            }
        };
        auto put = [&](const uint4 (&x)[2][2]) {       // the rows' bytes as they are: an A operand of QK
            const int as = g % kASlots;
            if (g >= kASlots) ok = ok && warp_wait(&afree[as], static_cast<uint32_t>((g / kASlots - 1) & 1), abort_flag);
            ++g;
            if (!ok) return;
            tc_after();
            uint32_t w[16];                            // word m of row e at 4 (m / 2) + 2 e + m % 2
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    w[8 * p + 2 * e] = x[e][p].x; w[8 * p + 2 * e + 1] = x[e][p].y;
                    w[8 * p + 4 + 2 * e] = x[e][p].z; w[8 * p + 5 + 2 * e] = x[e][p].w;
                }
            tmem_st_16x256_x4(a_base + 32 * as, w);
            tc_wait_st();
            tc_before();
            warp_arrive(&afull[as]);
        };
        if (nblk > 0) rows_of(0);
        if (nblk > 0 && ok) {
#pragma unroll
            for (int t = 0; t < 4; ++t) load(v[t], kRopeOn && t == 3 ? kTailOff : 128 * t);
        }
        for (int b = 0; b < nblk && ok; ++b) {
            const Meta& mt = meta[b % kMeta];
            const bool more = b + 1 < nblk;
            if (kRopeOn) {
                put(v[3]);
                load(v[3], 128 * 3);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) put(v[t]);
            if (more) rows_of(b + 1);
            // V: the product with scale / sigma, once PV of the block before has read the tile
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (b > 0) ok = ok && warp_wait(&vfree[t], static_cast<uint32_t>((b - 1) & 1), abort_flag);
                if (!ok) break;
                uint8_t* tile = smem + kOffV + 2 * t * kVChunk;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t f = mt.rs[t][r0 + 8 * e] * 0x10001u;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t x[4];
                            e4m3x4_to_f16x2x2(u == 0 ? v[t][e][p].x : v[t][e][p].z, x[0], x[1]);
                            e4m3x4_to_f16x2x2(u == 0 ? v[t][e][p].y : v[t][e][p].w, x[2], x[3]);
                            *reinterpret_cast<uint4*>(tile + swz(kN, r0 + 8 * e, 8 * p + 2 * c + u)) =
                                make_uint4(hmul2(x[0], f), hmul2(x[1], f), hmul2(x[2], f), hmul2(x[3], f));
                        }
                }
                if (more) load(v[t], kRopeOn && t == 3 ? kTailOff : 128 * t);
                fence_proxy_async_smem();
                warp_arrive(&vfull[t]);
            }
            if (!ok) break;
            warp_arrive(&mfree[b % kMeta]);
        }
    } else {
    deal_registers<kAuxRegs<kRopeOn>>();
    if (warp == kMmaWarp) {
        // ---- QK, one elected thread ----
        if (elect_one()) {
            const uint64_t dq = sw128_desc(smem_u32(smem) + kOffQ, 16, 1024);
            const int n_groups = nblk * kGroups;
            bool ok = true;
            int t = 4 - kGroups;                       // latent tile; -1: RoPE
#pragma unroll 1
            for (int g = 0; g < n_groups; ++g) {
                const int slot = g & 1, as = g % kASlots;
                ok = wait_or_abort(&afull[as], static_cast<uint32_t>((g / kASlots) & 1), abort_flag);
                if (g >= 2) ok = ok && wait_or_abort(&sfree[slot], static_cast<uint32_t>(((g >> 1) - 1) & 1), abort_flag);
                if (!ok) break;
                tc_after();
                const uint32_t d = tmem + kColS + kRows * slot, a = tmem + kColA + 32 * as;
                const uint64_t dt = dq + static_cast<uint64_t>(((t >= 0 ? 2 * t : 8) * kQChunk) >> 4);
                if (t < 0) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) umma_ts(d, a + 8 * ks, dt + static_cast<uint64_t>(2 * ks), kIdQR, ks > 0);
                } else {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ts8(d, a + 8 * (ks & 3), dt + static_cast<uint64_t>((ks >> 2) * (kQChunk >> 4) + 2 * (ks & 3)),
                                 ks < 4 ? kIdQK : kIdQK2, ks > 0);
                }
                umma_commit(&sfull[slot]);
                umma_commit(&afree[as]);
                if (++t == 4) t = 4 - kGroups;
            }
            // Every MMA issued has completed before tensor memory is freed.
            umma_commit(&fin[0]);
            (void)mbar_wait_bounded(&fin[0], 0);
        }
        __syncwarp();
    } else if (warp == kPvWarp) {
        // ---- PV, one elected thread ----
        if (elect_one()) {
            const uint32_t base = smem_u32(smem);
            const uint64_t dp = sw128_desc(base + kOffP, 16, 1024);
            bool ok = true;
#pragma unroll 1
            for (int b = 0; b < nblk && ok; ++b) {
                ok = wait_or_abort(pfull, static_cast<uint32_t>(b & 1), abort_flag);
#pragma unroll 1
                for (int t = 0; t < 4 && ok; ++t) {
                    ok = wait_or_abort(&vfull[t], static_cast<uint32_t>(b & 1), abort_flag);
                    if (!ok) break;
                    tc_after();
                    const uint64_t dv = sw128_desc(base + kOffV + 2 * t * kVChunk, kVChunk, 1024);
#pragma unroll
                    for (int ks = 0; ks < kN / 16; ++ks)
                        umma_ss(tmem + kRows * t, dv + static_cast<uint64_t>(ks * 128), dp + static_cast<uint64_t>(ks * 128), kIdPV,
                                b > 0 || ks > 0);
                    umma_commit(&vfree[t]);
                    if (t == 3) umma_commit(pvdone);
                }
            }
            umma_commit(&fin[1]);
            (void)mbar_wait_bounded(&fin[1], 0);
        }
        __syncwarp();
    } else if (warp < kMetaWarp + kMetaWarps) {
        // ---- meta: slots, scales and sigma, ahead of the others, each warp for half of a block's
        // positions: block b + 1's scales and block b + 2's table entries are on their way
        // before the stage of block b + 1 is waited for ----
        constexpr int kPer = kN / 32 / kMetaWarps;     // positions per lane
        const int mw = warp - kMetaWarp;
        const int32_t* bt = args.block_table + static_cast<int64_t>(pc.seq) * args.max_pages;
        const uint32_t row_bytes = static_cast<uint32_t>(args.row_bytes);
        float sigma[4] = {0.0f, 0.0f, 0.0f, 0.0f}, inv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int slot[kPer], slot1[kPer];                   // of blocks b and b + 1
        uint4 u[kPer];                                 // their scales
        auto look_up = [&](int b) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int j = kN * b + 32 * (kPer * mw + i) + lane;
                slot1[i] = j < n_keys ? static_cast<int>(chunk_slot(args, bt, pc.k0 + j)) : -1;
            }
        };
        auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                slot[i] = slot1[i];
                u[i] = ld_row(args.cache, slot[i], row_bytes, kScaleOff);
                if (slot[i] >= 0) {
                    const uint8_t* row = args.cache + static_cast<uint64_t>(static_cast<uint32_t>(slot[i])) * row_bytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k) prefetch_l2(row + 128 * k);
                    if (kRopeOn) prefetch_l2(row + kTailOff + 64);
                }
            }
        };
        // Block b's stage from its slots and scales; false when the call has failed.
        auto stage = [&](int b) {
            Meta& mt = meta[b % kMeta];
            int state[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool odd = !(isfinite(__uint_as_float(u[i].x)) && isfinite(__uint_as_float(u[i].y)) &&
                                   isfinite(__uint_as_float(u[i].z)) && isfinite(__uint_as_float(u[i].w)));
                state[i] = slot[i] < 0 ? 0 : odd ? 2 : 1;
                if (odd) u[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            bool ok = true;
            if (b >= kMeta) ok = warp_wait(&mfree[b % kMeta], static_cast<uint32_t>((b / kMeta - 1) & 1), abort_flag);
            // Whether a sigma moves (the first scale that is not 0, and later ones far above it): a
            // decision of both warps.
            bool far = false;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < kPer; ++i) far = far || fabsf(__uint_as_float(word4(u[i], t))) > sigma[t] * kSigmaSlack;
            const bool move = bar_sync_or(4, 32 * kMetaWarps, far || !ok);
            if (move) {
                if (bar_sync_or(4, 32 * kMetaWarps, !ok)) return false;
                // The writer gives a tile of zeros the scale 1, which beside small values would take the bits
                // of their scale / sigma for nothing: a tile of zeros counts with 0.
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    uint32_t ones = 0u;
#pragma unroll
                    for (int t = 0; t < 4; ++t) ones |= (word4(u[i], t) == 0x3f800000u ? 1u : 0u) << t;
                    if (__builtin_expect(ones != 0u, 0)) {
                        ones = zero_tiles(args.cache + static_cast<uint64_t>(static_cast<uint32_t>(slot[i])) * row_bytes, ones);
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (((ones >> t) & 1u) != 0u) clear4(u[i], t);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(__uint_as_float(word4(u[i], t))));
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    if (lane == 0) rd.smax[mw][t] = top;
                }
                bar_sync_or(4, 32 * kMetaWarps, false);
            }
            float f[4] = {1.0f, 1.0f, 1.0f, 1.0f};
            if (move) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float top = fmaxf(rd.smax[0][t], rd.smax[1][t]);
                    if (top > sigma[t] * kSigmaSlack) {
                        const float now = fmaxf(top, FLT_MIN);       // its reciprocal is finite
                        inv[t] = 1.0f / now;
                        f[t] = sigma[t] * inv[t];
                        sigma[t] = now;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int j = 32 * (kPer * mw + i) + lane;
                    const float sc = __uint_as_float(word4(u[i], t));
                    mt.sc[t][j] = sc;
                    mt.rs[t][j] = static_cast<uint16_t>(pack_f16x2(sc * inv[t], 0.0f));
                }
                if (mw == 0 && lane == 0) {
                    mt.f[t] = f[t];
                    mt.sigma[t] = sigma[t];
                }
            }
            if (move) bar_sync_or(4, 32 * kMetaWarps, false);      // the maxima have been read
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int j = 32 * (kPer * mw + i) + lane;
                mt.slot[j] = slot[i];
                mt.state[j] = static_cast<uint8_t>(state[i]);
            }
            warp_arrive(&mfull[b % kMeta]);
            return true;
        };
#pragma unroll 1
        for (int b = -2; b < nblk; ++b) {
            if (b >= 0 && !stage(b)) break;
            if (b >= -1 && b + 1 < nblk) fetch();
            if (b + 2 < nblk) look_up(b + 2);
        }
    }
    }
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) atomicOr(args.err, MLA_ERR_PIPELINE_TIMEOUT);
    if (warp == kMmaWarp) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

namespace mla_host {

bool launch_chunk_large(const mla_chunk::ChunkArgs& a, int64_t pieces, bool rope, void* stream) {
    const void* kernel = rope ? reinterpret_cast<const void*>(mla_chunk_large_kernel<true>)
                              : reinterpret_cast<const void*>(mla_chunk_large_kernel<false>);
    if (!max_dynamic_smem(kernel, kSmemTotal)) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pieces));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemTotal;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (rope ? cudaLaunchKernelEx(&cfg, mla_chunk_large_kernel<true>, a)
                 : cudaLaunchKernelEx(&cfg, mla_chunk_large_kernel<false>, a)) == cudaSuccess &&
           cudaGetLastError() == cudaSuccess;
}

}  // namespace mla_host
