// mla_chunk_attention: attention of a chunk of new tokens over the paged FP8 cache.
//
// Token i of a sequence's n new tokens, with L positions in the cache, attends the
// positions p <= L - n + i (all of them without `causal`):
//   s_p = sm_scale * (q . K_p), out = softmax(s) V, lse = ln sum exp s_p,
// K_p = the row's dequantised latent and its RoPE tail, V_p = the latent.
//
// The query rows of a sequence are its (token, head) pairs in order, so any number of
// heads fills tiles of consecutive rows. This file holds what the two kernels of the
// call share (the plan of the work and the merge of split tiles) and the kernel for
// few query rows, where reading the cache is what costs: tiles of 16 rows (one token
// of 16 heads) on m16n8k16, the same arithmetic as the sparse decode, with q.K exact
// before fp32 accumulation (codes and, down to 2^-24 of a row's largest value, q as exact
// f16, the fp32 tile scale applied to each tile's partial afterwards). Positions come in order, so a block of 32 that lies in
// one page is a single bulk copy.
//
// The host knows the sizes of the arrays, not the lengths in them: a first launch of
// one CTA reads the lengths and plans the pieces (chunk_plan_kernel), so a captured
// graph serves any lengths. A sequence's tiles are cut into as many pieces each as make the pieces of
// a tile of mean length about as long as was found best for the whole batch (half of a place's share of
// all work and more, at least kMinPiece positions); the pieces of one tile are equal parts of its own
// positions, so those of a causal chunk's first tiles are shorter, or empty, and those of its last up to twice
// as long. They write normalised partials that mla_chunk_merge_kernel joins in piece order.
//
// What bounds the kernel for few rows: 64 sequences of 1 .. 16,384 positions, one token of 16 heads each,
// take 111 us with plan and merge (4 and 4 us), 3.8 TB/s or 0.56 of the measured copy
// rate. The cache comes from DRAM at half its rate because each warp's chain of a block (QK, a
// barrier, softmax, a barrier, PV) is as long: 115 instead of 120 us when all of it is
// made to come from L2, tensor pipe 40 %, issue slots 39 %. Two CTAs an SM is what shared
// memory and registers (168) hold. The look for values that are not finite and the masks
// cost 5 us as long as every block paid for them. Whole blocks of full tiles are free of both; a tile of fewer than
// 16 rows (a token of 5 heads) still takes the masks, because the rows that fill it up attend nothing.
#include <cfloat>
#include <climits>
#include <cmath>

#include "mla_chunk.cuh"

namespace {

using namespace mla;
using namespace mla_chunk;

constexpr int kWarps = 4;                    // consumer warps (one per latent tile)
constexpr int kProducers = 2;                // copy-issuing warps (alternate blocks)
constexpr int kThreads = (kWarps + kProducers) * 32;
constexpr int kConsumerThreads = kWarps * 32;
constexpr int kNB = 32;                      // positions per block
constexpr int kStages = 4;
constexpr int kHeads = kSmallRows;           // query rows per CTA (M of m16n8k16)
constexpr int kStageBytes = kNB * kRowBytes;
constexpr int kSmemStages = kStages * kStageBytes;
constexpr int kSmemRed = kWarps * 4 * 32 * 16;       // QK tile partials: float4 [warp][n-tile][lane]
constexpr int kSmemP = 4 * 32 * 8;                   // P (f16): uint2 [n-tile][lane], A-fragment order
constexpr int kSmemQmax = 3 * kWarps * kHeads * 4;   // |q| maxima, block score maxima, l partials
constexpr int kSmemMisc = 2 * kStages * 8 + kStages * 4 + 16 + 16;   // barriers, present masks, poisoned rows, issued
constexpr int kSmemTotal = kSmemStages + kSmemRed + kSmemP + kSmemQmax + kSmemMisc;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The exp2 offset puts the largest score at kTop (log2 units) and moves only when one is
// kRescaleSlack above that: p <= 2^15 stays in f16's range, whose smallest is 2^-28 of the largest p.
constexpr float kTop = 4.0f, kRescaleSlack = 11.0f;

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Plan of the work (one CTA): how many pieces each sequence's tiles are cut into, and
// the prefixes by which a CTA finds its piece and the merge its rows. A sequence's tiles are
// counted with their mean length. C, the length aimed at for a piece of such a tile, is at least min_piece (the
// pieces themselves may be shorter: 129 positions at C = 128 are 96 and 33), and at least so many eighths
// (first_eighth) of a wave-th of all positions that tiles read, so the pieces number at most tiles +
// 8 / first_eighth wave, and those of split tiles (each more than C, so cut into less than 2 x its length
// / C) at most twice the latter: the sizes of the grid and the workspace.
constexpr int kPlanThreads = 512;
constexpr int kPlanTries = kPlanThreads / 32;

// The k-th piece length tried: first_eighth + k eighths of a wave-th of the work.
__device__ __forceinline__ int try_piece(const ChunkArgs& a, int64_t share, int k) {
    const int64_t most = INT_MAX & ~(a.align - 1);         // no context is longer: nothing is split then
    const int64_t e = a.first_eighth + k;
    int64_t c = share < most ? (share * e + 7) >> 3 : most;
    c = (c + a.align - 1) & ~static_cast<int64_t>(a.align - 1);
    c = c < a.min_piece ? a.min_piece : c;
    return static_cast<int>(c < most ? c : most);
}
// Pieces of a tile of `len` positions. (The quotient rounds: a piece more or less.)
__device__ __forceinline__ int pieces_of(int len, int C) {
    const float q = __fdiv_rn(static_cast<float>(len), static_cast<float>(C));
    return q <= 1.0f ? 1 : static_cast<int>(ceilf(q));
}

__device__ __forceinline__ int64_t plan_sum(int64_t v, int64_t* buf) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) t += buf[w];
    return t;
}

// Exclusive prefix over the CTA; total in `all`.
__device__ __forceinline__ int plan_scan(int v, int& all, int64_t* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int off = 0;
    all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int c = static_cast<int>(buf[w]);
        off += w < warp ? c : 0;
        all += c;
    }
    return off + incl - v;
}

// The largest value in the threads before this one (INT_MIN for the first); the CTA's in `all`.
__device__ __forceinline__ int plan_scan_max(int v, int& all, int64_t* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = max(incl, x);
    }
    __syncthreads();
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = INT_MIN;
    all = INT_MIN;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int c = static_cast<int>(buf[w]);
        if (w < warp) before = max(before, c);
        all = max(all, c);
    }
    return before;
}

__global__ void __launch_bounds__(kPlanThreads)
chunk_plan_kernel(const ChunkArgs a) {
    __shared__ int64_t buf[kPlanThreads / 32];
    __shared__ int64_t cost[kPlanTries];
    __shared__ int tries[kPlanTries], counts[kPlanTries];
    __shared__ int lengths[kPlanThreads], place[kPlanThreads];
    __shared__ int32_t tiles_s[kPlanThreads], lens_s[kPlanThreads];
    // Each sequence's tiles and mean length, until the prefixes take their place.
    int32_t* const tile_counts = a.n_seq <= kPlanThreads ? tiles_s : a.part0;
    int32_t* const lens = a.n_seq <= kPlanThreads ? lens_s : a.mrow0;
    pdl_wait();
    pdl_launch_dependents();
    // A sequence is taken if its start is not below any earlier one, nor its end below its
    // start or past T: so the sequences taken are disjoint, and together at most T tokens.
    int64_t work = 0;
    int longest = 0;
    int top = 0;                                       // the largest start so far
    for (int s0 = 0; s0 < a.n_seq; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        const int start = s < a.n_seq ? __ldg(a.q_start + s) : INT_MIN;
        int all;
        const int before = max(top, plan_scan_max(start, all, buf));
        top = max(top, all);
        if (s >= a.n_seq) continue;
        const Seq q = load_seq(a, s);
        const int end = __ldg(a.q_start + s + 1);
        const bool taken = start >= before && start <= end && end <= a.T;
        if (!taken || static_cast<int64_t>(q.len) > static_cast<int64_t>(a.max_pages) * a.page_size)
            atomicOr(a.err, MLA_ERR_CHUNK_RANGE);
        const int tiles = taken ? tiles_of(a, q) : 0, len = mean_limit(a, q);
        tile_counts[s] = tiles;
        lens[s] = len;
        if (tiles > 0) longest = max(longest, len);
        work += static_cast<int64_t>(tiles) * len;
    }
    work = plan_sum(work, buf);                        // (its barriers order the stores above, too)
    // Each warp counts the pieces of one C; the one with the least estimate is taken: pieces that
    // fit one wave end with the longest, more of them (each at piece_cost more) come in waves of
    // average ones. (One token each, 200 sequences of up to 16,384 positions: 249 us, 319 when pieces were at
    // least a place's share; 24 sequences of 2 x 128 heads: 246 and 430. An estimate of all work by the places and
    // half a piece instead of whole waves: 285 and 247.)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) tries[warp] = longest;
    const int64_t share = (work + a.wave - 1) / a.wave;
    __syncthreads();
    for (int w = 0; w < kPlanTries; ++w) longest = max(longest, tries[w]);
    {
        const int c = try_piece(a, share, warp), cut = min(c, longest);
        int n = 0;
        for (int s = lane; s < a.n_seq; s += 32) n += tile_counts[s] * pieces_of(lens[s], c);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) counts[warp] = n;
        if (lane == 0)
            cost[warp] = n <= a.wave ? cut + static_cast<int64_t>(a.piece_cost)
                                     : (n + a.wave - 1) / a.wave * (work / n + a.piece_cost);
    }
    __syncthreads();
    int best = 0;
#pragma unroll
    for (int w = 1; w < kPlanTries; ++w)
        if (cost[w] < cost[best]) best = w;
    const int C = try_piece(a, share, best);
    // More than a wave: the longest pieces first, so that the last to end are short (400 sequences of up
    // to 4,000 positions 189 -> 164 us, the 24 above 262 -> 248; costs under 1 us. Not in batches that would
    // need more than a thread per sequence.)
    const bool sorted = a.n_seq <= kPlanThreads && counts[best] > a.wave;
    if (sorted) {
        int mine = -1;
        if (threadIdx.x < a.n_seq && tile_counts[threadIdx.x] > 0) {
            const int len = lens[threadIdx.x];
            mine = len / pieces_of(len, C);
        }
        lengths[threadIdx.x] = mine;
        __syncthreads();
        if (threadIdx.x < a.n_seq) {
            int rank = 0;
            for (int k = 0; k < a.n_seq; ++k) {
                const int other = lengths[k];
                rank += other > mine || (other == mine && k < threadIdx.x) ? 1 : 0;
            }
            place[rank] = threadIdx.x;
        }
        __syncthreads();
    }
    int p_base = 0, q_base = 0, r_base = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += kPlanThreads) {
        const int i = s0 + threadIdx.x;
        const int s = sorted && i < a.n_seq ? place[i] : i;
        int nk = 1, pieces = 0, parts = 0, rows = 0;
        if (i < a.n_seq) {
            const int tiles = tile_counts[s];
            if (tiles > 0) nk = pieces_of(lens[s], C);
            pieces = tiles * nk;
            if (nk > 1) {
                parts = pieces;
                rows = load_seq(a, s).n * a.H;
            }
        }
        int all;
        const int p = plan_scan(pieces, all, buf) + p_base;
        p_base += all;
        const int k = plan_scan(parts, all, buf) + q_base;
        q_base += all;
        const int r = plan_scan(rows, all, buf) + r_base;
        r_base += all;
        if (i < a.n_seq) {                             // (those of this step have been read: the scans' barriers)
            a.order[i] = s;
            a.piece0[i] = p;
            a.part0[i] = k;
            a.mrow0[i] = r;
            a.split[i] = nk;
        }
    }
    if (threadIdx.x == 0) {
        a.piece0[a.n_seq] = p_base;
        a.part0[a.n_seq] = q_base;
        a.mrow0[a.n_seq] = r_base;
    }
}

// Joins the partials of the split tiles' rows in piece order: lse = ln sum exp(lse_k),
// out = sum exp(lse_k - lse) o_k; a NaN partial makes both NaN. kPerRow warps take a row at a
// time, thread x of a warp dims 128 j + 4x .. 4x + 3, the loads of a few pieces together. Bound by
// the latency of a row's dependent loads (its place, the pieces' lse, their values): four warps a row
// where the GPU holds them all at once (4 sequences: 17.4 us with the rest of the call, 18.6 with one),
// one where that would take several turns (9 sequences, 7,664 rows: 76.5 us with one, 84.1 with four;
// 24 sequences, 6,144 rows: 246.8 and 250.6).
constexpr int kMergeWarps = 4;

template <int kPerRow>
__global__ void __launch_bounds__(32 * kMergeWarps)
mla_chunk_merge_kernel(const ChunkArgs a) {
    constexpr int kDims = kMergeWarps / kPerRow;       // float4 per thread
    constexpr int kBatch = kPerRow == 1 ? 4 : 8;       // pieces whose loads are on their way together
    constexpr int kRows = kMergeWarps / kPerRow;       // rows of a CTA
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int total = a.mrow0[a.n_seq];
    for (int r = blockIdx.x * kRows + warp / kPerRow; r < total; r += gridDim.x * kRows) {
        const int at = find_seq(a.mrow0, a.n_seq, r, lane);
        const int s = a.order[at];
        const int local = r - a.mrow0[at];
        const int np = a.split[at];
        const int tile = local >> a.tile_shift;
        const int64_t row0 = (static_cast<int64_t>(a.part0[at]) + static_cast<int64_t>(tile) * np) * a.tile_rows +
                             (local - tile * a.tile_rows);
        const int64_t grow = static_cast<int64_t>(__ldg(a.q_start + s)) * a.H + local;
        float mx = -INFINITY;
        bool nan = false;
        for (int s0 = 0; s0 < np; s0 += kBatch) {
            float ls[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                ls[q] = (s0 + q < np) ? a.part_lse[row0 + static_cast<int64_t>(s0 + q) * a.tile_rows] : -INFINITY;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                mx = fmaxf(mx, ls[q]);
                nan = nan || ls[q] != ls[q];
            }
        }
        float wsum = 0.0f;
        float4 acc[kDims];
#pragma unroll
        for (int j = 0; j < kDims; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mx != -INFINITY && !nan) {
            for (int s0 = 0; s0 < np; s0 += kBatch) {
                float ls[kBatch];
                float4 v[kBatch][kDims];
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int64_t prow = row0 + static_cast<int64_t>(min(s0 + q, np - 1)) * a.tile_rows;
                    ls[q] = (s0 + q < np) ? a.part_lse[prow] : -INFINITY;
                    // A piece with nothing attended (lse -inf) left its o unwritten.
#pragma unroll
                    for (int j = 0; j < kDims; ++j)
                        v[q][j] = (ls[q] == -INFINITY)
                                      ? make_float4(0.f, 0.f, 0.f, 0.f)
                                      : *reinterpret_cast<const float4*>(a.part_o + prow * kLatent + 128 * (kPerRow == 1 ? j : warp) + 4 * lane);
                }
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const float w = (ls[q] == -INFINITY) ? 0.0f : expf(ls[q] - mx);
                    wsum += w;
#pragma unroll
                    for (int j = 0; j < kDims; ++j) {
                        acc[j].x = fmaf(w, v[q][j].x, acc[j].x);
                        acc[j].y = fmaf(w, v[q][j].y, acc[j].y);
                        acc[j].z = fmaf(w, v[q][j].z, acc[j].z);
                        acc[j].w = fmaf(w, v[q][j].w, acc[j].w);
                    }
                }
            }
        }
        float lse = mx + logf(wsum), inv = 1.0f / wsum;
        if (mx == -INFINITY) { lse = -INFINITY; inv = 0.0f; }
        if (nan) lse = inv = __int_as_float(0x7FC00000);
#pragma unroll
        for (int j = 0; j < kDims; ++j)
            *reinterpret_cast<uint2*>(a.out + grow * kLatent + 128 * (kPerRow == 1 ? j : warp) + 4 * lane) =
                make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
        if (lane == 0 && warp % kPerRow == 0) a.lse[grow] = lse;
    }
}

// Of a stage's 32 rows (lane l takes row l), the part that warp `warp` works on: its latent tile, that tile's scale
// and its 16 RoPE values. Rows where that holds a value that is not finite (a NaN code, a scale or RoPE value that is
// NaN or infinite) are returned; their codes of the tile and its scale become 0. So does the scale of a tile of
// zeros where it is 1, which is what the writer gives it.
template <bool kRopeOn>
__device__ __forceinline__ unsigned mend_part(uint8_t* st, int stride, int warp, int lane) {
    uint8_t* row = st + lane * stride;
    uint32_t odd = 0u, used = 0u;
#pragma unroll 1
    for (int k = 0; k < kTile / 16; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + kTile * warp + 16 * k);
        const uint32_t x = v.x & 0x7f7f7f7fu, y = v.y & 0x7f7f7f7fu, z = v.z & 0x7f7f7f7fu, w = v.w & 0x7f7f7f7fu;
        odd |= (x + 0x01010101u) | (y + 0x01010101u) | (z + 0x01010101u) | (w + 0x01010101u);
        used |= x | y | z | w;
    }
    odd &= 0x80808080u;
    uint32_t* scale = reinterpret_cast<uint32_t*>(row + kScaleOff + 4 * warp);
    odd |= ((*scale & 0x7f800000u) + 0x00800000u) & 0x80000000u;
    if (kRopeOn) {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(row + kTailOff + 32 * warp + 4 * k);
            odd |= ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        }
    }
    if (odd != 0u || (used == 0u && *scale == 0x3f800000u)) *scale = 0u;
    if (odd != 0u) {
#pragma unroll 1
        for (int k = 0; k < kTile / 16; ++k) *reinterpret_cast<uint4*>(row + kTile * warp + 16 * k) = make_uint4(0u, 0u, 0u, 0u);
    }
    return __ballot_sync(0xffffffffu, odd != 0u);
}

template <bool kRopeOn>
__global__ void __launch_bounds__(kThreads, 2)
mla_chunk_small_kernel(const ChunkArgs args) {
    constexpr uint32_t kRowRead = kRopeOn ? kRowBytes : kNopeReadBytes;
    constexpr int kStride = kRowRead;        // staged rows: 164 or 132 words apart, 4 mod 32
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* stages = smem;
    float4* red = reinterpret_cast<float4*>(smem + kSmemStages);
    uint32_t* pbuf = reinterpret_cast<uint32_t*>(smem + kSmemStages + kSmemRed);
    float* qmax_s = reinterpret_cast<float*>(smem + kSmemStages + kSmemRed + kSmemP);
    float* rmax_s = qmax_s + kWarps * kHeads;
    float* lsum_s = rmax_s + kWarps * kHeads;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kSmemStages + kSmemRed + kSmemP + kSmemQmax);
    uint64_t* empty = full + kStages;
    uint32_t* vmask = reinterpret_cast<uint32_t*>(empty + kStages);   // present positions of each stage
    uint32_t* poison_s = vmask + kStages;                             // [2] blocks in turn: positions whose row is not finite
    uint32_t* late_s = poison_s + 2;                                  // a wait ran out
    int* issued_s = reinterpret_cast<int*>(poison_s + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();

    const Piece pc = find_piece(args, blockIdx.x, lane);
    if (pc.seq < 0) return;
    const int k0 = pc.k0, n_keys = pc.k1 - pc.k0;
    const int nblk = (n_keys + kNB - 1) / kNB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        issued_s[0] = issued_s[1] = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < 4) poison_s[threadIdx.x] = 0u;
    __syncthreads();

    if (warp >= kWarps) {
        // ---- producers: warp kWarps + p copies blocks p, p + kProducers, ...; lane j
        // finds the slot of position 32 b + j one block ahead of its copy ----
        const int pw = warp - kWarps;
        const int32_t* bt = args.block_table + static_cast<int64_t>(pc.seq) * args.max_pages;
        int64_t slot = (pw < nblk && pw * kNB + lane < n_keys) ? chunk_slot(args, bt, k0 + pw * kNB + lane) : -1;
        int b = pw, cnt = 0;
        for (; b < nblk; b += kProducers, ++cnt) {
            const int s = b % kStages;
            const int nb = b + kProducers;
            const int64_t next =
                (nb < nblk && nb * kNB + lane < n_keys) ? chunk_slot(args, bt, k0 + nb * kNB + lane) : -1;
            if (b >= kStages && !mbar_wait_bounded(&empty[s], static_cast<uint32_t>(((b / kStages) - 1) & 1))) {
                if (lane == 0) atomicOr(args.err, MLA_ERR_PIPELINE_TIMEOUT);
                break;
            }
            uint8_t* dst = stages + s * kStageBytes;
            const bool present = slot >= 0;
            const unsigned mask = __ballot_sync(0xffffffffu, present);
            if (!present) {
                // An absent position loads nothing: its row is zeros (E4M3 0, scale 0.0).
                uint4* z = reinterpret_cast<uint4*>(dst + lane * kStride);
                for (int k = 0; k < kStride / 16; ++k) z[k] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            __syncwarp();
            const int64_t first = __shfl_sync(0xffffffffu, slot, 0);
            // All 32 rows side by side in the cache, and nothing but rows as staged: one copy.
            const bool run = __all_sync(0xffffffffu, present && slot == first + lane) && args.row_bytes == kRowRead;
            if (lane == 0) {
                vmask[s] = mask;
                mbar_arrive_expect_tx(&full[s], __popc(mask) * kRowRead);
            }
            __syncwarp();
            if (run) {
                if (lane == 0) bulk_g2s(dst, args.cache + first * args.row_bytes, kNB * kRowRead, &full[s]);
            } else if (present) {
                bulk_g2s(dst + lane * kStride, args.cache + slot * args.row_bytes, kRowRead, &full[s]);
            }
            slot = next;
        }
        if (lane == 0) issued_s[pw] = cnt;
        __syncthreads();     // matches the consumers' final barrier
        return;
    }

    // ---- consumers: q of this tile's rows, loads issued first ----
    const int g = lane >> 2;
    const int c = lane & 3;
    uint32_t qraw[2][16];
    uint32_t qr[2][2];
    int lim[2];                              // positions each row attends, counted from k0
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = pc.row0 + g + 8 * r;
        qr[r][0] = qr[r][1] = 0u;
        lim[r] = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) qraw[r][k] = 0u;
        if (row < pc.rows) {
            lim[r] = row_limit(args, pc, row) - k0;
            const __nv_bfloat16* qh = args.q + (pc.grow0 + row) * args.d_qk;
            const uint8_t* p = reinterpret_cast<const uint8_t*>(qh + 128 * warp + 32 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 v = ld_nc_v4(p + 16 * k);
                qraw[r][4 * k + 0] = v.x; qraw[r][4 * k + 1] = v.y;
                qraw[r][4 * k + 2] = v.z; qraw[r][4 * k + 3] = v.w;
            }
            if (kRopeOn) {
                const uint2 v = *reinterpret_cast<const uint2*>(qh + kLatent + 16 * warp + 4 * c);
                qr[r][0] = v.x; qr[r][1] = v.y;
            }
        }
    }
    // ---- consumers: q fragments ----
    float qm[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        qm[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) qm[r] = fmaxf(qm[r], fmaxf(fabsf(bf16lo(qraw[r][k])), fabsf(bf16hi(qraw[r][k]))));
#pragma unroll
        for (int k = 0; k < 2; ++k) qm[r] = fmaxf(qm[r], fmaxf(fabsf(bf16lo(qr[r][k])), fabsf(bf16hi(qr[r][k]))));
        qm[r] = quad_max(qm[r]);
    }
    if (c == 0) {
        qmax_s[warp * kHeads + g] = qm[0];
        qmax_s[warp * kHeads + g + 8] = qm[1];
    }
    bar_sync_or(1, kConsumerThreads, false);
    // A power of two per row brings its largest |q| into [2^7, 2^15): f16's range then holds every value
    // of at least 2^-17 exactly (8 bits of BF16, f16's smallest step is 2^-24), so down to 2^-24 of the row's
    // largest; a smaller one is off by at most 2^-25, 2^-32 of the largest. The RoPE part takes the same power,
    // which is undone on the scores through the per-row softmax factor.
    float qdown[2], rowf[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float mx = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, qmax_s[w * kHeads + g + 8 * r]);
        int e = 0;
        if (mx <= FLT_MAX) frexpf(mx, &e);           // mx < 2^e
        const int k = e > 15 ? e - 15 : e < 8 ? max(e - 8, -126) : 0;
        qdown[r] = ldexpf(1.0f, -k);
        rowf[r] = args.sm_scale_log2 * ldexpf(1.0f, k);
    }
    uint32_t qa[8][4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int wi = 8 * hf + 2 * kk;
            qa[4 * hf + kk][0] = pack_f16x2(bf16lo(qraw[0][wi]) * qdown[0], bf16hi(qraw[0][wi]) * qdown[0]);
            qa[4 * hf + kk][1] = pack_f16x2(bf16lo(qraw[1][wi]) * qdown[1], bf16hi(qraw[1][wi]) * qdown[1]);
            qa[4 * hf + kk][2] = pack_f16x2(bf16lo(qraw[0][wi + 1]) * qdown[0], bf16hi(qraw[0][wi + 1]) * qdown[0]);
            qa[4 * hf + kk][3] = pack_f16x2(bf16lo(qraw[1][wi + 1]) * qdown[1], bf16hi(qraw[1][wi + 1]) * qdown[1]);
        }
    }
    uint32_t qra[4];
    qra[0] = pack_bf16x2(bf16lo(qr[0][0]) * qdown[0], bf16hi(qr[0][0]) * qdown[0]);
    qra[1] = pack_bf16x2(bf16lo(qr[1][0]) * qdown[1], bf16hi(qr[1][0]) * qdown[1]);
    qra[2] = pack_bf16x2(bf16lo(qr[0][1]) * qdown[0], bf16hi(qr[0][1]) * qdown[0]);
    qra[3] = pack_bf16x2(bf16lo(qr[1][1]) * qdown[1], bf16hi(qr[1][1]) * qdown[1]);

    // ---- consumers: main loop ----
    // Per 32-position block: (1) QK partial of tile `warp` for all 32 positions, (2) the
    // four tile partials meet in shared memory and warp w finishes the scores of
    // positions 8w .. 8w+7 (its n-tile) and writes their P, (3) every warp multiplies
    // all 32 rows of P into V of its own tile.
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m_ref[2] = {-INFINITY, -INFINITY};   // exp2 offset per row (log2 units); -inf: nothing seen yet
    float l_run[2] = {0.0f, 0.0f};             // sum of p over this warp's positions
    const int lim_all = __reduce_min_sync(0xffffffffu, min(lim[0], lim[1]));
    float sigma = FLT_MIN;                     // running max of tile `warp`'s row scales
    float inv_sigma = 1.0f / FLT_MIN;
    bool failed = false;

    for (int b = 0; b < nblk; ++b) {
        const int s = b % kStages;
        const bool ok = mbar_wait_bounded(&full[s], static_cast<uint32_t>((b / kStages) & 1));
        uint8_t* st = stages + s * kStageBytes;
        const uint32_t present = vmask[s];
        float acc[4][4], accr[4][4];
        float sc[4][2];
        uint32_t rs[2][2];
        // (1) QK^T of tile `warp`: latent on f16 MMA, RoPE slice on bf16 MMA.
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = accr[nt][i] = 0.0f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint4 kv[4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
                kv[nt] = *reinterpret_cast<const uint4*>(st + (nt * 8 + g) * kStride + 128 * warp + 32 * c + 16 * hf);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const uint32_t wrd = kk == 0 ? kv[nt].x : kk == 1 ? kv[nt].y : kk == 2 ? kv[nt].z : kv[nt].w;
                    uint32_t b0, b1;
                    e4m3x4_to_f16x2x2(wrd, b0, b1);
                    mma_f16(acc[nt], qa[4 * hf + kk], b0, b1);
                }
            }
        }
        if (kRopeOn) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const uint2 rb = *reinterpret_cast<const uint2*>(st + (nt * 8 + g) * kStride + kTailOff + 32 * warp + 8 * c);
                mma_bf16(accr[nt], qra, rb.x, rb.y);
            }
        }
        // Scale of tile `warp` for rows nt*8 + 2c + e (absent rows were
        // zero-filled: scale 0). The same registers serve the PV step.
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                sc[nt][e] = *reinterpret_cast<const float*>(st + (nt * 8 + 2 * c + e) * kStride + kScaleOff + 4 * warp);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            red[(warp * 4 + nt) * 32 + lane] =
                make_float4(fmaf(acc[nt][0], sc[nt][0], accr[nt][0]), fmaf(acc[nt][1], sc[nt][1], accr[nt][1]),
                            fmaf(acc[nt][2], sc[nt][0], accr[nt][2]), fmaf(acc[nt][3], sc[nt][1], accr[nt][3]));
        // The part of PV that does not need P, ahead of the barriers: sigma (the
        // running max of tile `warp`'s scales, by size, so p * |scale| / sigma <= 2^15 in f16),
        // O rescaled when it moves, and the rows' scale / sigma as f16 pairs.
        float smax = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) smax = fmaxf(smax, fmaxf(fabsf(sc[nt][0]), fabsf(sc[nt][1])));
        smax = quad_max(smax);                 // all 32 rows: the same in every lane
        // A value that is not finite in a row's part of this warp shows in its products with any finite query
        // row (0 * it is not 0), so with rows 0 .. 7. A tile of zeros has the scale 1, which beside small values
        // would take the bits of their scale / sigma for nothing. Both are rare and looked into behind barrier 1.
        bool odd = false;
        if (smax > sigma) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) odd |= (sc[nt][0] == 1.0f) | (sc[nt][1] == 1.0f);
            odd = __any_sync(0xffffffffu, odd) | !(smax <= FLT_MAX);
            if (!odd) {
                const float f = sigma / smax;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] *= f; o[i][1] *= f; o[i][2] *= f; o[i][3] *= f;
                }
                sigma = smax;
                inv_sigma = 1.0f / smax;
            }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            rs[kb][0] = pack_f16x2(sc[2 * kb][0] * inv_sigma, sc[2 * kb][1] * inv_sigma);
            rs[kb][1] = pack_f16x2(sc[2 * kb + 1][0] * inv_sigma, sc[2 * kb + 1][1] * inv_sigma);
        }
        float sum[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            sum[nt] = fabsf(fmaf(acc[nt][0], sc[nt][0], accr[nt][0])) + fabsf(fmaf(acc[nt][1], sc[nt][1], accr[nt][1]));
        odd |= !((sum[0] + sum[1]) + (sum[2] + sum[3]) <= FLT_MAX);
        if (!ok) *late_s = 1u;
        uint32_t poison = 0u;                  // positions whose row holds a value that is not finite
        // Barrier 1 also carries that, or a timeout of any warp, to all of them (one answer per warp: it takes whole warps).
        if (bar_sync_or(1, kConsumerThreads, __any_sync(0xffffffffu, odd | !ok))) {
            if (*late_s != 0u) { failed = true; break; }
            // Each warp takes such rows out of its part: their codes become zeros, so that a position masked for a
            // query row cannot reach it through 0 * NaN in PV, and their products 0 (the other rows' stand: the
            // MMA's columns are apart); their scores become NaN below. Then sigma and the ratios again.
            const unsigned gone = mend_part<kRopeOn>(st, kStride, warp, lane);
            if (lane == 0 && gone != 0u) atomicOr(&poison_s[b & 1], gone);
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                float4 part = red[(warp * 4 + nt) * 32 + lane];
                if (((gone >> (nt * 8 + 2 * c)) & 1u) != 0u) part.x = part.z = 0.0f;
                if (((gone >> (nt * 8 + 2 * c + 1)) & 1u) != 0u) part.y = part.w = 0.0f;
                red[(warp * 4 + nt) * 32 + lane] = part;
            }
            const float* scale = reinterpret_cast<const float*>(st + kScaleOff + 4 * warp);
            const float large = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(scale[lane * (kStride / 4)]))));
            if (large > sigma) {
                const float f = sigma / large;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] *= f; o[i][1] *= f; o[i][2] *= f; o[i][3] *= f;
                }
                sigma = large;
                inv_sigma = 1.0f / large;
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 16 * kb + 8 * h + 2 * c;
                    rs[kb][h] = pack_f16x2(scale[row * (kStride / 4)] * inv_sigma, scale[(row + 1) * (kStride / 4)] * inv_sigma);
                }
            __syncwarp();
            bar_sync_or(1, kConsumerThreads, false);
            poison = poison_s[b & 1];
        }
        // (that word was last read ahead of the barrier 2 before, and is next written after this block's)
        if (threadIdx.x == 0) poison_s[(b + 1) & 1] = 0u;

        // (2) scores of n-tile `warp`: positions 8*warp + 2c + {0,1}, rows g and g+8.
        float4 a = red[warp * 32 + lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 bq = red[(w * 4 + warp) * 32 + lane];
            a.x += bq.x; a.y += bq.y; a.z += bq.z; a.w += bq.w;
        }
        float sv[4] = {a.x * rowf[0], a.y * rowf[0], a.z * rowf[1], a.w * rowf[1]};
        if ((~present | poison) != 0u || kNB * (b + 1) > lim_all) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 8 * warp + 2 * c + (i & 1);
                if (((poison >> j) & 1u) != 0u) sv[i] = __int_as_float(0x7FC00000);
                if (((present >> j) & 1u) == 0u || kNB * b + j >= lim[i >> 1]) sv[i] = -INFINITY;
            }
        }
        const float bm0 = quad_max(fmaxf(sv[0], sv[1]));
        const float bm1 = quad_max(fmaxf(sv[2], sv[3]));
        if (c == 0) {
            rmax_s[warp * kHeads + g] = bm0;
            rmax_s[warp * kHeads + g + 8] = bm1;
        }
        const bool need = bm0 > m_ref[0] + (kTop + kRescaleSlack) || bm1 > m_ref[1] + (kTop + kRescaleSlack);
        float p[4];
        // nothing seen yet: any finite offset makes the masked scores 0
        const float off0 = m_ref[0] == -INFINITY ? 0.0f : m_ref[0];
        const float off1 = m_ref[1] == -INFINITY ? 0.0f : m_ref[1];
        p[0] = ex2_approx(sv[0] - off0);
        p[1] = ex2_approx(sv[1] - off0);
        p[2] = ex2_approx(sv[2] - off1);
        p[3] = ex2_approx(sv[3] - off1);
        uint2* pw = reinterpret_cast<uint2*>(pbuf) + warp * 32 + lane;
        *pw = make_uint2(pack_f16x2(p[0], p[1]), pack_f16x2(p[2], p[3]));
        // V rows of the first PV step: loaded before barrier 2 (they do not depend on P).
        const uint8_t* vb = st + 128 * warp + 16 * g;
        uint4 Vn[4];
        Vn[0] = *reinterpret_cast<const uint4*>(vb + (2 * c + 0) * kStride);
        Vn[1] = *reinterpret_cast<const uint4*>(vb + (2 * c + 1) * kStride);
        Vn[2] = *reinterpret_cast<const uint4*>(vb + (2 * c + 8) * kStride);
        Vn[3] = *reinterpret_cast<const uint4*>(vb + (2 * c + 9) * kStride);
        if (bar_sync_or(1, kConsumerThreads, need)) {
            // Rare after the first block: move the offsets of the rows whose
            // block maximum ran ahead, rescale O and l, and rewrite this warp's P.
            float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                M0 = fmaxf(M0, rmax_s[w * kHeads + g]);
                M1 = fmaxf(M1, rmax_s[w * kHeads + g + 8]);
            }
            const float mn0 = (M0 > m_ref[0] + (kTop + kRescaleSlack)) ? M0 - kTop : m_ref[0];
            const float mn1 = (M1 > m_ref[1] + (kTop + kRescaleSlack)) ? M1 - kTop : m_ref[1];
            const float a0 = mn0 == m_ref[0] ? 1.0f : ex2_approx(m_ref[0] - mn0);     // -inf -> 0
            const float a1 = mn1 == m_ref[1] ? 1.0f : ex2_approx(m_ref[1] - mn1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i][0] *= a0; o[i][1] *= a0; o[i][2] *= a1; o[i][3] *= a1;
            }
            l_run[0] *= a0;
            l_run[1] *= a1;
            m_ref[0] = mn0;
            m_ref[1] = mn1;
            const float of0 = mn0 == -INFINITY ? 0.0f : mn0;
            const float of1 = mn1 == -INFINITY ? 0.0f : mn1;
            p[0] = ex2_approx(sv[0] - of0);
            p[1] = ex2_approx(sv[1] - of0);
            p[2] = ex2_approx(sv[2] - of1);
            p[3] = ex2_approx(sv[3] - of1);
            *pw = make_uint2(pack_f16x2(p[0], p[1]), pack_f16x2(p[2], p[3]));
            bar_sync_or(1, kConsumerThreads, false);
        }
        l_run[0] += p[0] + p[1];
        l_run[1] += p[2] + p[3];

        // (3) PV of tile `warp`.
        const uint2* pr = reinterpret_cast<const uint2*>(pbuf) + lane;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            // A: P of heads (g, g+8) x rows 16kb + 2c + {0,1} and + 8, times the
            // row's tile scale / sigma.
            const uint2 plo = pr[(2 * kb) * 32];
            const uint2 phi = pr[(2 * kb + 1) * 32];
            const uint32_t r01 = rs[kb][0];
            const uint32_t r89 = rs[kb][1];
            uint32_t pa[4];
            pa[0] = hmul2(plo.x, r01);
            pa[1] = hmul2(plo.y, r01);
            pa[2] = hmul2(phi.x, r89);
            pa[3] = hmul2(phi.y, r89);
            // B: V rows j0, j0+1, j0+8, j0+9; lane g takes dims 128w + 16g .. +15,
            // so n-tile (q, i) column n is dim 128w + 16n + 4q + i.
            const int j0 = 16 * kb + 2 * c;
            const uint4 V0 = kb == 0 ? Vn[0] : *reinterpret_cast<const uint4*>(vb + (j0 + 0) * kStride);
            const uint4 V1 = kb == 0 ? Vn[1] : *reinterpret_cast<const uint4*>(vb + (j0 + 1) * kStride);
            const uint4 V2 = kb == 0 ? Vn[2] : *reinterpret_cast<const uint4*>(vb + (j0 + 8) * kStride);
            const uint4 V3 = kb == 0 ? Vn[3] : *reinterpret_cast<const uint4*>(vb + (j0 + 9) * kStride);
#pragma unroll
            for (int qd = 0; qd < 4; ++qd) {
                const uint32_t W0 = qd == 0 ? V0.x : qd == 1 ? V0.y : qd == 2 ? V0.z : V0.w;
                const uint32_t W1 = qd == 0 ? V1.x : qd == 1 ? V1.y : qd == 2 ? V1.z : V1.w;
                const uint32_t W2 = qd == 0 ? V2.x : qd == 1 ? V2.y : qd == 2 ? V2.z : V2.w;
                const uint32_t W3 = qd == 0 ? V3.x : qd == 1 ? V3.y : qd == 2 ? V3.z : V3.w;
                uint32_t b0a, b0b, b0c, b0d, b1a, b1b, b1c, b1d;
                e4m3x4_to_f16x2x2(prmt(W0, W1, 0x5140), b0a, b0b);   // d offsets 0, 1
                e4m3x4_to_f16x2x2(prmt(W0, W1, 0x7362), b0c, b0d);   // d offsets 2, 3
                e4m3x4_to_f16x2x2(prmt(W2, W3, 0x5140), b1a, b1b);
                e4m3x4_to_f16x2x2(prmt(W2, W3, 0x7362), b1c, b1d);
                mma_f16(o[4 * qd + 0], pa, b0a, b1a);
                mma_f16(o[4 * qd + 1], pa, b0b, b1b);
                mma_f16(o[4 * qd + 2], pa, b0c, b1c);
                mma_f16(o[4 * qd + 3], pa, b0d, b1d);
            }
        }
        // The stage is next written by the async proxy (cp.async.bulk): order this
        // warp's generic accesses of it before that write.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }

    __syncthreads();     // all warps: producers done issuing, consumers done reading
    if (failed || issued_s[0] + issued_s[1] < nblk) {
        // A wait ran out: record it, let the copies already issued land (bounded)
        // and leave without touching the outputs.
        if (threadIdx.x == 0) {
            atomicOr(args.err, MLA_ERR_PIPELINE_TIMEOUT);
            for (int p = 0; p < kProducers; ++p) {
                const int cnt = issued_s[p];
                for (int k = max(0, cnt - kStages / kProducers); k < cnt; ++k) {
                    const int bb = p + kProducers * k;
                    (void)mbar_wait_bounded(&full[bb % kStages], static_cast<uint32_t>((bb / kStages) & 1));
                }
            }
        }
        return;
    }

    // ---- epilogue: l over the four warps' positions, then O * sigma / l ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float l = l_run[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (c == 0) lsum_s[warp * kHeads + g + 8 * r] = l;
    }
    bar_sync_or(1, kConsumerThreads, false);
    float lt[2] = {0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        lt[0] += lsum_s[w * kHeads + g];
        lt[1] += lsum_s[w * kHeads + g + 8];
    }
    // l = 0: nothing attended (out 0, lse -inf). l NaN: an attended row holds a value
    // that is not finite (out and lse NaN).
    const float kNaN = __int_as_float(0x7FC00000);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = pc.row0 + g + 8 * r;
        if (row >= pc.rows) continue;
        const float mm = lt[r] > 0.0f ? sigma / lt[r] : (lt[r] == 0.0f ? 0.0f : kNaN);
        const float lse = lt[r] > 0.0f ? (m_ref[r] + log2f(lt[r])) * kLn2 : (lt[r] == 0.0f ? -INFINITY : kNaN);
        // Thread (g, c) holds, for row r, dims 128w + 32c + 16e + 4q + i in
        // o[4q + i][2r + e]: 32 contiguous output values per row.
        if (pc.part < 0) {
            __nv_bfloat16* orow = args.out + (pc.grow0 + row) * kLatent + 128 * warp + 32 * c;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int hq = 0; hq < 2; ++hq) {
                    uint4 v;
                    v.x = pack_bf16x2(o[8 * hq + 0][2 * r + e] * mm, o[8 * hq + 1][2 * r + e] * mm);
                    v.y = pack_bf16x2(o[8 * hq + 2][2 * r + e] * mm, o[8 * hq + 3][2 * r + e] * mm);
                    v.z = pack_bf16x2(o[8 * hq + 4][2 * r + e] * mm, o[8 * hq + 5][2 * r + e] * mm);
                    v.w = pack_bf16x2(o[8 * hq + 6][2 * r + e] * mm, o[8 * hq + 7][2 * r + e] * mm);
                    st_v4(orow + 16 * e + 8 * hq, v);
                }
            }
            if (warp == 0 && c == 0) args.lse[pc.grow0 + row] = lse;
        } else {
            const int64_t prow = static_cast<int64_t>(pc.part) * args.tile_rows + g + 8 * r;
            if (warp == 0 && c == 0) args.part_lse[prow] = lse;
            if (lt[r] == 0.0f) continue;       // lse = -inf: the merge skips this partial's o
            float* orow = args.part_o + prow * kLatent + 128 * warp + 32 * c;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int qd = 0; qd < 4; ++qd)
                    reinterpret_cast<float4*>(orow + 16 * e + 4 * qd)[0] =
                        make_float4(o[4 * qd + 0][2 * r + e] * mm, o[4 * qd + 1][2 * r + e] * mm,
                                    o[4 * qd + 2][2 * r + e] * mm, o[4 * qd + 3][2 * r + e] * mm);
        }
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Two CTAs of the kernel for few rows fit an SM, one of the kernel for many. A piece
// shorter than the minimum saves less than its partial and its share of the merge cost.
constexpr int kCtasPerSm = 2;
constexpr int kMinPiece = 128;
constexpr int kLargeMinPiece = 256;
// What a piece costs beside its positions, in positions (few rows: 192 took 146 us for 90 sequences of up to
// 16,384, 300 and 400 140; many: 384 to 640 are alike), and the shortest length tried, in eighths of
// a place's share (few rows: 3 and 4 alike, 8 took 319 instead of 249 us for 200 sequences; many: 2 and 3
// alike, 8 took 430 instead of 335 for the 24).
constexpr int kPieceCost = 300, kLargePieceCost = 512;
constexpr int kFirstEighth = 4, kLargeFirstEighth = 3;

// The kernel for many rows is taken from this many query rows per sequence, on average (64
// sequences of up to 16,384 positions: 32 rows each 211 us small, 270 large, 36 rows 292
// and 270, 64 rows 418 and 247), and from so many pairs of query rows and positions that a context
// may have (the table's width; the host knows no lengths): it starts about 10 us later (64 rows each, tables as
// wide as the contexts, pairs in millions: 4 sequences, 1.5: 29 us small, 34 large, 2.9: 41 and 43, 5.9: 62 and
// 59; 64 sequences, 2.8: 39 and 38). A table much wider than the contexts always passes: 4 sequences of 64 rows
// and 0.2 million pairs then take 30 us and more instead of 18.
constexpr int kLargeFrom = 36;
constexpr int64_t kLargeWork = 4 << 20;

struct Sizes {
    bool large;
    int tile_rows, wave, first_eighth;
    int64_t max_pieces;
    size_t parts_o, parts_lse, prefix;     // bytes
    size_t total() const { return parts_o + parts_lse + 5 * prefix; }
};

Sizes sizes_of(int T, int H, int n_seq, int64_t positions, int sms) {
    Sizes z;
    const int64_t rows_all = static_cast<int64_t>(T) * H;
    z.large = rows_all >= static_cast<int64_t>(kLargeFrom) * n_seq &&
              (positions > kLargeWork || rows_all * positions >= kLargeWork);
    z.tile_rows = z.large ? kLargeRows : kSmallRows;
    z.wave = z.large ? sms : kCtasPerSm * sms;
    // (a few more than the plan's bounds: the quotient that counts a tile's pieces rounds)
    z.first_eighth = z.large ? kLargeFirstEighth : kFirstEighth;
    const int extra = (8 * z.wave + z.first_eighth - 1) / z.first_eighth + 16;
    z.max_pieces = rows_all / z.tile_rows + (n_seq < T ? n_seq : T) + extra;
    const size_t rows = 2 * static_cast<size_t>(extra) * z.tile_rows;
    z.parts_o = rows * kLatent * sizeof(float);
    z.parts_lse = align256(rows * sizeof(float));
    z.prefix = align256((static_cast<size_t>(n_seq) + 1) * sizeof(int32_t));
    return z;
}

template <typename K, typename... A>
bool launch(K kernel, int64_t grid, int threads, size_t smem, void* stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

}  // namespace

extern "C" size_t mla_chunk_attention_workspace_bytes(int T, int H, int n_seq) {
    if (T <= 0 || H < 1 || H > 128 || n_seq <= 0) return 0;
    const int sms = mla_host::sm_count();
    if (sms <= 0) return 0;
    // whichever kernel the contexts' capacity decides for
    const size_t few = sizes_of(T, H, n_seq, 0, sms).total(), many = sizes_of(T, H, n_seq, INT64_MAX, sms).total();
    return few > many ? few : many;
}

extern "C" int mla_chunk_attention(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv, const int32_t* q_start,
                                   const int32_t* kv_len, const int32_t* block_table, int n_seq, int max_pages,
                                   int page_size, int causal, float sm_scale, void* out_bf16, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    if (T < 0 || n_seq < 0 || max_pages < 0 || page_size <= 0 || kv.num_slots < 0 || !std::isfinite(sm_scale))
        return MLA_EINVAL;
    if (kv.row_bytes != MLA_ROW_BYTES && kv.row_bytes != MLA_ROW_BYTES_NOPE) return MLA_EINVAL;
    if (d_qk != kLatent && d_qk != kLatent + kRope) return MLA_EUNSUPPORTED;
    if (kv.row_bytes == MLA_ROW_BYTES_NOPE && d_qk != kLatent) return MLA_EUNSUPPORTED;   // no tail to read
    if (H < 1 || H > 128) return MLA_EUNSUPPORTED;
    if (T == 0 || n_seq == 0) return MLA_OK;
    if (static_cast<int64_t>(T) * H > INT_MAX / 4 || kv.num_slots > INT_MAX ||
        static_cast<int64_t>(max_pages) * page_size > INT_MAX - 4096)      // positions, rounded up, are an int
        return MLA_EUNSUPPORTED;
    if (q_bf16 == nullptr || out_bf16 == nullptr || lse == nullptr || q_start == nullptr || kv_len == nullptr ||
        (max_pages > 0 && (block_table == nullptr || kv.data == nullptr)))
        return MLA_EINVAL;
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(kv.data, 16) || !aligned(lse, 4) ||
        !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4))
        return MLA_EINVAL;
    int* err = mla_host::device_error_word();
    const int sms = mla_host::sm_count();
    if (err == nullptr || sms <= 0) return MLA_ECUDA;
    const Sizes z = sizes_of(T, H, n_seq, static_cast<int64_t>(max_pages) * page_size, sms);
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < mla_chunk_attention_workspace_bytes(T, H, n_seq))
        return MLA_ENOWORKSPACE;
    const bool rope = d_qk == kLatent + kRope;
    const void* kernel = rope ? reinterpret_cast<const void*>(mla_chunk_small_kernel<true>)
                              : reinterpret_cast<const void*>(mla_chunk_small_kernel<false>);
    if (!mla_host::max_dynamic_smem(kernel, kSmemTotal)) return MLA_ECUDA;

    ChunkArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q_bf16);
    a.cache = static_cast<const uint8_t*>(kv.data);
    a.out = static_cast<__nv_bfloat16*>(out_bf16);
    a.lse = lse;
    a.num_slots = kv.num_slots;
    a.row_bytes = kv.row_bytes;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.block_table = block_table;
    a.n_seq = n_seq;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.T = T;
    a.H = H;
    a.d_qk = d_qk;
    a.causal = causal != 0;
    a.sm_scale_log2 = sm_scale * kLog2e;
    a.err = err;
    a.tile_rows = z.tile_rows;
    a.tile_shift = z.large ? 6 : 4;
    static_assert(kLargeRows == 1 << 6 && kSmallRows == 1 << 4, "tile shift");
    a.align = z.large ? kLargeBlock : kNB;
    a.wave = z.wave;
    a.min_piece = z.large ? kLargeMinPiece : kMinPiece;
    a.first_eighth = z.first_eighth;
    a.piece_cost = z.large ? kLargePieceCost : kPieceCost;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(w);
    w += z.parts_o;
    a.part_lse = reinterpret_cast<float*>(w);
    w += z.parts_lse;
    int32_t** prefixes[5] = {&a.order, &a.piece0, &a.part0, &a.mrow0, &a.split};
    for (int32_t** p : prefixes) {
        *p = reinterpret_cast<int32_t*>(w);
        w += z.prefix;
    }
    if (!launch(chunk_plan_kernel, 1, kPlanThreads, 0, stream, a)) return MLA_ECUDA;
    const bool ok = z.large ? mla_host::launch_chunk_large(a, z.max_pieces, rope, stream)
                    : rope  ? launch(mla_chunk_small_kernel<true>, z.max_pieces, kThreads, kSmemTotal, stream, a)
                            : launch(mla_chunk_small_kernel<false>, z.max_pieces, kThreads, kSmemTotal, stream, a);
    if (!ok) return MLA_ECUDA;
    const int64_t rows = static_cast<int64_t>(T) * H, held = static_cast<int64_t>(sms) * 16;
    if (rows <= held) return launch(mla_chunk_merge_kernel<4>, rows, 32 * kMergeWarps, 0, stream, a) ? MLA_OK : MLA_ECUDA;
    const int64_t ctas = (rows + kMergeWarps - 1) / kMergeWarps;
    return launch(mla_chunk_merge_kernel<1>, ctas < held ? ctas : held, 32 * kMergeWarps, 0, stream, a) ? MLA_OK : MLA_ECUDA;
}
