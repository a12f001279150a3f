// Block-sparse attention, the parts before the attention: mla_block_keys (a mean key for each complete page of the
// cache) and mla_block_select (the blocks that each token attends, from their scores). A block is a page.
#include <climits>

#include "mla_seq.cuh"

namespace {

using namespace mla;

// ---- mean keys: K = (sum over the page's rows of [code x scale | rope]) / rows, BF16 ----
//
// A CTA takes a page that a sequence's new tokens completed, a warp every eighth row: lane l values 16 l .. 16 l + 15
// of the latent (tile l / 8) and, l < 8, RoPE values 8 l .. 8 l + 7, kAhead rows' loads on their way; sums in fp32, the
// warps' joined in shared memory. 256 sequences that complete four pages take 4.1 us in a graph, a launch and the
// chain of its loads; 20,000 tokens of four prompts (283 pages) 6.0 us; 1,048,576 rows 176 us, 4.0 TB/s, 0.59 of the
// measured copy rate: the loads of a page's rows wait for its place, and each warp sums what it loaded before it loads
// on. (Eight pages a CTA: 168 us, but the prompts' case 6.7.)
constexpr int kKeyThreads = 256;
constexpr int kKeyWarps = kKeyThreads / 32;
constexpr int kAhead = 4;

template <bool kRopeOn>
__global__ void __launch_bounds__(kKeyThreads)
block_keys_kernel(const Batch b, const uint8_t* __restrict__ cache, int64_t num_slots, int64_t row_bytes,
                  __nv_bfloat16* __restrict__ keys, int num_keys) {
    constexpr int kDim = kLatent + (kRopeOn ? kRope : 0);
    __shared__ __align__(16) float part[kKeyWarps][kDim];
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) check_lengths(b);
    // pages complete after the new tokens, less those before them
    auto first_page = [&](const Sequence& q) { return max(0, q.len - q.n) / b.page_size; };
    const int2 u = find_unit<kKeyThreads>(b.n_seq, blockIdx.x, [&](int s) {
        const Sequence q = sequence_of(b, s);
        return q.n > 0 ? max(0, min(q.len, capacity(b)) / b.page_size - first_page(q)) : 0;
    });
    if (u.x < 0) return;
    const int page = first_page(sequence_of(b, u.x)) + u.y;
    const int phys = __ldg(b.block_table + static_cast<int64_t>(u.x) * b.max_pages + page);
    if (phys < 0) return;
    const int64_t slot0 = static_cast<int64_t>(phys) * b.page_size;
    const int there = static_cast<int>(min(static_cast<int64_t>(b.page_size), max(static_cast<int64_t>(0), num_slots - slot0)));
    if (phys >= num_keys || there < b.page_size) {
        if (threadIdx.x == 0) atomicOr(b.err, MLA_ERR_PAGE_RANGE);
        if (phys >= num_keys) return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int skip = slot0 == 0 ? 1 : 0;                   // the reserved slot is no row
    float v[16], r[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.0f;
    for (int i0 = skip + warp; i0 < there; i0 += kAhead * kKeyWarps) {
        uint4 code[kAhead], tail[kAhead];
        float scale[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kKeyWarps;
            code[k] = tail[k] = make_uint4(0u, 0u, 0u, 0u);
            scale[k] = 0.0f;
            if (i < there) {
                const uint8_t* row = cache + (slot0 + i) * row_bytes;
                code[k] = ld_nc_v4(row + 16 * lane);
                scale[k] = __ldg(reinterpret_cast<const float*>(row + kScaleOff) + (lane >> 3));
                if (kRopeOn && lane < 8) tail[k] = ld_nc_v4(row + kTailOff + 16 * lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo, hi;
                e4m3x4_to_f16x2x2(w[j], lo, hi);
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                v[4 * j] = fmaf(x.x, scale[k], v[4 * j]);
                v[4 * j + 1] = fmaf(x.y, scale[k], v[4 * j + 1]);
                v[4 * j + 2] = fmaf(y.x, scale[k], v[4 * j + 2]);
                v[4 * j + 3] = fmaf(y.y, scale[k], v[4 * j + 3]);
            }
            if (kRopeOn) {
                const uint32_t t[4] = {tail[k].x, tail[k].y, tail[k].z, tail[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r[2 * j] += bf16lo(t[j]);
                    r[2 * j + 1] += bf16hi(t[j]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(&part[warp][16 * lane + 4 * j]) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    if (kRopeOn && lane < 8) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4*>(&part[warp][kLatent + 8 * lane + 4 * j]) =
                make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    }
    __syncthreads();
    const float rows = static_cast<float>(max(1, there - skip));
    for (int d = 2 * threadIdx.x; d < kDim; d += 2 * kKeyThreads) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kKeyWarps; ++w) {
            const float2 p = *reinterpret_cast<const float2*>(&part[w][d]);
            x += p.x;
            y += p.y;
        }
        *reinterpret_cast<uint32_t*>(keys + static_cast<int64_t>(phys) * kDim + d) = pack_bf16x2(x / rows, y / rows);
    }
}

// ---- selection ----
//
// A score becomes a 32-bit key that orders like it (0: not to be chosen). The last one wanted is found a digit at a time from
// the top, by counting the keys; those above it are taken, and of those equal to it the first ones. The passes over the keys, which are in
// registers, end when a digit's keys are exactly those wanted, and bits in which no two scores differ take none: exponents are near
// each other, and rounded scores end in zeros.
// Up to 512 blocks a warp takes a token, a bit a pass, with no more registers of keys than the token has blocks for: 4,096 tokens
// of up to 256 blocks of a table of 258 take 7.2 us in a graph, bound by instructions. (Keys for the whole table 10.2 us, so two to
// eight tokens a CTA 11.9, two bits a pass 12.3, halving the range of the keys, which equal scores take to the last bit, 14.9, a
// count for each value of a digit 34.) With more blocks a CTA does, two bits a pass, as a pass has a barrier:
// 64 tokens of up to 2,048 blocks 7.3 us, a chain of passes. Beyond 8,192 each pass reads the scores again (from L2).
__device__ __forceinline__ uint32_t order_key(float x) {
    if (!(x > -INFINITY)) return 0u;                       // -inf or NaN: not chosen
    const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);       // (-0 is 0)
    return (u >> 31) != 0u ? ~u : u | 0x80000000u;
}

// The list of a token with n blocks, at most 32 x kPer. A pass counts the keys that are not below the threshold with the next bit set.
template <int kPer>
__device__ __forceinline__ void select_in_warp(const float* __restrict__ row, int n, int sink, int local, int width, int lane,
                                               int32_t* __restrict__ out) {
    uint32_t key[kPer], ones = 0u, zeros = 0u;             // set in any score's key, clear in any
    int there = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = 32 * k + lane;
        const bool always = i < n && (i < sink || i > n - 1 - local);
        key[k] = i < n && !always ? order_key(__ldg(row + i)) : 0u;
        ones |= key[k];
        zeros |= key[k] != 0u ? ~key[k] : 0u;
        key[k] = always ? ~0u : key[k];                    // above all scores' keys
        there += key[k] != 0u ? 1 : 0;
    }
    there = __reduce_add_sync(0xffffffffu, there);
    uint32_t found = 1u;                                   // keys from here on are taken,
    int equal = 0;                                         // or, if above 0, those above and so many of those equal to it
    if (there > width) {
        ones = __reduce_or_sync(0xffffffffu, ones);
        uint32_t differ = ones & __reduce_or_sync(0xffffffffu, zeros);     // bits in which two differ: the others need no pass
        found = ones & ~differ;                            // (from here on there are more than wanted)
        equal = width - sink - local;                      // (there are more blocks than wanted: the two are apart)
        if (equal == 0) found = ~0u;
#pragma unroll 1
        while (differ != 0u && equal != 0) {
            const uint32_t bit = 0x80000000u >> __clz(differ), mid = found | bit;
            differ ^= bit;
            int c = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) c += key[k] >= mid ? 1 : 0;
            c = __reduce_add_sync(0xffffffffu, c);
            if (c >= width) found = mid;                   // (else the bit is clear)
            if (c <= width) equal = width - c;
        }
    }
    // In ascending order; of equal ones the first.
    const uint32_t lower = (1u << lane) - 1u;
    int placed = 0;
    if (equal == 0) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const unsigned taken = __ballot_sync(0xffffffffu, key[k] >= found);
            if (key[k] >= found) out[placed + __popc(taken & lower)] = 32 * k + lane;
            placed += __popc(taken);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const unsigned same = __ballot_sync(0xffffffffu, key[k] == found);
            const bool take = key[k] > found || (key[k] == found && __popc(same & lower) < equal);
            const unsigned taken = __ballot_sync(0xffffffffu, take);
            if (take) out[placed + __popc(taken & lower)] = 32 * k + lane;
            placed += __popc(taken);
            equal = max(0, equal - __popc(same));
        }
    }
    for (int i = placed + lane; i < width; i += 32) out[i] = -1;
}

constexpr int kWarpBlocks = 512;

__global__ void __launch_bounds__(32)
block_select_warp_kernel(const Batch b, const float* __restrict__ scores, int columns, int sink, int local, int width,
                         int32_t* __restrict__ blocks) {
    const int lane = threadIdx.x;
    const int t = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (t == 0) check_lengths(b);
    const int s = sequence_at(b, t, lane);
    if (s < 0) return;
    const Sequence q = sequence_of(b, s);
    const int pos = position_of(b, q, t - q.start);
    int32_t* const out = blocks + static_cast<int64_t>(t) * width;
    const int n = pos < 0 ? 0 : pos / b.page_size + 1;     // blocks up to the token's own
    const float* const row = scores + static_cast<int64_t>(t) * columns;
    if (n <= 128) select_in_warp<4>(row, n, sink, local, width, lane, out);
    else if (n <= 256) select_in_warp<8>(row, n, sink, local, width, lane, out);
    else select_in_warp<kWarpBlocks / 32>(row, n, sink, local, width, lane, out);
}

// kWarps warps with kPer keys a thread hold a token's keys; kWide: more are read again for each pass.
template <int kWarps, int kPer, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
block_select_kernel(const Batch b, const float* __restrict__ scores, int columns, int sink, int local, int width,
                    int32_t* __restrict__ blocks) {
    constexpr int kThreads = 32 * kWarps, kChunk = kThreads * kPer;
    __shared__ uint32_t counts[2][kWarps][3];              // of a pass and the one before, which a slow warp may still read
    __shared__ uint32_t bits[kWarps][2];                   // (apart from them: a warp reads it while others count)
    __shared__ int place[kPer][kWarps];                    // keys above the threshold, and (upper half) equal to it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (t == 0) check_lengths(b);
    const int s = sequence_at(b, t, lane);
    if (s < 0) return;
    const Sequence q = sequence_of(b, s);
    const int pos = position_of(b, q, t - q.start);
    int32_t* out = blocks + static_cast<int64_t>(t) * width;
    const int n = pos < 0 ? 0 : pos / b.page_size + 1;     // blocks up to the token's own
    const float* row = scores + static_cast<int64_t>(t) * columns;
    auto always = [&](int i) { return i < sink || i > n - 1 - local; };
    uint32_t key[kPer];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = base + k * kThreads + threadIdx.x;
            key[k] = 0u;
            if (base + k * kThreads < n) key[k] = i >= n || always(i) ? 0u : order_key(__ldg(row + i));
        }
    };
    load(0);
    const int chunks = kWide ? parts_of(n, kChunk) : 1;
    // The threshold's digits; `left`: how many keys that agree with it so far are still wanted. Where there are no more
    // keys than wanted, all are taken: the threshold is 0, and a key of 0 never is.
    uint32_t found = 0u;
    int left = width - sink - local;                       // (of n > width blocks so many are taken anyway)
    bool all = n <= width;                                 // every key from the threshold on is taken
    // Bits in which no two of the scores differ need no pass: exponents are near each other, and rounded scores end in zeros.
    uint32_t ones = 0u, zeros = 0u;                        // set in any, clear in any
#pragma unroll 1
    for (int c = 0; c < chunks && !all; ++c) {
        if (kWide) load(c * kChunk);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (c * kChunk + k * kThreads < n && key[k] != 0u) {
                ones |= key[k];
                zeros |= ~key[k];
            }
    }
    ones = __reduce_or_sync(0xffffffffu, ones);
    zeros = __reduce_or_sync(0xffffffffu, zeros);
    if (lane == 0) {
        bits[warp][0] = ones;
        bits[warp][1] = zeros;
    }
    __syncthreads();
    ones = __reduce_or_sync(0xffffffffu, lane < kWarps ? bits[lane][0] : 0u);
    zeros = __reduce_or_sync(0xffffffffu, lane < kWarps ? bits[lane][1] : 0u);
    const uint32_t differ = ones & zeros;
    int turn = 0;
#pragma unroll 1
    for (int shift = 30; shift >= 0 && !all; shift -= 2) {
        if (((differ >> shift) & 3u) == 0u) {
            found |= ones & (3u << shift);
            continue;
        }
        turn ^= 1;
        int c1 = 0, c2 = 0, c3 = 0;                        // keys whose next digit is 1, 2, 3
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            if (kWide) load(c * kChunk);
            uint32_t packed = 0u;                          // ten bits each: at most 32 x kPer in a warp
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (c * kChunk + k * kThreads >= n) break;
                const uint32_t d = ((key[k] ^ found) >> shift) - 1u;       // agrees above: -1 .. 2, the digit less 1
                packed += d < 3u ? 1u << (10u * d) : 0u;
            }
            packed = __reduce_add_sync(0xffffffffu, packed);
            c1 += packed & 1023u;
            c2 += (packed >> 10) & 1023u;
            c3 += packed >> 20;
        }
        if (lane == 0) {
            counts[turn][warp][0] = c1;
            counts[turn][warp][1] = c2;
            counts[turn][warp][2] = c3;
        }
        __syncthreads();
        c1 = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[turn][lane][0] : 0);
        c2 = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[turn][lane][1] : 0);
        c3 = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[turn][lane][2] : 0);
        uint32_t digit = 3u;
        int here = c3;
        if (left > here) { left -= here; here = c2; digit = 2u; }
        if (digit == 2u && left > here) { left -= here; here = c1; digit = 1u; }
        if (digit == 1u && left > here) { left -= here; digit = 0u; }
        found |= digit << shift;
        all = digit != 0u && left == here;                 // (the lower digits stay 0: any are taken)
    }
    // Those above the threshold and the first `left` of those equal to it, in ascending order.
    auto above = [&](uint32_t x, int i) { return (x != 0u && (all ? x >= found : x > found)) || (i < n && always(i)); };
    auto equal = [&](uint32_t x) { return !all && found != 0u && x == found; };
    const uint32_t lower = (1u << lane) - 1u;
    int n_above = 0, n_equal = 0;                          // before this step's
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        if (kWide) load(c * kChunk);
        __syncthreads();                                   // (the chunk before has been placed)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const unsigned a = __ballot_sync(0xffffffffu, above(key[k], c * kChunk + k * kThreads + threadIdx.x)), e = __ballot_sync(0xffffffffu, equal(key[k]));
            if (lane == 0) place[k][warp] = __popc(a) | __popc(e) << 16;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (c * kChunk + k * kThreads >= n) break;
            const int i = c * kChunk + k * kThreads + threadIdx.x;
            const bool a = above(key[k], i), e = equal(key[k]);
            const unsigned am = __ballot_sync(0xffffffffu, a), em = __ballot_sync(0xffffffffu, e);
            const int mine = lane < kWarps ? place[k][lane] : 0;
            const int total = __reduce_add_sync(0xffffffffu, mine), before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
            const int e_rank = n_equal + (before >> 16) + __popc(em & lower);
            if (a || (e && e_rank < left))
                out[n_above + (before & 0xffff) + __popc(am & lower) + min(e_rank, left)] = i;
            n_above += total & 0xffff;
            n_equal += total >> 16;
        }
    }
    for (int i = n_above + min(n_equal, left) + threadIdx.x; i < width; i += kThreads) out[i] = -1;
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

extern "C" int mla_block_keys(mla_kv_cache_t kv, int d_qk, const int32_t* q_start, const int32_t* kv_len,
                              const int32_t* block_table, int n_seq, int max_pages, int page_size, int T, void* keys_bf16,
                              int num_keys, void* stream) {
    Batch b = {q_start, kv_len, block_table, n_seq, max_pages, page_size, T, nullptr};
    if (num_keys < 0 || kv.num_slots < 0) return MLA_EINVAL;
    if (kv.row_bytes != MLA_ROW_BYTES && kv.row_bytes != MLA_ROW_BYTES_NOPE) return MLA_EINVAL;
    if (d_qk != kLatent && d_qk != kLatent + kRope) return MLA_EUNSUPPORTED;
    if (kv.row_bytes == MLA_ROW_BYTES_NOPE && d_qk != kLatent) return MLA_EUNSUPPORTED;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0 || max_pages == 0) return rc;
    if (kv.data == nullptr || off(kv.data, 16) || off(keys_bf16, 16) || (keys_bf16 == nullptr && num_keys > 0)) return MLA_EINVAL;
    b.err = mla_host::device_error_word();
    if (b.err == nullptr) return MLA_ECUDA;
    // n tokens complete at most (n - 1) / page_size + 1 pages
    const int64_t units = static_cast<int64_t>(T) / page_size + (n_seq < T ? n_seq : T);
    return mla_host::launch_pdl(d_qk == kLatent ? block_keys_kernel<false> : block_keys_kernel<true>, units, kKeyThreads, 0,
                                stream, b, static_cast<const uint8_t*>(kv.data), kv.num_slots, kv.row_bytes,
                                static_cast<__nv_bfloat16*>(keys_bf16), num_keys)
               ? MLA_OK : MLA_ECUDA;
}

extern "C" int mla_block_select(const float* scores, int T, int columns, const int32_t* q_start, const int32_t* kv_len,
                                int n_seq, int page_size, int sink, int local, int width, int32_t* blocks, void* stream) {
    // (the scores have a column for each block of the table)
    Batch b = {q_start, kv_len, nullptr, n_seq, 0, page_size, T, nullptr};
    if (columns < 0 || sink < 0 || local < 1 || width < 0 || static_cast<int64_t>(sink) + local > width) return MLA_EINVAL;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0 || columns == 0) return rc;
    if (static_cast<int64_t>(columns) * page_size > INT_MAX - 4096) return MLA_EUNSUPPORTED;
    if (scores == nullptr || blocks == nullptr || off(scores, 4) || off(blocks, 4)) return MLA_EINVAL;
    b.max_pages = columns;
    b.err = mla_host::device_error_word();
    if (b.err == nullptr) return MLA_ECUDA;
    void (*kernel)(const Batch, const float*, int, int, int, int, int32_t*) = block_select_kernel<32, 8, true>;
    int warps = 32;
    if (columns <= kWarpBlocks) { kernel = block_select_warp_kernel; warps = 1; }
    else if (columns <= 1024) { kernel = block_select_kernel<4, 8, false>; warps = 4; }
    else if (columns <= 4096) { kernel = block_select_kernel<16, 8, false>; warps = 16; }
    else if (columns <= 8192) { kernel = block_select_kernel<32, 8, false>; warps = 32; }
    return mla_host::launch_pdl(kernel, T, 32 * warps, 0, stream, b, scores, columns, sink, local, width, blocks) ? MLA_OK
                                                                                                                : MLA_ECUDA;
}
