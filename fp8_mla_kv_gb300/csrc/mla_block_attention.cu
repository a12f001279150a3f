// mla_block_attention: attention over the blocks (pages) that are listed for each token.
//
// The kernels are chunk attention's (mla_chunk.cu, mla_chunk_large.cu); what differs is which positions they
// walk and which of a tile's tokens attend each. A tile's query rows are the (token, head) pairs of a group of
// consecutive tokens (one token where it has 16 heads and more, for few rows, or 64, for many); its positions are those of
// the blocks that any of the group's tokens lists, one after the other, and each block carries a bit per
// token. Neighbouring tokens of a prompt want mostly the same blocks, so a group of four reads and multiplies a
// block once that would be read four times token by token. Tokens of different sequences may share a group: their
// blocks stand side by side then.
//
// 4,096 tokens of 16 heads with 32 blocks of 64 of up to 256 each: 800 us, 360 TFLOP/s of the listed pairs (a group of four has
// 49 blocks, of which each token lists two thirds; of the pairs that are multiplied it is 555). What bounds it is what
// bounds the kernel for many rows, and 20,000 + 8,000 of a tile's 229,000 cycles are its start and end. 64 single tokens:
// 34.2 us, 2.3 TB/s, bound as the kernel for few rows (256 pieces of 16 blocks of 32 positions for 304 places).
//
// Where a tile is one token's of few rows, its CTAs, a cluster, read the list themselves (read_list) and join their parts
// through their shared memory (join_parts). Otherwise a first launch makes the groups' lists (block_lists_kernel; with
// it and the merge the 64 tokens took 38.7 us): a CTA per group marks the listed blocks in a bit
// map, so that a block counts once however often and in whatever order it is listed, and ranks them by prefix counts.
// The pieces of the tiles are planned on the host: it knows how long lists are at most. A captured call serves any
// lengths and lists.
#include <climits>
#include <cmath>

#include "mla_chunk.cuh"
#include "mla_seq.cuh"

namespace {

using namespace mla;
using namespace mla_chunk;

constexpr int kThreads = 256;
constexpr int kWords = 2048;                           // of the bit map: 65,536 blocks at a time
constexpr int kPerThread = kWords / kThreads;

// Blocks of the group's tokens, ascending by sequence and block. A thread keeps up to kKeep entries of the lists (and looks
// the others up again each time). Bound by its chain of loads (sequences, lists, table) and barriers: 10.9 us for 4,096
// tokens' lists of 32 in groups of four.
constexpr int kKeep = 4;

__global__ void __launch_bounds__(kThreads)
block_lists_kernel(const Batch b, const int32_t* __restrict__ blocks, int width, int group_tokens, int64_t num_slots,
                   BlockEntry* __restrict__ entries, int entry_cap, int2* __restrict__ groups) {
    __shared__ uint32_t bits[kWords];
    __shared__ int before[kWords];                     // set bits in the words before
    __shared__ int seq_s[32], pos_s[32];
    __shared__ int sums[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int first = blockIdx.x * group_tokens, n_tokens = min(group_tokens, b.T - first);
    const int32_t* const lists = blocks + static_cast<int64_t>(first) * width;
    const int total = n_tokens * width;
    int block[kKeep], phys[kKeep], token[kKeep];
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = threadIdx.x + j * kThreads;
        block[j] = i < total ? __ldg(lists + i) : -1;
    }
    if (blockIdx.x == 0) check_lengths(b);
    for (int k = warp; k < n_tokens; k += kThreads / 32) {
        const int s = sequence_at(b, first + k, lane);
        int pos = -1;
        if (s >= 0) {
            const Sequence q = sequence_of(b, s);
            pos = position_of(b, q, first + k - q.start);
        }
        if (lane == 0) {
            seq_s[k] = s;
            pos_s[k] = pos;
        }
    }
    __syncthreads();
    // Its page where token k attends something of the block (at or before its own, with a page), else -1.
    auto page_of = [&](int at, int k) {
        const int s = seq_s[k], pos = pos_s[k];
        if (at < 0 || s < 0) return -1;
        if (at >= b.max_pages) atomicOr(b.err, MLA_ERR_DECODE_INDEX_RANGE);
        if (pos < 0 || at > pos / b.page_size) return -1;
        const int page = __ldg(b.block_table + static_cast<int64_t>(s) * b.max_pages + at);
        if (page >= 0 && static_cast<int64_t>(page) * b.page_size >= num_slots) {
            atomicOr(b.err, MLA_ERR_DECODE_INDEX_RANGE);
            return -1;
        }
        return page;
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = threadIdx.x + j * kThreads;
        token[j] = 0;
        phys[j] = -1;
        if (i < total) {
            token[j] = i / width;
            phys[j] = page_of(block[j], token[j]);
        }
    }
    BlockEntry* out = entries + static_cast<int64_t>(blockIdx.x) * entry_cap;
    uint32_t live = 0u;
    int count = 0;                                     // entries so far
    for (int k0 = 0, k1; k0 < n_tokens; k0 = k1) {     // the group's tokens of one sequence
        const int s = seq_s[k0];
        for (k1 = k0 + 1; k1 < n_tokens && seq_s[k1] == s;) ++k1;
        if (s < 0) continue;
        live |= (0xffffffffu >> (32 - (k1 - k0))) << k0;
        if (pos_s[k1 - 1] < 0) continue;               // (their positions ascend)
        const int ahead0 = k0 - pos_s[k0];             // position p is that of the group's token p + ahead0
        const int last = pos_s[k1 - 1] / b.page_size;
        for (int w0 = 0;; w0 += 32 * kWords) {
            const int words = min(kWords, (last - w0) / 32 + 1);
            // f(block, page, token) for the listed ones of these tokens in these words
            auto each = [&](auto f) {
#pragma unroll
                for (int j = 0; j < kKeep; ++j)
                    if (phys[j] >= 0 && token[j] >= k0 && token[j] < k1 && block[j] >= w0 && block[j] - w0 < 32 * words)
                        f(block[j], phys[j], token[j]);
                for (int i = max(k0 * width, kKeep * kThreads) + threadIdx.x; i < k1 * width; i += kThreads) {
                    const int at = __ldg(lists + i), k = i / width;
                    if (at < w0 || at - w0 >= 32 * words) {
                        if (at >= b.max_pages) atomicOr(b.err, MLA_ERR_DECODE_INDEX_RANGE);
                        continue;
                    }
                    const int page = page_of(at, k);
                    if (page >= 0) f(at, page, k);
                }
            };
            __syncthreads();                           // (the step before has read the words)
            for (int i = threadIdx.x; i < words; i += kThreads) bits[i] = 0u;
            __syncthreads();
            each([&](int at, int, int) { atomicOr(&bits[(at - w0) >> 5], 1u << (at & 31)); });
            __syncthreads();
            // Prefix counts: kPerThread words a thread.
            int mine = 0;
#pragma unroll
            for (int j = 0; j < kPerThread; ++j) {
                const int w = threadIdx.x * kPerThread + j;
                mine += w < words ? __popc(bits[w]) : 0;
            }
            int incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += x;
            }
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            int at = count + incl - mine, found = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                at += w < warp ? sums[w] : 0;
                found += sums[w];
            }
#pragma unroll
            for (int j = 0; j < kPerThread; ++j) {
                const int w = threadIdx.x * kPerThread + j;
                if (w >= words) break;
                before[w] = at;
                at += __popc(bits[w]);
            }
            __syncthreads();
            // A block's entry is written by all who list it, alike; then each adds its token's bit.
            auto rank = [&](int x) { return before[(x - w0) >> 5] + __popc(bits[(x - w0) >> 5] & ((1u << (x & 31)) - 1u)); };
            const uint32_t alone = k1 - k0 == 1 ? 1u << k0 : 0u;
            each([&](int x, int page, int) {
                *reinterpret_cast<int4*>(out + rank(x)) = make_int4(page * b.page_size, x * b.page_size + ahead0, static_cast<int>(alone), 0);
            });
            if (alone == 0u) {
                __syncthreads();
                each([&](int x, int, int k) { atomicOr(&out[rank(x)].tokens, 1u << k); });
            }
            count += found;
            if (last - w0 < 32 * kWords) break;
        }
    }
    if (threadIdx.x == 0) groups[blockIdx.x] = make_int2(count, static_cast<int>(live));
}

// What a piece costs beside its positions, in positions, as in chunk attention's plan.
constexpr int kPieceCost = 300, kLargePieceCost = 512;
// The kernel for many rows, as there: from so many query rows per sequence on average, and so many pairs of rows and listed
// positions.
constexpr int kLargeFrom = 36;
constexpr int64_t kLargeWork = 4 << 20;

struct Sizes {
    bool large;
    int tile_rows, group_tokens, group_tiles, nk;
    int64_t groups, tiles;
    size_t parts_o, parts_lse, heads, entries;         // bytes
    size_t total() const { return parts_o + parts_lse + heads + entries; }
};

// nk: the pieces per tile that make the least of waves x (positions of a piece + its cost); without positions, as many
// as are ever taken.
Sizes sizes_of(int T, int H, int width, int64_t positions, bool large, bool alone, int sms) {
    Sizes z;
    z.large = large;
    z.tile_rows = large ? kLargeRows : kSmallRows;
    z.group_tokens = H < z.tile_rows && !alone ? z.tile_rows / H : 1;
    if (z.group_tokens > 32) z.group_tokens = 32;      // a bit each
    z.group_tiles = (H + z.tile_rows - 1) / z.tile_rows;
    z.groups = (static_cast<int64_t>(T) + z.group_tokens - 1) / z.group_tokens;
    z.tiles = z.groups * z.group_tiles;
    const int64_t wave = large ? sms : kCtasPerSm * sms, most = 4 * wave / z.tiles + 1;
    const int cost = large ? kLargePieceCost : kPieceCost, least = large ? kLargeMinPiece : kMinPiece;
    z.nk = positions < 0 ? static_cast<int>(most) : 1;
    int64_t best = INT64_MAX;
    for (int64_t nk = 1; positions >= 0 && nk <= most; ++nk) {
        const int64_t per = (positions + nk - 1) / nk;
        if (nk > 1 && per < least) break;
        const int64_t waves = (z.tiles * nk + wave - 1) / wave, time = waves * (per + cost);
        if (time < best) {
            best = time;
            z.nk = static_cast<int>(nk);
        }
    }
    const size_t rows = z.nk > 1 ? static_cast<size_t>(z.tiles) * z.nk * z.tile_rows : 0;
    z.parts_o = rows * kLatent * sizeof(float);
    z.parts_lse = align256(rows * sizeof(float));
    z.heads = align256(z.groups * sizeof(int2));
    z.entries = static_cast<size_t>(z.groups) * z.group_tokens * width * sizeof(BlockEntry);
    return z;
}

bool takes_large(int T, int H, int n_seq, int64_t positions) {
    const int64_t rows = static_cast<int64_t>(T) * H;
    return rows >= static_cast<int64_t>(kLargeFrom) * n_seq && rows * positions >= kLargeWork;
}

}  // namespace

extern "C" size_t mla_block_attention_workspace_bytes(int T, int H, int width) {
    if (T <= 0 || H < 1 || H > 128 || width < 0) return 0;
    const int sms = mla_host::sm_count();
    if (sms <= 0) return 0;
    // whatever the page size: the most pieces, of either kernel
    size_t most = 0;
    for (const bool large : {false, true}) {
        const Sizes z = sizes_of(T, H, width, -1, large, false, sms);
        if (z.total() > most) most = z.total();
    }
    return most;
}

extern "C" int mla_block_attention(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv, const int32_t* blocks,
                                   int width, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                   int n_seq, int max_pages, int page_size, float sm_scale, void* out_bf16, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    Batch b = {q_start, kv_len, block_table, n_seq, max_pages, page_size, T, nullptr};
    if (width < 0 || kv.num_slots < 0 || !std::isfinite(sm_scale)) return MLA_EINVAL;
    if (kv.row_bytes != MLA_ROW_BYTES && kv.row_bytes != MLA_ROW_BYTES_NOPE) return MLA_EINVAL;
    if (d_qk != kLatent && d_qk != kLatent + kRope) return MLA_EUNSUPPORTED;
    if (kv.row_bytes == MLA_ROW_BYTES_NOPE && d_qk != kLatent) return MLA_EUNSUPPORTED;   // no tail to read
    if (H < 1 || H > 128) return MLA_EUNSUPPORTED;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0) return rc;
    if (static_cast<int64_t>(T) * H > INT_MAX / 4 || kv.num_slots > INT_MAX) return MLA_EUNSUPPORTED;
    if (q_bf16 == nullptr || out_bf16 == nullptr || lse == nullptr || (width > 0 && blocks == nullptr) ||
        (max_pages > 0 && kv.data == nullptr))
        return MLA_EINVAL;
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(kv.data, 16) || !aligned(lse, 4) || !aligned(blocks, 4))
        return MLA_EINVAL;
    // (a token's blocks are at most the table's, however many entries its list has)
    const int64_t listed = width < max_pages ? width : max_pages, positions = listed * page_size;
    const int sms = mla_host::sm_count();
    b.err = mla_host::device_error_word();
    if (b.err == nullptr || sms <= 0) return MLA_ECUDA;
    // Few rows, and tokens that share a tile with none (16 heads and more) or with none of their own sequence (mostly
    // single tokens): each CTA reads its token's list itself, and the pieces of a tile, a cluster, join it. (In groups: 64
    // tokens of 16 heads 38.7 instead of 33.8 us, 8 of 5 heads 25.3 instead of 15.5, 64 of one head 86 instead of 29, but 200 of
    // 8 heads 75 instead of 86.)
    const bool large = takes_large(T, H, n_seq, positions);
    const bool alone = !large && width <= kListMax && static_cast<int64_t>(width) * page_size <= INT_MAX - 4096 &&
                       (H >= kSmallRows || T < 2 * static_cast<int64_t>(n_seq));
    const Sizes z = sizes_of(T, H, width, positions, large, alone, sms);
    if (positions * z.group_tokens > INT_MAX - 4096 || z.tiles * z.nk > INT_MAX ||
        static_cast<int64_t>(z.group_tokens) * width > INT_MAX)
        return MLA_EUNSUPPORTED;
    if (z.total() > 0 && (workspace == nullptr || !aligned(workspace, 16) ||
                          workspace_bytes < mla_block_attention_workspace_bytes(T, H, width)))
        return MLA_ENOWORKSPACE;

    ChunkArgs a = {};
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
    a.sm_scale_log2 = sm_scale * kLog2e;
    a.err = b.err;
    a.tile_rows = z.tile_rows;
    a.tile_shift = z.large ? 6 : 4;
    a.align = z.large ? kLargeBlock : 32;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(w);
    w += z.parts_o;
    a.part_lse = reinterpret_cast<float*>(w);
    w += z.parts_lse;
    int2* groups = reinterpret_cast<int2*>(w);
    w += z.heads;
    BlockEntry* entries = reinterpret_cast<BlockEntry*>(w);
    a.groups = groups;
    a.entries = entries;
    a.entry_cap = z.group_tokens * width;
    a.group_tokens = z.group_tokens;
    a.group_tiles = z.group_tiles;
    a.nk = z.nk;
    a.lists = blocks;
    a.width = width;
    if (alone) {
        a.nk = z.nk < kListPieces ? z.nk : kListPieces;
        return mla_host::launch_chunk_small(a, kListed, z.tiles * a.nk, stream) ? MLA_OK : MLA_ECUDA;
    }
    if (!mla_host::launch_pdl(block_lists_kernel, z.groups, kThreads, 0, stream, b, blocks, width, z.group_tokens,
                              kv.num_slots, entries, a.entry_cap, groups))
        return MLA_ECUDA;
    const bool ok = z.large ? mla_host::launch_chunk_large(a, kBlocks, z.tiles * z.nk, stream)
                            : mla_host::launch_chunk_small(a, kBlocks, z.tiles * z.nk, stream);
    return ok && (z.nk == 1 || mla_host::launch_chunk_merge(a, kBlocks, stream)) ? MLA_OK : MLA_ECUDA;
}
