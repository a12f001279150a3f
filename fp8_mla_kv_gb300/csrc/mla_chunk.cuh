// What the kernels of mla_chunk_attention, mla_tree_attention and mla_block_attention
// share: their arguments, the plan of the work and how a CTA finds its piece in it.
#pragma once

#include "mla_device.cuh"

namespace mla_chunk {

using namespace mla;

constexpr int kSmallRows = 16;         // query rows per tile of the kernel for few rows
constexpr int kLargeRows = 64;         // of the kernel for many rows
constexpr int kLargeBlock = 128;       // positions per block there

// What a token attends: the positions up to its own, or all of them (a limit for each query row); the context before
// the chunk and those of the chunk's tokens that its mask names; or the positions up to its own of the blocks
// that are listed for it, in groups of tokens or (kListed) a token a tile, whose list the CTA reads itself. kTree and kBlocks
// have a mask of the tile's tokens for each position.
enum Form { kDense, kTree, kBlocks, kListed };
constexpr bool has_masks(int form) { return form == kTree || form == kBlocks; }
constexpr int kListMax = 512;          // entries of a list that a CTA reads itself
constexpr int kListPieces = 8;         // pieces of such a token's tile, at most: a cluster

// kBlocks: a block that tokens of a group list.
struct __align__(16) BlockEntry {
    int32_t slot0;                     // of its first position
    int32_t ahead;                     // that position, less the position of the group's first token
    uint32_t tokens;                   // tokens of the group that list it
    int32_t pad;
};

struct ChunkArgs {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    __nv_bfloat16* out;
    float* lse;
    int64_t num_slots, row_bytes;
    const int32_t* q_start;            // [n_seq + 1]
    const int32_t* kv_len;             // [n_seq]
    const int32_t* block_table;        // [n_seq, max_pages]
    int n_seq, max_pages, page_size;
    int T, H, d_qk, causal;
    float sm_scale_log2;
    int* err;
    // The plan (workspace): an order of the sequences, exclusive prefixes in that order, and pieces per
    // tile.
    int tile_rows, tile_shift;         // query rows per tile, a power of two
    int align;                         // positions per block, a power of two: pieces start at multiples of it
    int wave;                          // pieces that fill the GPU once
    int min_piece, first_eighth;       // least length aimed at: positions, eighths of a wave-th of the work
    int piece_cost;                    // of a piece, beside its positions
    int32_t* order;                    // [n_seq] sequences; longest pieces first, where there is more than a wave
    int32_t* piece0;                   // [n_seq + 1] pieces
    int32_t* part0;                    // [n_seq + 1] pieces of split tiles
    int32_t* mrow0;                    // [n_seq + 1] query rows of split tiles
    int32_t* split;                    // [n_seq] pieces per tile
    float* part_o;                     // [parts, tile_rows, 512] normalised partials
    float* part_lse;                   // [parts, tile_rows]
    // kTree
    const uint32_t* mask;              // [T, mask_words]: bit j of row t: token t attends its chunk's token j
    int mask_words;
    // kBlocks: groups of consecutive tokens, each with the blocks that any of its tokens lists, ascending
    const BlockEntry* entries;         // [groups, entry_cap]
    const int2* groups;                // [groups]: number of entries; tokens that are in a sequence
    int entry_cap, group_tokens, group_tiles;      // group_tiles: tiles per group
    int nk;                            // pieces per tile
    // kListed
    const int32_t* lists;              // [T, width]
    int width;
    bool paired;                       // kTree: the plan counts what two waves take by pairs
};

// A sequence's new tokens and context, as far as they are valid.
struct Seq {
    int start, n, len;                 // first token, tokens, context length (the chunk included)
};

__device__ __forceinline__ Seq load_seq(const ChunkArgs& a, int s) {
    Seq q;
    q.start = __ldg(a.q_start + s);
    const int end = __ldg(a.q_start + s + 1);
    q.n = (q.start >= 0 && q.start <= end && end <= a.T) ? end - q.start : 0;
    q.len = max(0, __ldg(a.kv_len + s));
    return q;
}

// Positions that token i of the sequence attends: the first this many.
__device__ __forceinline__ int token_limit(const ChunkArgs& a, const Seq& q, int i) {
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    int64_t lim = a.causal ? static_cast<int64_t>(q.len) - q.n + i + 1 : q.len;
    lim = lim < cap ? lim : cap;
    return lim > 0 ? static_cast<int>(lim) : 0;
}

// What one tile of the sequence reads on average; the plan splits by it.
__device__ __forceinline__ int mean_limit(const ChunkArgs& a, const Seq& q) {
    return q.n == 0 ? 0 : token_limit(a, q, q.n / 2);
}

__device__ __forceinline__ int tiles_of(const ChunkArgs& a, const Seq& q) {
    return (q.n * a.H + a.tile_rows - 1) >> a.tile_shift;
}

struct Piece {
    int seq;                           // -1: no piece; kBlocks: the group
    Seq s;
    int row0, rows;                    // first query row of the tile; query rows of the sequence
    int64_t grow0;                     // the sequence's first row in q, out and lse
    int k0, k1;                        // positions
    int part;                          // partial slot, or -1 when the tile is not split
};

// The largest s in [0, n) with first[s] <= v (first is nondecreasing, first[0] <= v),
// by a 32-way search of the whole warp.
__device__ __forceinline__ int find_seq(const int32_t* first, int n, int v, int lane) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, i < hi && first[min(i, n)] <= v);
        lo += (__popc(at) - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ Piece find_piece(const ChunkArgs& a, int b, int lane) {
    Piece p;
    p.seq = -1;
    if (b >= a.piece0[a.n_seq]) return p;
    const int at = find_seq(a.piece0, a.n_seq, b, lane);
    p.seq = a.order[at];
    p.s = load_seq(a, p.seq);
    const int nk = a.split[at];
    const int local = b - a.piece0[at];
    p.rows = p.s.n * a.H;
    const int tiles = tiles_of(a, p.s);
    const int back = local / nk;
    const int tile = tiles - 1 - back;               // a causal chunk's last tiles are the longest: first
    const int k = local - back * nk;
    p.row0 = tile * a.tile_rows;
    p.grow0 = static_cast<int64_t>(p.s.start) * a.H;
    const int last = min(p.rows, p.row0 + a.tile_rows) - 1;
    const int lim = token_limit(a, p.s, last / a.H);
    const int per = ((lim + nk - 1) / nk + a.align - 1) & ~(a.align - 1);
    p.k0 = static_cast<int>(min(static_cast<int64_t>(lim), static_cast<int64_t>(k) * per));
    p.k1 = static_cast<int>(min(static_cast<int64_t>(lim), static_cast<int64_t>(p.k0) + per));   // (k0 + per may pass 2^31)
    p.part = nk > 1 ? a.part0[at] + tile * nk + k : -1;
    return p;
}

__device__ __forceinline__ int row_limit(const ChunkArgs& a, const Piece& p, int row) {
    return token_limit(a, p.s, row / a.H);
}

// kBlocks, kListed: positions are counted through the group's entries (`count`), one block after the other. The pieces of a
// tile are equal parts of them.
__device__ __forceinline__ Piece block_piece(const ChunkArgs& a, int b, int count) {
    Piece p;
    const int tile = b / a.nk, k = b - tile * a.nk;
    p.seq = tile / a.group_tiles;
    const int first = p.seq * a.group_tokens;
    p.s.start = first;
    p.s.n = min(a.group_tokens, a.T - first);
    p.s.len = count * a.page_size;
    p.rows = p.s.n * a.H;
    p.row0 = (tile - p.seq * a.group_tiles) * a.tile_rows;
    p.grow0 = static_cast<int64_t>(first) * a.H;
    const int per = ((p.s.len + a.nk - 1) / a.nk + a.align - 1) & ~(a.align - 1);
    p.k0 = static_cast<int>(min(static_cast<int64_t>(p.s.len), static_cast<int64_t>(k) * per));
    p.k1 = static_cast<int>(min(static_cast<int64_t>(p.s.len), static_cast<int64_t>(p.k0) + per));
    p.part = a.nk > 1 ? tile * a.nk + k : -1;
    return p;
}

template <int kForm>
__device__ __forceinline__ Piece piece_of(const ChunkArgs& a, int b, int lane) {
    if (kForm != kBlocks) return find_piece(a, b, lane);
    const int2 head = __ldg(&a.groups[b / a.nk / a.group_tiles]);
    Piece p = block_piece(a, b, head.x);
    // (a tile past the group's rows is none: the last group may have fewer)
    if (p.row0 >= p.rows || head.y == 0) p.seq = -1;
    return p;
}

// A tile's tokens are numbered from 0: the one of query row `row`, as a bit.
__device__ __forceinline__ uint32_t token_bit(const ChunkArgs& a, const Piece& p, int row) {
    return 1u << (row / a.H - p.row0 / a.H);
}
// All tokens of a tile (at most 32; rows: of the tile).
__device__ __forceinline__ uint32_t tile_tokens(const ChunkArgs& a, const Piece& p, int rows) {
    const int n = (p.row0 + rows - 1) / a.H - p.row0 / a.H + 1;
    return 0xffffffffu >> (32 - n);
}
// Whether the query row belongs to a token that has an output.
template <int kForm>
__device__ __forceinline__ bool row_lives(const ChunkArgs& a, const Piece& p, int row) {
    return kForm != kBlocks || ((static_cast<uint32_t>(__ldg(&a.groups[p.seq].y)) >> (row / a.H)) & 1u) != 0u;
}

// Slot of a position, or -1 when it is absent: no page there, the reserved slot, or a
// slot past the cache (which is flagged).
__device__ __forceinline__ int64_t chunk_slot(const ChunkArgs& a, const int32_t* bt, int pos) {
    const int page = pos / a.page_size;              // < max_pages: limits are capped
    const int phys = __ldg(bt + page);
    if (phys < 0) return -1;
    const int64_t slot = static_cast<int64_t>(phys) * a.page_size + (pos - page * a.page_size);
    if (slot == 0) return -1;
    if (slot >= a.num_slots) {
        atomicOr(a.err, MLA_ERR_DECODE_INDEX_RANGE);
        return -1;
    }
    return slot;
}

// The same for any form, with the tokens of the tile that attend the position (`rows` query rows in the tile). One that none
// attends (past all of them in their own block, a drafted token that no mask names) is absent: what its row holds, which may
// be past the context, must not move the scale that the tile's values are held by.
template <int kForm>
__device__ __forceinline__ int64_t form_slot(const ChunkArgs& a, const Piece& p, const int32_t* bt, int pos, int rows,
                                             uint32_t& tokens) {
    if (kForm == kBlocks) {
        const int e = pos / a.page_size, off = pos - e * a.page_size;
        const int4 v = __ldg(reinterpret_cast<const int4*>(a.entries + static_cast<int64_t>(p.seq) * a.entry_cap + e));
        const int64_t slot = static_cast<int64_t>(v.x) + off;
        const int ahead = v.y + off;                 // token k of the group attends it from k = ahead on
        tokens = ahead <= 0 ? v.z : ahead > 31 ? 0u : static_cast<uint32_t>(v.z) & (0xffffffffu << ahead);
        if (slot == 0 || tokens == 0u) return -1;
        if (slot >= a.num_slots) {
            atomicOr(a.err, MLA_ERR_DECODE_INDEX_RANGE);
            return -1;
        }
        return slot;
    }
    tokens = 0xffffffffu;
    const int j = pos - (p.s.len - p.s.n);
    if (kForm == kTree && j >= 0) {
        tokens = 0u;
        const int t0 = p.row0 / a.H, n = (p.row0 + rows - 1) / a.H - t0 + 1;
        if (j >> 5 < a.mask_words) {
            const uint32_t* m = a.mask + (static_cast<int64_t>(p.s.start) + t0) * a.mask_words + (j >> 5);
#pragma unroll 1
            for (int i = 0; i < n; ++i) tokens |= ((__ldg(m + static_cast<int64_t>(i) * a.mask_words) >> (j & 31)) & 1u) << i;
        }
        if (tokens == 0u) return -1;
    }
    return chunk_slot(a, bt, pos);
}

template <typename K, typename... A>
bool launch(K kernel, int64_t grid, int threads, size_t smem, void* stream, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

constexpr float kLog2e = 1.4426950408889634f;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Two CTAs of the kernel for few rows fit an SM, one of the kernel for many. A piece
// shorter than the minimum saves less than its partial and its share of the merge cost.
constexpr int kCtasPerSm = 2;
constexpr int kMinPiece = 128;
constexpr int kLargeMinPiece = 256;

}  // namespace mla_chunk

namespace mla_host {
// The kernel for few query rows, the kernel for many (grid bound `pieces`), and the merge of split tiles'
// rows; false on a CUDA error.
bool launch_chunk_small(const mla_chunk::ChunkArgs& a, mla_chunk::Form form, int64_t pieces, void* stream);
bool launch_chunk_large(const mla_chunk::ChunkArgs& a, mla_chunk::Form form, int64_t pieces, void* stream);
bool launch_chunk_merge(const mla_chunk::ChunkArgs& a, mla_chunk::Form form, void* stream);
}
