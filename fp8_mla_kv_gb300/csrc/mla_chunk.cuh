// What the kernels of mla_chunk_attention share: their arguments, the plan of the
// work and how a CTA finds its piece in it.
#pragma once

#include "mla_device.cuh"

namespace mla_chunk {

using namespace mla;

constexpr int kSmallRows = 16;         // query rows per tile of the kernel for few rows
constexpr int kLargeRows = 64;         // of the kernel for many rows
constexpr int kLargeBlock = 128;       // positions per block there

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
    int seq;                           // -1: no piece
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

}  // namespace mla_chunk

namespace mla_host {
// Launches the kernel for many query rows (grid bound `pieces`), false on a CUDA error.
bool launch_chunk_large(const mla_chunk::ChunkArgs& a, int64_t pieces, bool rope, void* stream);
}
