// Drafted trees: mla_tree_mask (who attends whom, and where each token stands) and
// mla_tree_commit (the accepted path's rows moved together). The attention itself is a form of
// chunk attention (mla_chunk.cu).
//
// A sequence's drafted tokens are the last of its positions, in the order in which they were drafted: a
// token's parent comes before it. Token i stands for the position L - n + depth(i), which is the one
// its rotary part is turned by, while its row lies at L - n + i.
#include <climits>

#include "mla_seq.cuh"

namespace {

using namespace mla;

// A thread walks one token's ancestors, which come in descending order: a word of the mask is complete when the
// walk leaves it. Bound by the walk's dependent loads, one per level of the tree: 16 trees of up to 31 tokens
// take 4.4 us by themselves, 8 trees of 60 tokens 5.7.
constexpr int kMaskThreads = 128;

__global__ void __launch_bounds__(kMaskThreads)
tree_mask_kernel(const Batch b, const int32_t* __restrict__ parent, uint32_t* __restrict__ mask, int words,
                 int32_t* __restrict__ positions) {
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) check_lengths(b);
    const int2 u = find_unit<kMaskThreads>(b.n_seq, blockIdx.x, [&](int s) {
        return parts_of(sequence_of(b, s).n, kMaskThreads);
    });
    if (u.x < 0) return;
    const Sequence q = sequence_of(b, u.x);
    const int i = u.y * kMaskThreads + threadIdx.x;
    if (i >= q.n) return;
    uint32_t* row = mask + (static_cast<int64_t>(q.start) + i) * words;
    int word = words - 1, depth = 0;
    uint32_t bits = 0u;
    bool bad = words > 0 && i >= 32 * static_cast<int64_t>(words);
    for (int at = i; at >= 0;) {
        if (at >> 5 <= word) {                       // (a token past the mask has no bit)
            for (; word > at >> 5; --word) {
                row[word] = bits;
                bits = 0u;
            }
            bits |= 1u << (at & 31);
        }
        int up = __ldg(parent + q.start + at);
        if (up >= at) {                              // not before it: taken as a root, and the walk ends
            bad = true;
            up = -1;
        }
        if (up >= 0) ++depth;
        at = up;
    }
    for (; word >= 0; --word) {
        row[word] = bits;
        bits = 0u;
    }
    if (positions != nullptr) positions[q.start + i] = q.len - q.n + depth;
    if (bad) atomicOr(b.err, MLA_ERR_CHUNK_RANGE);
}

// A CTA takes a sequence, a warp a row at a time. Rows move towards the front (path[j] >= j), so a batch of rows is in
// registers before the first of them is stored, and no later batch reads what an earlier one wrote.
// Bound by its chain of dependent loads (lengths, path, table, rows): in a graph 2.4 us for 16 paths of up to 6 rows,
// 3.0 us for 256 of up to 9 (1.5 MB).
constexpr int kCommitThreads = 256;
constexpr int kCommitWarps = kCommitThreads / 32;

__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(const Batch b, uint8_t* __restrict__ cache, int64_t num_slots, int row_bytes,
                   const int32_t* __restrict__ path, const int32_t* __restrict__ path_len, int max_path, int32_t* len_out) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int start = __ldg(b.q_start + s), end = __ldg(b.q_start + s + 1), len = b.kv_len[s];
    const int prefix = len - (end - start);
    if (start < 0 || end < start || len > capacity(b) || prefix < 0) {
        if (threadIdx.x == 0) {
            atomicOr(b.err, MLA_ERR_CHUNK_RANGE);
            if (len_out != nullptr) len_out[s] = len;
        }
        return;
    }
    const int n = end - start;
    const int32_t* p = path + static_cast<int64_t>(s) * max_path;
    const int asked = __ldg(path_len + s);
    int count = max(0, min(asked, min(max_path, n)));
    // Up to the first entry that is not above the one before it, or not one of the tokens.
    __shared__ int cut;
    if (threadIdx.x == 0) cut = count;
    __syncthreads();
    for (int j = threadIdx.x; j < count; j += kCommitThreads) {
        const int at = __ldg(p + j);
        if (at < 0 || at >= n || (j > 0 && at <= __ldg(p + j - 1))) atomicMin(&cut, j);
    }
    __syncthreads();
    count = cut;
    if (threadIdx.x == 0) {
        if (count != asked) atomicOr(b.err, MLA_ERR_CHUNK_RANGE);
        if (len_out != nullptr) len_out[s] = prefix + count;
    }
    const int32_t* bt = b.block_table + static_cast<int64_t>(s) * b.max_pages;
    auto slot_of = [&](int pos) -> int64_t {         // -1: not there
        const int page = pos / b.page_size, phys = __ldg(bt + page);
        const int64_t slot = static_cast<int64_t>(phys) * b.page_size + (pos - page * b.page_size);
        if (phys >= 0 && slot > 0 && slot < num_slots) return slot;
        if (lane == 0) atomicOr(b.err, MLA_ERR_PAGE_RANGE);
        return -1;
    };
    const int units = row_bytes / 16;                // 41 or 33
    for (int j0 = 0; j0 < count; j0 += kCommitWarps) {
        const int j = j0 + warp;
        const int at = j < count ? __ldg(p + j) : j;
        int64_t dst = -1, src = -1;
        if (at != j) {
            src = slot_of(prefix + at);
            dst = slot_of(prefix + j);
        }
        const bool moves = src >= 0 && dst >= 0;
        uint4 v[2];
        if (moves) {
            const uint4* from = reinterpret_cast<const uint4*>(cache + src * row_bytes);
            v[0] = from[lane];
            if (lane + 32 < units) v[1] = from[lane + 32];
        }
        __syncthreads();
        if (moves) {
            uint4* to = reinterpret_cast<uint4*>(cache + dst * row_bytes);
            to[lane] = v[0];
            if (lane + 32 < units) to[lane + 32] = v[1];
        }
        __syncthreads();                             // (the next batch may store where this one has loaded)
    }
}

bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

extern "C" int mla_tree_mask(const int32_t* parent, int T, const int32_t* q_start, const int32_t* kv_len, int n_seq,
                             uint32_t* mask, int mask_words, int32_t* positions, void* stream) {
    // (no table: any length is in order)
    Batch b = {q_start, kv_len, nullptr, n_seq, 0, INT_MAX, T, nullptr};
    if (mask_words < 0) return MLA_EINVAL;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0) return rc;
    if (parent == nullptr || (mask == nullptr && mask_words > 0) || off4(parent) || off4(mask) || off4(positions)) return MLA_EINVAL;
    b.max_pages = 1;
    b.err = mla_host::device_error_word();
    if (b.err == nullptr) return MLA_ECUDA;
    const int64_t units = static_cast<int64_t>(T) / kMaskThreads + (n_seq < T ? n_seq : T);
    return mla_host::launch_pdl(tree_mask_kernel, units, kMaskThreads, 0, stream, b, parent, mask, mask_words, positions)
               ? MLA_OK : MLA_ECUDA;
}

extern "C" int mla_tree_commit(mla_kv_cache_t kv, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                               int n_seq, int max_pages, int page_size, const int32_t* path, const int32_t* path_len,
                               int max_path, int32_t* kv_len_out, void* stream) {
    // (the tokens are no array of this call: only their numbers count)
    Batch b = {q_start, kv_len, block_table, n_seq, max_pages, page_size, INT_MAX, nullptr};
    if (max_path < 0 || kv.num_slots < 0 || (kv.row_bytes != MLA_ROW_BYTES && kv.row_bytes != MLA_ROW_BYTES_NOPE))
        return MLA_EINVAL;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || n_seq == 0) return rc;
    if (path_len == nullptr || (path == nullptr && max_path > 0) || (kv.data == nullptr && max_pages > 0) || off4(path) ||
        off4(path_len) || off4(kv_len_out) || (reinterpret_cast<uintptr_t>(kv.data) & 15u) != 0)
        return MLA_EINVAL;
    b.err = mla_host::device_error_word();
    if (b.err == nullptr) return MLA_ECUDA;
    return mla_host::launch_pdl(tree_commit_kernel, n_seq, kCommitThreads, 0, stream, b, static_cast<uint8_t*>(kv.data),
                                kv.num_slots, static_cast<int>(kv.row_bytes), path, path_len, max_path, kv_len_out)
               ? MLA_OK : MLA_ECUDA;
}
