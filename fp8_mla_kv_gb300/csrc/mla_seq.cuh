// Ragged batches: which sequence a token belongs to, and which sequence a CTA's share of the work is in.
// Sequence s has the tokens q_start[s] .. q_start[s+1]-1 and kv_len[s] positions, its tokens' last. A q_start that is
// not nondecreasing within [0, T] is flagged; which tokens are then found in which sequence is not said, but
// every token found lies in [0, T).
#pragma once

#include "mla_device.cuh"

namespace mla {

struct Batch {
    const int32_t* q_start;            // [n_seq + 1]
    const int32_t* kv_len;             // [n_seq]
    const int32_t* block_table;        // [n_seq, max_pages]
    int n_seq, max_pages, page_size, T;
    int* err;
};

struct Sequence {
    int start, n, len;                 // first token, tokens, positions (at least 0)
};

__device__ __forceinline__ Sequence sequence_of(const Batch& b, int s) {
    Sequence q;
    q.start = __ldg(b.q_start + s);
    const int end = __ldg(b.q_start + s + 1);
    q.n = (q.start >= 0 && q.start <= end && end <= b.T) ? end - q.start : 0;
    q.len = max(0, __ldg(b.kv_len + s));
    return q;
}

// How many parts of `per` make n, for any n: sums like n + per - 1 may pass 2^31.
__host__ __device__ __forceinline__ int parts_of(int n, int per) { return n / per + (n % per != 0 ? 1 : 0); }

// Positions that the table has room for (below 2^31: checked on the host).
__device__ __forceinline__ int capacity(const Batch& b) { return b.max_pages * b.page_size; }

// Position of the sequence's token i: below 0 where the sequence has fewer positions than tokens; one past the
// table counts as the table's last.
__device__ __forceinline__ int position_of(const Batch& b, const Sequence& q, int i) {
    return min(q.len - q.n + i, capacity(b) - 1);
}

// One CTA of a launch looks whether the lengths are in order.
__device__ __forceinline__ void check_lengths(const Batch& b) {
    bool bad = false;
    for (int s = threadIdx.x; s < b.n_seq; s += blockDim.x) {
        const int start = __ldg(b.q_start + s), end = __ldg(b.q_start + s + 1);
        bad = bad || start < 0 || end < start || end > b.T || __ldg(b.kv_len + s) > capacity(b);
    }
    if (bad) atomicOr(b.err, MLA_ERR_CHUNK_RANGE);
}

// The sequence of token t, or -1: the last one that starts at or before t. The whole warp, 32 ways at a time.
__device__ __forceinline__ int sequence_at(const Batch& b, int t, int lane) {
    int lo = 0, hi = b.n_seq;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, i < hi && __ldg(b.q_start + i) <= t) | 1u;
        lo += (__popc(at) - 1) * step;
        hi = min(hi, lo + step);
    }
    const Sequence q = sequence_of(b, lo);
    return t >= q.start && t < q.start + q.n ? lo : -1;
}

// Unit u of the batch, where sequence s has count(s) of them: its sequence (-1: there is none) and which of that
// sequence's it is. All kThreads of the CTA.
template <int kThreads, typename F>
__device__ __forceinline__ int2 find_unit(int n_seq, int u, F count) {
    __shared__ int sums[kThreads / 32];
    __shared__ int2 found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0;
    for (int s0 = 0; s0 < n_seq; s0 += kThreads) {
        const int s = s0 + static_cast<int>(threadIdx.x);
        const int v = s < n_seq ? count(s) : 0;
        int incl = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int off = base, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            off += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        const int first = off + incl - v;
        if (u >= first && u < first + v) found = make_int2(s, u - first);
        __syncthreads();
        if (u < base + all) return found;
        base += all;
    }
    return make_int2(-1, 0);
}

}  // namespace mla

namespace mla_host {

// The checks that the calls on ragged batches share: MLA_OK, or why not.
inline int check_batch(const mla::Batch& b) {
    if (b.T < 0 || b.n_seq < 0 || b.max_pages < 0 || b.page_size <= 0) return MLA_EINVAL;
    if (b.T == 0 || b.n_seq == 0) return MLA_OK;
    if (static_cast<int64_t>(b.max_pages) * b.page_size > INT32_MAX - 4096) return MLA_EUNSUPPORTED;
    const auto off = [](const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    return off(b.q_start) || off(b.kv_len) || (b.max_pages > 0 && off(b.block_table)) ? MLA_EINVAL : MLA_OK;
}

// A launch that may begin while the kernel before it ends (griddepcontrol.wait is its first statement).
template <typename K, typename... A>
bool launch_pdl(K kernel, int64_t grid, int threads, size_t smem, void* stream, A... args) {
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

}  // namespace mla_host
