// The pages of a cache: copying, forking, freeing and compacting them.
//
// A page is page_size consecutive slots; a block table row holds the physical page of
// each logical page of a sequence (-1: none), and refcount[p] counts the table rows
// that hold page p. Page 0 contains the reserved slot: it is never handed out, moved
// or counted. All of it is whole numbers and byte copies, so every result is exact
// and independent of the order in which CTAs run: counts change by commutative
// integer atomics, and which page goes where is decided by ranks (prefix counts over
// the pages in ascending order), never by arrival.
//
// What bounds each call is the bytes of the pages it copies; the bookkeeping is a
// few short dependent launches, chained by programmatic stream serialization. 1,500 pages
// of 64 rows copied: 126 MB in 18.9 us, the measured copy rate. 32 rows freed and forked: 8.6
// us in a graph, three launches.
#include <climits>

#include "mla_device.cuh"

namespace {

using namespace mla;

constexpr int kScanThreads = 256;
constexpr int kScanPer = 8;                              // pages per thread in a scan
constexpr int kScanPages = kScanThreads * kScanPer;      // pages per scanning CTA
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;                              // 16-byte pieces in flight per lane
constexpr int kUnitBytes = 32 * 16 * kCopyVec;           // bytes a warp moves per unit

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

__device__ __forceinline__ int warp_incl(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += x;
    }
    return v;
}

// Exclusive prefix over the CTA's threads; `total` is the CTA's sum.
__device__ __forceinline__ int block_excl(int v, int& total) {
    __shared__ int wsum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int incl = warp_incl(v, lane);
    __syncthreads();
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int off = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        off += w < warp ? wsum[w] : 0;
        all += wsum[w];
    }
    total = all;
    return off + incl - v;
}

// A warp copies bytes [at, at + kUnitBytes) of a region of `bytes` bytes (multiples of 16).
__device__ __forceinline__ void copy_unit(uint8_t* dst, const uint8_t* src, int64_t at, int64_t bytes, int lane) {
    uint4 v[kCopyVec];
#pragma unroll
    for (int k = 0; k < kCopyVec; ++k) {
        const int64_t o = at + (k * 32 + lane) * 16;
        if (o < bytes) v[k] = ld_nc_v4(src + o);
    }
#pragma unroll
    for (int k = 0; k < kCopyVec; ++k) {
        const int64_t o = at + (k * 32 + lane) * 16;
        if (o < bytes) st_v4(dst + o, v[k]);
    }
}

// ---- copy ----
__global__ void __launch_bounds__(kCopyThreads)
mla_page_copy_kernel(uint8_t* __restrict__ dst_data, const uint8_t* __restrict__ src_data, int64_t page_bytes,
                     int64_t dst_pages, int64_t src_pages, const int32_t* __restrict__ dst,
                     const int32_t* __restrict__ src, int64_t n, int64_t units_per_page, int* __restrict__ err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t units = n * units_per_page;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; u < units; u += nw) {
        const int64_t i = u / units_per_page;
        const int s = __ldg(src + i), d = __ldg(dst + i);
        if (s < 0 || d <= 0) continue;                     // absent, or aimed at the reserved page
        if (s >= src_pages || d >= dst_pages) {
            if (lane == 0) atomicOr(err, MLA_ERR_PAGE_RANGE);
            continue;
        }
        copy_unit(dst_data + d * page_bytes, src_data + s * page_bytes, (u - i * units_per_page) * kUnitBytes, page_bytes,
                  lane);
    }
}

// ---- free ----
__global__ void __launch_bounds__(128)
mla_page_free_kernel(int32_t* __restrict__ refcount, int num_pages, int32_t* __restrict__ table, int n_seq,
                     int max_pages, const int32_t* __restrict__ rows, int* __restrict__ err) {
    pdl_wait();
    pdl_launch_dependents();
    const int r = __ldg(rows + blockIdx.x);
    if (r < 0) return;
    if (r >= n_seq) {
        if (threadIdx.x == 0) atomicOr(err, MLA_ERR_PAGE_RANGE);
        return;
    }
    int32_t* row = table + static_cast<int64_t>(r) * max_pages;
    for (int k = threadIdx.x; k < max_pages; k += blockDim.x) {
        const int p = atomicExch(row + k, -1);             // a row listed twice is freed once
        if (p <= 0) continue;
        if (p >= num_pages) {
            atomicOr(err, MLA_ERR_PAGE_RANGE);
        } else if (atomicSub(refcount + p, 1) <= 0) {      // nobody counted this holder
            atomicAdd(refcount + p, 1);
            atomicOr(err, MLA_ERR_PAGE_COUNT);
        }
    }
}

// ---- fork ----
struct ForkArgs {
    uint8_t* cache;
    int64_t row_bytes;
    int page_size;
    int32_t* refcount;
    int num_pages;
    int32_t* table;
    int n_seq, max_pages;
    const int32_t* parent;
    const int32_t* child;
    const int32_t* lens;
    int n;
    int32_t* chunk_count;      // free pages in each scanned chunk
    int32_t* free_list;        // [chunks, kScanPages] free pages of each chunk, ascending
    int32_t* rank;             // [n] how many new pages the forks before this one take, or -1
    int* err;
};

// What fork f does: its rows and whole pages; false when it is skipped.
__device__ __forceinline__ bool fork_rows(const ForkArgs& a, int f, int& p, int& c, int& len) {
    p = __ldg(a.parent + f);
    c = __ldg(a.child + f);
    len = __ldg(a.lens + f);
    return p >= 0 && c >= 0 && p < a.n_seq && c < a.n_seq && p != c && len >= 0 &&
           static_cast<int64_t>(len) <= static_cast<int64_t>(a.max_pages) * a.page_size;
}

// The physical page that holds the parent's last, not full page; -1 if there is none (page 0,
// whose slot 0 is absent for the parent and would not be in a copy, is none).
__device__ __forceinline__ int fork_part(const ForkArgs& a, int p, int len) {
    if (len % a.page_size == 0) return -1;
    const int e = __ldg(a.table + static_cast<int64_t>(p) * a.max_pages + len / a.page_size);
    if (e >= a.num_pages) atomicOr(a.err, MLA_ERR_PAGE_RANGE);
    return (e > 0 && e < a.num_pages) ? e : -1;
}

// First launch. CTAs 0 .. n-1: fork f's shared pages, in the child's row and in the
// counts. The next CTA ranks the forks that need a page. The others list the free
// pages of their chunk: sharing never changes whether a page is free, because a page
// that a parent holds has a count already.
__global__ void __launch_bounds__(kScanThreads)
mla_fork_plan_kernel(const ForkArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x;
    int p, c, len;
    if (b < a.n) {
        if (!fork_rows(a, b, p, c, len)) {
            if (threadIdx.x == 0 && p >= 0 && c >= 0) atomicOr(a.err, MLA_ERR_PAGE_RANGE);
            return;
        }
        const int whole = len / a.page_size;
        const int32_t* from = a.table + static_cast<int64_t>(p) * a.max_pages;
        int32_t* to = a.table + static_cast<int64_t>(c) * a.max_pages;
        for (int k = threadIdx.x; k < a.max_pages; k += blockDim.x) {
            int e = k < whole ? from[k] : -1;
            if (e >= a.num_pages) {
                atomicOr(a.err, MLA_ERR_PAGE_RANGE);
                e = -1;
            }
            if (e > 0) atomicAdd(a.refcount + e, 1);
            to[k] = e;
        }
    } else if (b == a.n) {
        int before = 0;
        for (int base = 0; base < a.n; base += blockDim.x) {
            const int f = base + threadIdx.x;
            const bool need = f < a.n && fork_rows(a, f, p, c, len) && fork_part(a, p, len) >= 0;
            int total;
            const int excl = block_excl(need ? 1 : 0, total);
            if (f < a.n) a.rank[f] = need ? before + excl : -1;
            before += total;
        }
    } else {
        const int chunk = b - a.n - 1;
        const int first = chunk * kScanPages + threadIdx.x * kScanPer;
        bool is_free[kScanPer];
        int cnt = 0;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) {
            const int i = first + k;
            is_free[k] = i > 0 && i < a.num_pages && a.refcount[i] == 0;
            cnt += is_free[k] ? 1 : 0;
        }
        int total;
        int at = block_excl(cnt, total);
        int32_t* list = a.free_list + static_cast<int64_t>(chunk) * kScanPages;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k)
            if (is_free[k]) list[at++] = first + k;
        if (threadIdx.x == 0) a.chunk_count[chunk] = total;
    }
}

// The r-th free page in ascending order, or -1 (one warp; every lane gets it).
__device__ __forceinline__ int nth_free(const ForkArgs& a, int r, int chunks, int lane) {
    int before = 0;
    for (int base = 0; base < chunks; base += 32) {
        const int k = base + lane;
        const int cnt = k < chunks ? a.chunk_count[k] : 0;
        const int incl = warp_incl(cnt, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, r >= before + incl - cnt && r < before + incl);
        if (hit != 0u) {
            const int src = __ffs(hit) - 1;
            const int in = r - before - __shfl_sync(0xffffffffu, incl - cnt, src);
            return a.free_list[static_cast<int64_t>(base + src) * kScanPages + in];
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

// Second launch, one warp per (fork, kUnitBytes of a page): the new page of each fork
// that needs one, and the rows of the parent's last page in it.
__global__ void __launch_bounds__(kCopyThreads)
mla_fork_part_kernel(const ForkArgs a, int chunks, int units_per_page) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t units = static_cast<int64_t>(a.n) * units_per_page;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; u < units; u += nw) {
        const int f = static_cast<int>(u / units_per_page);
        const int piece = static_cast<int>(u - static_cast<int64_t>(f) * units_per_page);
        const int r = a.rank[f];
        if (r < 0) continue;
        int p, c, len;
        fork_rows(a, f, p, c, len);
        const int64_t bytes = static_cast<int64_t>(len % a.page_size) * a.row_bytes;
        if (piece > 0 && static_cast<int64_t>(piece) * kUnitBytes >= bytes) continue;
        const int page = nth_free(a, r, chunks, lane);
        if (page < 0) {                                    // the pool ran out: the child's entry stays -1
            if (lane == 0) atomicOr(a.err, MLA_ERR_POOL_EMPTY);
            continue;
        }
        const int64_t page_bytes = a.row_bytes * a.page_size;
        const int from = fork_part(a, p, len);
        if (from < 0) continue;                            // the parent's row was changed meanwhile: not allowed, not read
        copy_unit(a.cache + page * page_bytes, a.cache + from * page_bytes, static_cast<int64_t>(piece) * kUnitBytes, bytes, lane);
        if (piece == 0 && lane == 0) {
            a.table[static_cast<int64_t>(c) * a.max_pages + len / a.page_size] = page;
            a.refcount[page] = 1;
        }
    }
}

// ---- compact ----
struct CompactArgs {
    uint8_t* cache;
    int64_t page_bytes;
    const int32_t* refcount;
    int32_t* refcount_out;
    int num_pages;
    const int32_t* table;
    int32_t* table_out;
    int64_t entries;           // n_seq * max_pages
    int32_t* page_map;         // may be null
    int32_t* chunk_count;      // live pages in each scanned chunk
    uint32_t* live;            // one bit per page
    int32_t* before;           // [num_pages] live pages below each page
    int32_t* low;              // [num_pages] k-th vacant page below the live count
    int32_t* high;             // [num_pages] k-th live page above it
    int32_t* high_ref;         // [num_pages] its count
    int32_t* head;             // [0] live pages, [1] how many of them move
    int* err;
};

// First launch: the live pages as bits, and their number per chunk.
__global__ void __launch_bounds__(kScanThreads)
mla_compact_count_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int base = blockIdx.x * kScanPages;
    const int lane = threadIdx.x & 31;
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) {
        const int i = base + k * kScanThreads + threadIdx.x;
        const bool on = i > 0 && i < a.num_pages && a.refcount[i] > 0;
        const unsigned bits = __ballot_sync(0xffffffffu, on);
        if (lane == 0) {
            a.live[i >> 5] = bits;
            cnt += __popc(bits);
        }
    }
    int total;
    block_excl(cnt, total);
    if (threadIdx.x == 0) a.chunk_count[blockIdx.x] = total;
}

// Second launch: each page's rank among the live ones. With n live pages, a live page
// above n moves to the vacant page of the same rank among the vacant ones in 1 .. n.
__global__ void __launch_bounds__(kScanThreads)
mla_compact_rank_kernel(const CompactArgs a, int chunks) {
    pdl_wait();
    pdl_launch_dependents();
    // live pages in all chunks, and in the chunks before this one
    int mine = 0, all = 0;
    for (int k = threadIdx.x; k < chunks; k += blockDim.x) {
        const int c = a.chunk_count[k];
        all += c;
        mine += k < static_cast<int>(blockIdx.x) ? c : 0;
    }
    int n, start;
    block_excl(all, n);
    block_excl(mine, start);
    // live pages among 1 .. n: the chunks before page n + 1, then the bits of its chunk
    const int cut = n + 1;                                 // pages below this index are counted
    const int cc = cut / kScanPages;
    int upto = 0;
    for (int k = threadIdx.x; k < min(cc, chunks); k += blockDim.x) upto += a.chunk_count[k];
    if (cc < chunks) {
        const int w = cc * (kScanPages / 32) + threadIdx.x;
        if (threadIdx.x < kScanPages / 32 && w * 32 < cut) {
            const int bits = min(32, cut - w * 32);
            upto += __popc(a.live[w] & (bits == 32 ? 0xffffffffu : (1u << bits) - 1u));
        }
    }
    int inside;
    block_excl(upto, inside);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head[0] = n;
        a.head[1] = n - inside;
    }
    const int first = blockIdx.x * kScanPages + threadIdx.x * kScanPer;
    const uint32_t word = a.live[first >> 5] >> (first & 31);
    const uint32_t bits8 = word & ((1u << kScanPer) - 1u);
    int total;
    int rank = start + block_excl(__popc(bits8), total);
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) {
        const int i = first + k;
        if (i >= a.num_pages) break;
        const bool on = (bits8 >> k) & 1u;
        a.before[i] = rank;
        const int count = a.refcount[i];
        if (on && i > n) {
            a.high[rank - inside] = i;
            a.high_ref[rank - inside] = count;
        } else if (!on && i > 0 && i <= n) {
            a.low[i - 1 - rank] = i;                       // pages 1 .. i-1 less the live ones
        }
        a.refcount_out[i] = (on && i > n) ? 0 : count;
        rank += on ? 1 : 0;
    }
}

// Both of these in one CTA, for pools whose live bits fit its shared memory: the whole call
// takes 10.9 us instead of 13.4 for 1,000 pages, 63.7 instead of 66.7 for 16,384 of which a
// quarter move (343 MB, 5.4 TB/s; the move alone runs at the copy rate).
constexpr int kPlanThreads = 1024;
constexpr int kPlanWords = 2 * kPlanThreads;             // 65,536 pages

__global__ void __launch_bounds__(kPlanThreads)
mla_compact_plan_kernel(const CompactArgs a) {
    __shared__ uint32_t bits[kPlanWords];
    __shared__ int below[kPlanWords];                      // live pages before each word
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (a.num_pages + 31) / 32;
    constexpr int kWarps = kPlanThreads / 32, kAhead = 8;   // words of a warp whose counts are on their way together
    for (int w = warp; w < words; w += kWarps * kAhead) {
        int count[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = 32 * (w + kWarps * k) + lane;
            count[k] = i > 0 && i < a.num_pages ? a.refcount[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned on = __ballot_sync(0xffffffffu, count[k] > 0);
            if (lane == 0 && w + kWarps * k < words) {
                bits[w + kWarps * k] = on;
                a.live[w + kWarps * k] = on;
            }
        }
    }
    __syncthreads();
    const int w0 = 2 * threadIdx.x;
    const int c0 = w0 < words ? __popc(bits[w0]) : 0, c1 = w0 + 1 < words ? __popc(bits[w0 + 1]) : 0;
    int n;
    const int first = block_excl(c0 + c1, n);
    below[w0] = first;
    below[w0 + 1] = first + c0;
    __syncthreads();
    const int cut = n + 1;                                 // pages below this index, live: `inside`
    const int inside = (cut >> 5) < words ? below[cut >> 5] + __popc(bits[cut >> 5] & ((1u << (cut & 31)) - 1u)) : n;
    if (threadIdx.x == 0) {
        a.head[0] = n;
        a.head[1] = n - inside;
    }
    for (int w = warp; w < words; w += kWarps * kAhead) {
        int count[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = 32 * (w + kWarps * k) + lane;
            count[k] = i < a.num_pages ? a.refcount[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int at = w + kWarps * k, i = 32 * at + lane;
            if (i >= a.num_pages) break;
            const bool on = (bits[at] >> lane) & 1u;
            const int rank = below[at] + __popc(bits[at] & ((1u << lane) - 1u));
            a.before[i] = rank;
            if (on && i > n) {
                a.high[rank - inside] = i;
                a.high_ref[rank - inside] = count[k];
            } else if (!on && i > 0 && i <= n) {
                a.low[i - 1 - rank] = i;                   // pages 1 .. i-1 less the live ones
            }
            a.refcount_out[i] = (on && i > n) ? 0 : count[k];
        }
    }
}

// Where page p goes: itself, its new place, or -1 when it is not live.
__device__ __forceinline__ int page_target(const CompactArgs& a, int p, int n, int inside) {
    if (p == 0) return 0;
    if (!((a.live[p >> 5] >> (p & 31)) & 1u)) return -1;
    return p <= n ? p : a.low[a.before[p] - inside];
}

// Third launch: the pages' bytes and counts, the table and the map. Sources are live
// pages above n, destinations vacant pages up to n, so no byte is both.
__global__ void __launch_bounds__(kCopyThreads)
mla_compact_move_kernel(const CompactArgs a, int64_t units_per_page) {
    pdl_wait();
    pdl_launch_dependents();
    const int n = a.head[0], moves = a.head[1], inside = n - moves;
    const int64_t nt = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = me; i < a.entries; i += nt) {
        const int e = a.table[i];
        int to = e;
        if (e >= a.num_pages) {
            atomicOr(a.err, MLA_ERR_PAGE_RANGE);
            to = -1;
        } else if (e >= 0) {
            to = page_target(a, e, n, inside);
        }
        a.table_out[i] = to;
    }
    if (a.page_map != nullptr)
        for (int64_t i = me; i < a.num_pages; i += nt) a.page_map[i] = page_target(a, static_cast<int>(i), n, inside);
    const int lane = threadIdx.x & 31;
    const int64_t nw = nt >> 5;
    const int64_t units = moves * units_per_page;
    for (int64_t u = me >> 5; u < units; u += nw) {
        const int64_t m = u / units_per_page;
        const int64_t piece = u - m * units_per_page;
        const int64_t from = a.high[m], to = a.low[m];
        copy_unit(a.cache + to * a.page_bytes, a.cache + from * a.page_bytes, piece * kUnitBytes, a.page_bytes, lane);
        if (piece == 0 && lane == 0) a.refcount_out[to] = a.high_ref[m];
    }
}

int chunks_of(int num_pages) { return (num_pages + kScanPages - 1) / kScanPages; }

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <typename K, typename... A>
bool launch(K kernel, int64_t grid, int threads, void* stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

bool cache_ok(const mla_kv_cache_t& kv) {
    return kv.num_slots >= 0 && (kv.row_bytes == MLA_ROW_BYTES || kv.row_bytes == MLA_ROW_BYTES_NOPE);
}

// Number of whole pages of a cache; a last page that is not whole is not one.
int64_t pages_of(const mla_kv_cache_t& kv, int page_size) { return kv.num_slots / page_size; }

constexpr int kCopyCtasPerSm = 8;

}  // namespace

extern "C" int mla_page_copy(mla_kv_cache_t dst_kv, mla_kv_cache_t src_kv, int page_size, const int32_t* dst,
                             const int32_t* src, int64_t n, void* stream) {
    if (n < 0 || page_size <= 0 || !cache_ok(dst_kv) || !cache_ok(src_kv) || dst_kv.row_bytes != src_kv.row_bytes)
        return MLA_EINVAL;
    if (n == 0) return MLA_OK;
    if (dst_kv.data == nullptr || src_kv.data == nullptr || dst == nullptr || src == nullptr) return MLA_EINVAL;
    if (!aligned(dst_kv.data, 16) || !aligned(src_kv.data, 16) || !aligned(dst, 4) || !aligned(src, 4)) return MLA_EINVAL;
    int* err = mla_host::device_error_word();
    const int sms = mla_host::sm_count();
    if (err == nullptr || sms <= 0) return MLA_ECUDA;
    const int64_t page_bytes = static_cast<int64_t>(page_size) * dst_kv.row_bytes;
    const int64_t upp = (page_bytes + kUnitBytes - 1) / kUnitBytes;
    if (n > INT64_MAX / upp) return MLA_EINVAL;
    int64_t blocks = (n * upp + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    if (blocks > static_cast<int64_t>(sms) * kCopyCtasPerSm) blocks = static_cast<int64_t>(sms) * kCopyCtasPerSm;
    return launch(mla_page_copy_kernel, blocks, kCopyThreads, stream, static_cast<uint8_t*>(dst_kv.data),
                  static_cast<const uint8_t*>(src_kv.data), page_bytes, pages_of(dst_kv, page_size),
                  pages_of(src_kv, page_size), dst, src, n, upp, err)
               ? MLA_OK
               : MLA_ECUDA;
}

extern "C" int mla_page_free(int32_t* refcount, int num_pages, int32_t* block_table, int n_seq, int max_pages,
                             const int32_t* rows, int n, void* stream) {
    if (n < 0 || num_pages <= 0 || n_seq <= 0 || max_pages <= 0) return MLA_EINVAL;
    if (n == 0) return MLA_OK;
    if (refcount == nullptr || block_table == nullptr || rows == nullptr || !aligned(refcount, 4) ||
        !aligned(block_table, 4) || !aligned(rows, 4))
        return MLA_EINVAL;
    int* err = mla_host::device_error_word();
    if (err == nullptr) return MLA_ECUDA;
    return launch(mla_page_free_kernel, n, 128, stream, refcount, num_pages, block_table, n_seq, max_pages, rows, err)
               ? MLA_OK
               : MLA_ECUDA;
}

extern "C" size_t mla_page_workspace_bytes(int num_pages, int n_forks) {
    if (num_pages <= 0 || n_forks < 0) return 0;
    const size_t chunks = static_cast<size_t>(chunks_of(num_pages));
    const size_t padded = chunks * kScanPages;
    const size_t fork = align256(chunks * 4) + align256(padded * 4) + align256(static_cast<size_t>(n_forks) * 4);
    const size_t compact = 256 + align256(chunks * 4) + align256(padded / 8) + 4 * align256(padded * 4);
    return fork > compact ? fork : compact;
}

extern "C" int mla_page_fork(mla_kv_cache_t kv, int page_size, int32_t* refcount, int num_pages, int32_t* block_table,
                             int n_seq, int max_pages, const int32_t* parent, const int32_t* child,
                             const int32_t* lens, int n, void* workspace, size_t workspace_bytes, void* stream) {
    if (n < 0 || page_size <= 0 || num_pages <= 0 || n_seq <= 0 || max_pages <= 0 || !cache_ok(kv)) return MLA_EINVAL;
    if (num_pages > pages_of(kv, page_size) || num_pages > INT_MAX - 2 * kScanPages) return MLA_EINVAL;
    if (n == 0) return MLA_OK;
    if (kv.data == nullptr || refcount == nullptr || block_table == nullptr || parent == nullptr || child == nullptr ||
        lens == nullptr)
        return MLA_EINVAL;
    if (!aligned(kv.data, 16) || !aligned(refcount, 4) || !aligned(block_table, 4) || !aligned(parent, 4) ||
        !aligned(child, 4) || !aligned(lens, 4))
        return MLA_EINVAL;
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < mla_page_workspace_bytes(num_pages, n))
        return MLA_ENOWORKSPACE;
    const int chunks = chunks_of(num_pages);
    if (n > INT_MAX - 1 - chunks) return MLA_EINVAL;
    int* err = mla_host::device_error_word();
    const int sms = mla_host::sm_count();
    if (err == nullptr || sms <= 0) return MLA_ECUDA;
    ForkArgs a;
    a.cache = static_cast<uint8_t*>(kv.data);
    a.row_bytes = kv.row_bytes;
    a.page_size = page_size;
    a.refcount = refcount;
    a.num_pages = num_pages;
    a.table = block_table;
    a.n_seq = n_seq;
    a.max_pages = max_pages;
    a.parent = parent;
    a.child = child;
    a.lens = lens;
    a.n = n;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.chunk_count = reinterpret_cast<int32_t*>(w);
    w += align256(static_cast<size_t>(chunks) * 4);
    a.free_list = reinterpret_cast<int32_t*>(w);
    w += align256(static_cast<size_t>(chunks) * kScanPages * 4);
    a.rank = reinterpret_cast<int32_t*>(w);
    a.err = err;
    const int64_t page_bytes = static_cast<int64_t>(page_size) * kv.row_bytes;
    const int64_t upp = (page_bytes + kUnitBytes - 1) / kUnitBytes;
    if (upp > INT_MAX) return MLA_EINVAL;
    int64_t blocks = (static_cast<int64_t>(n) * upp + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    if (blocks > static_cast<int64_t>(sms) * kCopyCtasPerSm) blocks = static_cast<int64_t>(sms) * kCopyCtasPerSm;
    if (!launch(mla_fork_plan_kernel, static_cast<int64_t>(n) + 1 + chunks, kScanThreads, stream, a)) return MLA_ECUDA;
    return launch(mla_fork_part_kernel, blocks, kCopyThreads, stream, a, chunks, static_cast<int>(upp)) ? MLA_OK : MLA_ECUDA;
}

extern "C" int mla_page_compact(mla_kv_cache_t kv, int page_size, const int32_t* refcount, int32_t* refcount_out,
                                int num_pages, const int32_t* block_table, int32_t* table_out, int n_seq,
                                int max_pages, int32_t* page_map, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (page_size <= 0 || num_pages <= 0 || n_seq < 0 || max_pages < 0 || !cache_ok(kv)) return MLA_EINVAL;
    if (num_pages > pages_of(kv, page_size) || num_pages > INT_MAX - 2 * kScanPages) return MLA_EINVAL;
    const int64_t entries = static_cast<int64_t>(n_seq) * max_pages;
    if (kv.data == nullptr || refcount == nullptr || refcount_out == nullptr ||
        (entries > 0 && (block_table == nullptr || table_out == nullptr)))
        return MLA_EINVAL;
    if (!aligned(kv.data, 16) || !aligned(refcount, 4) || !aligned(refcount_out, 4) || !aligned(block_table, 4) ||
        !aligned(table_out, 4) || !aligned(page_map, 4))
        return MLA_EINVAL;
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < mla_page_workspace_bytes(num_pages, 0))
        return MLA_ENOWORKSPACE;
    int* err = mla_host::device_error_word();
    const int sms = mla_host::sm_count();
    if (err == nullptr || sms <= 0) return MLA_ECUDA;
    const int chunks = chunks_of(num_pages);
    const size_t padded = static_cast<size_t>(chunks) * kScanPages;
    CompactArgs a;
    a.cache = static_cast<uint8_t*>(kv.data);
    a.page_bytes = static_cast<int64_t>(page_size) * kv.row_bytes;
    a.refcount = refcount;
    a.refcount_out = refcount_out;
    a.num_pages = num_pages;
    a.table = block_table;
    a.table_out = table_out;
    a.entries = entries;
    a.page_map = page_map;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.head = reinterpret_cast<int32_t*>(w);
    w += 256;
    a.chunk_count = reinterpret_cast<int32_t*>(w);
    w += align256(static_cast<size_t>(chunks) * 4);
    a.live = reinterpret_cast<uint32_t*>(w);
    w += align256(padded / 8);
    int32_t** lists[4] = {&a.before, &a.low, &a.high, &a.high_ref};
    for (int32_t** l : lists) {
        *l = reinterpret_cast<int32_t*>(w);
        w += align256(padded * 4);
    }
    a.err = err;
    const int64_t upp = (a.page_bytes + kUnitBytes - 1) / kUnitBytes;
    // The host does not know how many pages move: enough CTAs for half of them, the
    // most that can (a page that moves leaves one that stays vacant).
    int64_t work = (static_cast<int64_t>(num_pages) / 2 * upp + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const int64_t rows = (entries + num_pages + kCopyThreads - 1) / kCopyThreads;
    if (work < rows) work = rows;
    if (work > static_cast<int64_t>(sms) * kCopyCtasPerSm) work = static_cast<int64_t>(sms) * kCopyCtasPerSm;
    if (work < 1) work = 1;
    if (num_pages <= 32 * kPlanWords) {
        if (!launch(mla_compact_plan_kernel, 1, kPlanThreads, stream, a)) return MLA_ECUDA;
    } else {
        if (!launch(mla_compact_count_kernel, chunks, kScanThreads, stream, a)) return MLA_ECUDA;
        if (!launch(mla_compact_rank_kernel, chunks, kScanThreads, stream, a, chunks)) return MLA_ECUDA;
    }
    return launch(mla_compact_move_kernel, work, kCopyThreads, stream, a, upp) ? MLA_OK : MLA_ECUDA;
}
