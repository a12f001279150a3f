// mla_rope and mla_rope_kv_write: rotary positions with several axes, alone on any
// strided [rows, heads, 64] view, or fused with the cache write.
//
// Mathematics: pair i of a row at position p (of the axis that pair belongs to) turns
// by p * inv_freq[i] radians. Only the fraction of a turn matters, so the host gives
// each pair its turns per position as a 64-bit binary fraction F = frac(inv_freq /
// 2 pi) * 2^64 and the kernel takes p * F modulo 2^64: one integer product, exact for
// every 32-bit position, negative ones too, where an fp32 angle at position 10^6 would
// be off by 0.03 rad. Its top 32 bits as a signed number of half turns go to
// sincospif, so cos and sin are good to fp32 rounding. Products and sums of the turn
// are fp32, rounded to BF16 once.
//
// Work: a warp takes one unit. A rotation unit is up to kHeadsPerUnit heads of one
// row: lane i computes the cos and sin of pair i, four lanes hold a head (16 values =
// 8 pairs each, two 16-byte loads), so the eight pairs of a lane come by shuffle once
// and serve all the heads of the unit. A write unit is one cache row: the writer's
// quantiser plus the row's own pair in each lane. What bounds it is bytes; the number
// of heads per unit trades the angle work (about 60 instructions a unit) against
// parallelism of small batches. Back to back in a graph: 67 rows of 128 heads 2.4 us, 1,024 of
// 16 heads on three axes 4.1 us (a launch), 8,192 of 64 heads, a quarter of them not kept, 28.2 us:
// 145 MB at 5.2 TB/s, 0.76 of the measured copy rate; the 128-byte pieces of q, one per
// head, are what a plain copy has not.
#include <cmath>

#include "mla_writer.cuh"

namespace {

using namespace mla;

constexpr int kRotThreads = 128;      // 4 warps
constexpr int kRotWarpsPerSm = 32;
constexpr int kHeadsPerPass = 8;      // heads a warp has in its lanes at once
constexpr int kPasses = 2;            // passes in flight (8,192 rows: 1 30.2 us, 2 28.9, 4 35.1; 1,024: 3.9, 4.1, 5.3)
constexpr int kUnitsPerWarp = 6;      // 8,192 rows of 64 heads: 1 29.6 us, 3 29.0, 6 28.2

struct RopeParams {
    uint64_t turn[32];                // fraction of a turn per position, times 2^64
    float scale;                      // of cos and sin
    uint8_t axis[32];
    int interleaved;
};

struct RotArgs {
    const uint16_t* x;                // nullptr: no rotation units
    uint16_t* y;
    int64_t x_row, x_head, y_row, y_head;   // strides in values
    const int32_t* pos;
    int64_t pos_stride;               // between axes
    int64_t rows;
    int heads;
    int parts;                        // rotation units per row
    int heads_per_unit;               // a multiple of kHeadsPerPass
};

struct WriteArgs {
    uint8_t* cache;
    int64_t num_slots, row_bytes, reserved_slot;
    const int64_t* slot_idx;
    const uint16_t* latent;
    const uint16_t* k_pe;
    int* err;
};

// cos and sin of this lane's pair at row r.
__device__ __forceinline__ float2 lane_turn(const RopeParams& p, const int32_t* pos, int64_t pos_stride, int64_t r,
                                            int lane) {
    const int64_t at = __ldg(pos + static_cast<int64_t>(p.axis[lane]) * pos_stride + r);
    const uint64_t turns = static_cast<uint64_t>(at) * p.turn[lane];
    const float half = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;   // half turns, [-1, 1]
    float s, c;
    sincospif(half, &s, &c);
    return make_float2(c * p.scale, s * p.scale);
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Eight pairs in two 16-byte pieces. Interleaved: pieces hold pairs (2 values each)
// in order; halves: lo holds the first values, hi the second values of the pairs.
template <bool kInter>
__device__ __forceinline__ void turn8(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8]) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t u = word(lo, k), v = word(hi, k);
        if (kInter) {
            const float x0 = bf16lo(u), y0 = bf16hi(u), x1 = bf16lo(v), y1 = bf16hi(v);
            a[k] = pack_bf16x2(x0 * c[k] - y0 * s[k], x0 * s[k] + y0 * c[k]);
            b[k] = pack_bf16x2(x1 * c[k + 4] - y1 * s[k + 4], x1 * s[k + 4] + y1 * c[k + 4]);
        } else {
            const float x0 = bf16lo(u), x1 = bf16hi(u), y0 = bf16lo(v), y1 = bf16hi(v);
            a[k] = pack_bf16x2(x0 * c[2 * k] - y0 * s[2 * k], x1 * c[2 * k + 1] - y1 * s[2 * k + 1]);
            b[k] = pack_bf16x2(x0 * s[2 * k] + y0 * c[2 * k], x1 * s[2 * k + 1] + y1 * c[2 * k + 1]);
        }
    }
    lo = make_uint4(a[0], a[1], a[2], a[3]);
    hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// One rotation unit: heads [h0, h1) of row r.
template <bool kInter>
__device__ __forceinline__ void rotate_heads(const RotArgs& a, const RopeParams& p, int64_t r, int h0, int h1,
                                             int lane) {
    const int k = lane & 3;
    // halves: values 8k .. 8k+7 and 32+8k ..; interleaved: values 16k .. 16k+15
    const int off_lo = kInter ? 16 * k : 8 * k;
    const int off_hi = kInter ? 16 * k + 8 : 32 + 8 * k;
    const uint16_t* xr = a.x + r * a.x_row;
    uint16_t* yr = a.y + r * a.y_row;
    uint4 lo[kPasses], hi[kPasses];
    // the first passes' values are on their way while the angles are computed
#pragma unroll
    for (int q = 0; q < kPasses; ++q) {
        const int h = h0 + q * kHeadsPerPass + (lane >> 2);
        if (h < h1) {
            lo[q] = *reinterpret_cast<const uint4*>(xr + h * a.x_head + off_lo);
            hi[q] = *reinterpret_cast<const uint4*>(xr + h * a.x_head + off_hi);
        }
    }
    const float2 cs = lane_turn(p, a.pos, a.pos_stride, r, lane);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = __shfl_sync(0xffffffffu, cs.x, 8 * k + i);
        s[i] = __shfl_sync(0xffffffffu, cs.y, 8 * k + i);
    }
    for (int hb = h0; hb < h1; hb += kPasses * kHeadsPerPass) {
#pragma unroll
        for (int q = 0; q < kPasses; ++q) {
            const int h = hb + q * kHeadsPerPass + (lane >> 2);
            const int next = h + kPasses * kHeadsPerPass;
            if (h >= h1) continue;
            uint4 u = lo[q], v = hi[q];
            if (next < h1) {
                lo[q] = *reinterpret_cast<const uint4*>(xr + next * a.x_head + off_lo);
                hi[q] = *reinterpret_cast<const uint4*>(xr + next * a.x_head + off_hi);
            }
            turn8<kInter>(u, v, c, s);
            st_v4(yr + h * a.y_head + off_lo, u);
            st_v4(yr + h * a.y_head + off_hi, v);
        }
    }
}

// One write unit: cache row of input row r, its rotary tail turned.
template <bool kInter>
__device__ __forceinline__ void write_row(const WriteArgs& w, const RotArgs& a, const RopeParams& p, int64_t r,
                                          int lane) {
    const int64_t slot = __ldg(w.slot_idx + r);
    if (!keep_slot(slot, w.num_slots, w.reserved_slot, w.err, lane)) return;   // none of its inputs is read
    const RowIn in = load_row(w.latent, nullptr, r, lane);
    const uint16_t* k = w.k_pe + r * kRope;
    float x, y;
    if (kInter) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(k + 2 * lane);
        x = bf16lo(v);
        y = bf16hi(v);
    } else {
        x = __uint_as_float(static_cast<uint32_t>(k[lane]) << 16);
        y = __uint_as_float(static_cast<uint32_t>(k[lane + 32]) << 16);
    }
    const float2 cs = lane_turn(p, a.pos, a.pos_stride, r, lane);
    const float u = x * cs.x - y * cs.y, v = x * cs.y + y * cs.x;
    uint8_t* row = w.cache + slot * w.row_bytes;
    if (kInter) {
        *reinterpret_cast<uint32_t*>(row + kTailOff + 4 * lane) = pack_bf16x2(u, v);
    } else {
        const uint32_t both = pack_bf16x2(u, v);
        *reinterpret_cast<uint16_t*>(row + kTailOff + 2 * lane) = static_cast<uint16_t>(both);
        *reinterpret_cast<uint16_t*>(row + kTailOff + 64 + 2 * lane) = static_cast<uint16_t>(both >> 16);
    }
    quantise_store<false>(in, row, w.row_bytes, lane);
}

// Units: the write units first (rows of them, when w.cache is given), then the
// rotation units, row by row.
template <bool kInter>
__global__ void __launch_bounds__(kRotThreads, kRotWarpsPerSm * 32 / kRotThreads)
mla_rope_kernel(const __grid_constant__ RopeParams p, const RotArgs a, const WriteArgs w) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t writes = w.cache != nullptr ? a.rows : 0;
    const int64_t units = writes + (a.x != nullptr ? a.rows * a.parts : 0);
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; u < units; u += nw) {
        if (u < writes) {
            write_row<kInter>(w, a, p, u, lane);
        } else {
            const int64_t r = (u - writes) / a.parts;
            const int h0 = static_cast<int>((u - writes) - r * a.parts) * a.heads_per_unit;
            rotate_heads<kInter>(a, p, r, h0, min(a.heads, h0 + a.heads_per_unit), lane);
        }
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_rope(const mla_rope_t* rope) {
    if (rope == nullptr || rope->n_axes < 1 || rope->n_axes > MLA_ROPE_MAX_AXES || !std::isfinite(rope->scale))
        return MLA_EINVAL;
    for (int i = 0; i < kRope / 2; ++i)
        if (!std::isfinite(rope->inv_freq[i]) || rope->axis[i] >= rope->n_axes) return MLA_EINVAL;
    return MLA_OK;
}

// Axes are apart, or one row of positions that all of them read.
bool axes_ok(int n_axes, int64_t pos_stride, int64_t n_rows) {
    return n_axes == 1 || pos_stride == 0 || pos_stride >= n_rows;
}

// Strided view of rows x heads x 64 values: every 16-byte piece aligned. Strides of a
// single row or head are never used.
bool view_ok(const void* p, int64_t row, int64_t head, int64_t rows, int heads) {
    if (p == nullptr || !aligned(p, 16)) return false;
    if (rows > 1 && (row % 8 != 0)) return false;
    return heads <= 1 || head % 8 == 0;
}

// Whether no two of a view's 64 values lie on one another: i outer strides and j inner ones are never
// within 64 values of each other. A view that is written has to be so (in place, values that several
// heads share would be turned again and again); one that is only read need not.
bool apart(int64_t row, int64_t head, int64_t rows, int64_t heads) {
    const uint64_t r = row < 0 ? 0 - static_cast<uint64_t>(row) : row, h = head < 0 ? 0 - static_cast<uint64_t>(head) : head;
    if ((rows > 1 && r < kRope) || (heads > 1 && h < kRope)) return false;
    if (rows <= 1 || heads <= 1) return true;
    const unsigned __int128 outer = r > h ? r : h, inner = r > h ? h : r, reach = inner * ((r > h ? heads : rows) - 1) + kRope;
    const int64_t n_outer = r > h ? rows : heads;
    for (int64_t i = 1; i < n_outer && outer * i < reach; ++i) {   // (rows or heads behind one another: not once)
        const unsigned __int128 off = outer * i % inner;
        if (off < kRope || inner - off < kRope) return false;
    }
    return true;
}

RopeParams make_params(const mla_rope_t& rope) {
    RopeParams p;
    for (int i = 0; i < kRope / 2; ++i) {
        double f = std::fabs(rope.inv_freq[i]) / 6.283185307179586476925286766559;
        f -= std::floor(f);                                   // [0, 1)
        const uint64_t turn = static_cast<uint64_t>(std::ldexp(f, 64));
        // the other way round: the negative modulo 2^64 exactly (1 - f would be rounded to 2^-54 of a turn)
        p.turn[i] = (rope.inv_freq[i] < 0) != (rope.inverse != 0) ? 0 - turn : turn;
        p.axis[i] = rope.axis[i];
    }
    p.scale = rope.scale;
    p.interleaved = rope.interleaved != 0;
    return p;
}

int launch_rope(const mla_rope_t* rope, RotArgs a, const WriteArgs& w, void* stream) {
    const int sms = mla_host::sm_count();
    if (sms <= 0) return MLA_ECUDA;
    // Heads per unit: as many of a row's as leave every warp kUnitsPerWarp units, so that the last
    // round of them is short, and a small batch's rows spread over several warps.
    a.heads_per_unit = (a.heads + kHeadsPerPass - 1) / kHeadsPerPass * kHeadsPerPass;
    const int64_t want = static_cast<int64_t>(sms) * kRotWarpsPerSm;
    while (a.heads_per_unit > kHeadsPerPass &&
           a.rows * ((a.heads + a.heads_per_unit - 1) / a.heads_per_unit) < want * kUnitsPerWarp)
        a.heads_per_unit = (a.heads_per_unit / 2 + kHeadsPerPass - 1) / kHeadsPerPass * kHeadsPerPass;
    a.parts = a.heads > 0 ? (a.heads + a.heads_per_unit - 1) / a.heads_per_unit : 0;
    const int64_t units = (w.cache != nullptr ? a.rows : 0) + (a.x != nullptr ? a.rows * a.parts : 0);
    if (units == 0) return MLA_OK;
    const int64_t warps = kRotThreads / 32;
    int64_t blocks = (units + warps - 1) / warps;
    if (blocks > want / warps) blocks = want / warps;
    const RopeParams p = make_params(*rope);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kRotThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t lr = p.interleaved ? cudaLaunchKernelEx(&cfg, mla_rope_kernel<true>, p, a, w)
                                         : cudaLaunchKernelEx(&cfg, mla_rope_kernel<false>, p, a, w);
    return (lr == cudaSuccess && cudaGetLastError() == cudaSuccess) ? MLA_OK : MLA_ECUDA;
}

}  // namespace

extern "C" int mla_rope(const void* x_bf16, int64_t x_row, int64_t x_head, void* y_bf16, int64_t y_row,
                        int64_t y_head, int64_t n_rows, int n_heads, const int32_t* pos, int64_t pos_stride,
                        const mla_rope_t* rope, void* stream) {
    if (n_rows < 0 || n_heads < 0 || pos_stride < 0) return MLA_EINVAL;
    if (const int rc = check_rope(rope)) return rc;
    if (n_rows == 0 || n_heads == 0) return MLA_OK;
    if (!view_ok(x_bf16, x_row, x_head, n_rows, n_heads) || !view_ok(y_bf16, y_row, y_head, n_rows, n_heads) ||
        !apart(y_row, y_head, n_rows, n_heads) || pos == nullptr || !aligned(pos, 4) || !axes_ok(rope->n_axes, pos_stride, n_rows))
        return MLA_EINVAL;
    RotArgs a = {static_cast<const uint16_t*>(x_bf16), static_cast<uint16_t*>(y_bf16), x_row, x_head, y_row, y_head,
                 pos, pos_stride, n_rows, n_heads, 0, 0};
    const WriteArgs none = {};
    return launch_rope(rope, a, none, stream);
}

extern "C" int mla_rope_kv_write(mla_kv_cache_t kv, const int64_t* slot_idx, const void* latent_bf16,
                                 const void* k_pe_bf16, int64_t n_rows, int64_t reserved_slot, const int32_t* pos,
                                 int64_t pos_stride, const mla_rope_t* rope, const void* q_bf16, int64_t q_row,
                                 int64_t q_head, void* q_out_bf16, int64_t q_out_row, int64_t q_out_head, int n_heads,
                                 void* stream) {
    if (n_rows < 0 || n_heads < 0 || pos_stride < 0 || kv.num_slots < 0) return MLA_EINVAL;
    if (kv.row_bytes != MLA_ROW_BYTES) return MLA_EINVAL;                 // a 528-byte row has no rotary tail
    if (const int rc = check_rope(rope)) return rc;
    if (n_rows == 0) return MLA_OK;
    if (kv.data == nullptr || slot_idx == nullptr || latent_bf16 == nullptr || k_pe_bf16 == nullptr || pos == nullptr)
        return MLA_EINVAL;
    if (!aligned(kv.data, 16) || !aligned(latent_bf16, 16) || !aligned(k_pe_bf16, 4) || !aligned(slot_idx, 8) ||
        !aligned(pos, 4) || !axes_ok(rope->n_axes, pos_stride, n_rows))
        return MLA_EINVAL;
    if ((q_bf16 == nullptr) != (q_out_bf16 == nullptr)) return MLA_EINVAL;
    if (q_bf16 != nullptr && n_heads > 0 &&
        (!view_ok(q_bf16, q_row, q_head, n_rows, n_heads) || !view_ok(q_out_bf16, q_out_row, q_out_head, n_rows, n_heads) ||
         !apart(q_out_row, q_out_head, n_rows, n_heads)))
        return MLA_EINVAL;
    int* err = mla_host::device_error_word();
    if (err == nullptr) return MLA_ECUDA;
    const bool rot = q_bf16 != nullptr && n_heads > 0;
    RotArgs a = {rot ? static_cast<const uint16_t*>(q_bf16) : nullptr, static_cast<uint16_t*>(q_out_bf16), q_row, q_head,
                 q_out_row, q_out_head, pos, pos_stride, n_rows, rot ? n_heads : 0, 0, 0};
    const WriteArgs w = {static_cast<uint8_t*>(kv.data), kv.num_slots, kv.row_bytes, reserved_slot, slot_idx,
                         static_cast<const uint16_t*>(latent_bf16), static_cast<const uint16_t*>(k_pe_bf16), err};
    return launch_rope(rope, a, w, stream);
}
