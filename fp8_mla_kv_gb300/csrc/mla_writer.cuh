// Row quantisation shared by the cache writers: one warp turns one BF16 latent row
// into 512 E4M3 codes and four fp32 tile scales (lane l owns values 16l .. 16l+15).
#pragma once

#include "mla_device.cuh"

namespace mla {

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

// x0 / s and x1 / s rounded to nearest even, by the residual-corrected
// reciprocal product of div_by_scale computed on both values at once with the
// packed fp32 pipe (the same IEEE operations per value: q0 = RN(x*y), r = x -
// q0*s exactly, q = RN(q0 + r*y)), then round-to-nearest-even E4M3 with
// saturation.
__device__ __forceinline__ uint32_t quant2_fast(float x0, float x1, uint64_t y2, uint64_t ns2) {
    const uint64_t x = f32x2(x0, x1);
    uint64_t q0, r, q;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q0) : "l"(x), "l"(y2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q0), "l"(ns2), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(y2), "l"(q0));
    float q_lo, q_hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q_lo), "=f"(q_hi) : "l"(q));
    const float2 v = make_float2(copysignf(q_lo, x0), copysignf(q_hi, x1));   // a zero quotient keeps x's sign
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3));
}

// The same with the IEEE division, for a tile whose scale is outside the range
// where the residual above is exact.
__device__ __forceinline__ uint32_t quant2_ieee(float x0, float x1, float scale) {
    const float2 v = make_float2(__fdiv_rn(x0, scale), __fdiv_rn(x1, scale));
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3));
}

// Inputs of one row in flight: lane l's 32 latent bytes and, for lanes 0..7, 16
// bytes of the RoPE tail.
struct RowIn {
    uint4 a, b, tail;
};

__device__ __forceinline__ RowIn load_row(const uint16_t* __restrict__ latent, const uint16_t* __restrict__ rope,
                                          int64_t r, int lane) {
    RowIn in;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(latent + r * kLatent) + 32 * lane;
    in.a = ld_nc_v4(src);
    in.b = ld_nc_v4(src + 16);
    in.tail = make_uint4(0u, 0u, 0u, 0u);
    if (rope != nullptr && lane < 8)
        in.tail = ld_nc_v4(reinterpret_cast<const uint8_t*>(rope + r * kRope) + 16 * lane);
    return in;
}

// Tile amax, scale, E4M3 codes and the row's stores (the whole warp); the tail of a
// 656-byte row too unless the caller stores it itself.
template <bool kTail>
__device__ __forceinline__ void quantise_store(const RowIn& in, uint8_t* row, int64_t row_bytes, int lane) {
    const uint32_t w[8] = {in.a.x, in.a.y, in.a.z, in.a.w, in.b.x, in.b.y, in.b.z, in.b.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
    }
    float amax = 0.0f;                                   // fmaxf ignores NaN
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
    const float scale = (amax > 0.0f) ? __fdiv_rn(amax, MLA_FP8_MAX) : 1.0f;
    const bool fast = scale >= kDivFastMin && scale <= kDivFastMax;   // false only for extreme tiles
    const float rcp = __frcp_rn(scale);

    // One branch for the whole warp: every tile of the row in the fast range
    // (the rule), or the IEEE division on the tiles that are not.
    uint32_t qv[4];
    if (__all_sync(0xffffffffu, fast)) {
        const uint64_t y2 = f32x2(rcp, rcp), ns2 = f32x2(-scale, -scale);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            qv[k] = quant2_fast(v[4 * k], v[4 * k + 1], y2, ns2) |
                    (quant2_fast(v[4 * k + 2], v[4 * k + 3], y2, ns2) << 16);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            qv[k] = fast ? (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                                make_float2(div_by_scale(v[4 * k], scale, rcp), div_by_scale(v[4 * k + 1], scale, rcp)),
                                __NV_SATFINITE, __NV_E4M3)) |
                            (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                                make_float2(div_by_scale(v[4 * k + 2], scale, rcp), div_by_scale(v[4 * k + 3], scale, rcp)),
                                __NV_SATFINITE, __NV_E4M3)) << 16))
                         : (quant2_ieee(v[4 * k], v[4 * k + 1], scale) |
                            (quant2_ieee(v[4 * k + 2], v[4 * k + 3], scale) << 16));
    }

    st_v4(row + 16 * lane, make_uint4(qv[0], qv[1], qv[2], qv[3]));
    const float s0 = __shfl_sync(0xffffffffu, scale, 0);
    const float s1 = __shfl_sync(0xffffffffu, scale, 8);
    const float s2 = __shfl_sync(0xffffffffu, scale, 16);
    const float s3 = __shfl_sync(0xffffffffu, scale, 24);
    if (lane < 8) {
        if (kTail && row_bytes == kRowBytes) st_v4(row + kTailOff + 16 * lane, in.tail);
    } else if (lane == 8) {
        st_v4(row + kScaleOff, make_uint4(__float_as_uint(s0), __float_as_uint(s1),
                                          __float_as_uint(s2), __float_as_uint(s3)));
    }
}

// Whether a row with this slot is written; an out-of-range slot sets the error
// word (lane 0) and is dropped like the reserved slot and negative slots.
__device__ __forceinline__ bool keep_slot(int64_t slot, int64_t num_slots, int64_t reserved_slot, int* err,
                                          int lane) {
    if (slot == reserved_slot || slot < 0) return false;
    if (slot >= num_slots) {
        if (lane == 0) atomicOr(err, MLA_ERR_WRITE_SLOT_RANGE);
        return false;
    }
    return true;
}

}  // namespace mla
