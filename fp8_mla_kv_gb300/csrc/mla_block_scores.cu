// mla_block_scores: how much each token's heads want each complete block before the token's own,
//   score[t, b] = sum over heads h of softmax over b of (sm_scale q[t, h] . K_b),
// K_b the mean keys of mla_block_keys.
#include <climits>
#include <cmath>

#include "mla_seq.cuh"

namespace {

using namespace mla;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct ScoreArgs {
    Batch b;
    const __nv_bfloat16* q;
    const __nv_bfloat16* keys;
    float* scores;
    int H, d_qk, num_keys;
    float scale_log2;
};

// A CTA takes a token, a warp every eighth block: products first for the heads' maxima and sums, then again for the scores.
__global__ void __launch_bounds__(kThreads)
block_scores_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) __nv_bfloat16 sq[];    // [H][d_qk]
    __shared__ float m_s[kWarps][128], l_s[kWarps][128], off_s[128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (t == 0) check_lengths(a.b);
    const int s = sequence_at(a.b, t, lane);
    if (s < 0) return;
    const Sequence q = sequence_of(a.b, s);
    const int pos = position_of(a.b, q, t - q.start);
    const int n = pos < 0 ? 0 : pos / a.b.page_size;
    for (int i = threadIdx.x; i < a.H * a.d_qk; i += kThreads)
        sq[i] = a.q[static_cast<int64_t>(t) * a.H * a.d_qk + i];
    for (int i = threadIdx.x; i < kWarps * 128; i += kThreads) {
        m_s[i / 128][i % 128] = -INFINITY;
        l_s[i / 128][i % 128] = 0.0f;
    }
    __syncthreads();
    const int32_t* bt = a.b.block_table + static_cast<int64_t>(s) * a.b.max_pages;
    float* row = a.scores + static_cast<int64_t>(t) * a.b.max_pages;
    for (int pass = 0; pass < 2; ++pass) {
        for (int blk = warp; blk < n; blk += kWarps) {
            const int phys = __ldg(bt + blk);
            if (phys < 0 || phys >= a.num_keys) {
                if (lane == 0 && pass == 1) {
                    row[blk] = -INFINITY;
                    if (phys >= 0) atomicOr(a.b.err, MLA_ERR_PAGE_RANGE);
                }
                continue;
            }
            float k[18];
#pragma unroll
            for (int i = 0; i < 18; ++i)
                k[i] = 32 * i + lane < a.d_qk ? __bfloat162float(a.keys[static_cast<int64_t>(phys) * a.d_qk + 32 * i + lane]) : 0.0f;
            float sum = 0.0f;
            for (int h = 0; h < a.H; ++h) {
                float x = 0.0f;
#pragma unroll
                for (int i = 0; i < 18; ++i)
                    if (32 * i + lane < a.d_qk) x = fmaf(k[i], __bfloat162float(sq[h * a.d_qk + 32 * i + lane]), x);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                x *= a.scale_log2;
                if (pass == 0) {
                    if (lane == 0) {
                        const float m = m_s[warp][h], now = fmaxf(m, x);
                        l_s[warp][h] = l_s[warp][h] * exp2f(m - now) + exp2f(x - now);
                        m_s[warp][h] = now;
                    }
                } else {
                    sum += exp2f(x - off_s[h]);
                }
            }
            if (pass == 1 && lane == 0) row[blk] = sum;
        }
        __syncthreads();
        if (pass == 0) {
            for (int h = threadIdx.x; h < a.H; h += kThreads) {
                float m = -INFINITY, l = 0.0f;
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, m_s[w][h]);
                for (int w = 0; w < kWarps; ++w) l += m_s[w][h] == -INFINITY ? 0.0f : l_s[w][h] * exp2f(m_s[w][h] - m);
                off_s[h] = m + log2f(l);
            }
            __syncthreads();
        }
    }
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

extern "C" int mla_block_scores(const void* q_bf16, int T, int H, int d_qk, const void* keys_bf16, int num_keys,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int n_seq,
                                int max_pages, int page_size, float sm_scale, float* scores, void* stream) {
    Batch b = {q_start, kv_len, block_table, n_seq, max_pages, page_size, T, nullptr};
    if (num_keys < 0 || !std::isfinite(sm_scale)) return MLA_EINVAL;
    if ((d_qk != kLatent && d_qk != kLatent + kRope) || H < 1 || H > 128) return MLA_EUNSUPPORTED;
    const int rc = mla_host::check_batch(b);
    if (rc != MLA_OK || T == 0 || n_seq == 0 || max_pages == 0) return rc;
    if (static_cast<int64_t>(T) * H > INT_MAX / 4) return MLA_EUNSUPPORTED;
    if (q_bf16 == nullptr || scores == nullptr || (keys_bf16 == nullptr && num_keys > 0) || off(q_bf16, 16) ||
        off(keys_bf16, 16) || off(scores, 4))
        return MLA_EINVAL;
    b.err = mla_host::device_error_word();
    if (b.err == nullptr) return MLA_ECUDA;
    const ScoreArgs a = {b, static_cast<const __nv_bfloat16*>(q_bf16), static_cast<const __nv_bfloat16*>(keys_bf16), scores,
                         H, d_qk, num_keys, sm_scale * kLog2e};
    constexpr int kMostSmem = 128 * (kLatent + kRope) * 2;
    if (!mla_host::max_dynamic_smem(reinterpret_cast<const void*>(block_scores_kernel), kMostSmem)) return MLA_ECUDA;
    return mla_host::launch_pdl(block_scores_kernel, T, kThreads, H * d_qk * 2, stream, a) ? MLA_OK : MLA_ECUDA;
}
