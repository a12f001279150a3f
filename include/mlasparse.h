/*
 * libmlasparse - FP8 MLA KV cache writer and sparse top-k MLA decode on one
 * GB300 GPU (sm_103a). Plain C ABI: device pointers, sizes, a CUDA stream.
 *
 * Row layout (vLLM PR #55277 "Support NoPE sparse MLA (GLM-5.3-Flash) on the
 * FlashInfer SM120 backend", Purpose item 1): every cache slot is one 656-byte
 * row
 *     bytes [  0, 512)  512 E4M3 latent values, value i at byte i, in four
 *                       tiles of 128 values (tile t = bytes 128t .. 128t+127)
 *     bytes [512, 528)  four little-endian fp32 tile scales, tile t at 512 + 4t
 *     bytes [528, 656)  64 bf16 RoPE values, or 128 zero bytes for NoPE rows
 * and a stored value decodes as e4m3(byte) * scale[tile].
 *
 * Slot 0 is reserved (sglang PR #47013 "zero-RoPE writer skips reserved slot 0",
 * Summary and Motivation): the allocators never hand it out, padding rows aim
 * at it, and no write may land there.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers on the current CUDA device, owned
 *     by the caller; the library never allocates, frees or retains them.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream). Calls are asynchronous on that stream.
 *   - The return value is MLA_OK (0) or a negative MLA_E* code; arguments are
 *     validated on the host before any launch and nothing is launched on error.
 *     No C++ exception crosses this boundary.
 *   - Range violations found on the device (a slot or a top-k index past the
 *     cache) never trap: the row or entry is dropped and a bit is set in the
 *     library's device error word, read with mla_get_error().
 */
#ifndef MLASPARSE_H
#define MLASPARSE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- row layout (vLLM PR #55277, Purpose item 1) ---- */
#define MLA_ROW_BYTES      656
#define MLA_LATENT_DIM     512
#define MLA_TILE_VALUES    128
#define MLA_NUM_TILES      4
#define MLA_SCALE_OFFSET   512
#define MLA_TAIL_OFFSET    528
#define MLA_ROPE_DIM       64
#define MLA_FP8_MAX        448.0f   /* largest finite E4M3 value */
/* The canonical NoPE row of flashinfer#5075 (sglang PR #39288, "Relation to
 * other changes"): the 656-byte row without its 128-byte tail. */
#define MLA_ROW_BYTES_NOPE 528

/* ---- return codes ---- */
#define MLA_OK             0
#define MLA_EINVAL        (-1)   /* null pointer, negative size, misaligned pointer, bad layout */
#define MLA_EUNSUPPORTED  (-2)   /* d_qk not in {512, 576}, H outside [1, 128] */
#define MLA_ENOWORKSPACE  (-3)   /* workspace NULL, misaligned, or smaller than the call's *_workspace_bytes() */
#define MLA_ECUDA         (-4)   /* a CUDA runtime call or a kernel launch failed */

/* ---- device error word bits (mla_get_error) ---- */
#define MLA_ERR_WRITE_SLOT_RANGE   0x1  /* mla_kv_write: slot >= num_slots, row dropped */
#define MLA_ERR_DECODE_INDEX_RANGE 0x2  /* mla_sparse_decode: index >= num_slots, entry absent */
#define MLA_ERR_PIPELINE_TIMEOUT   0x4  /* a kernel's bounded wait on its own copies ran out */
#define MLA_ERR_GATHER_INDEX_RANGE 0x8  /* mla_gather_upconvert: slot >= num_slots, zero row */
#define MLA_ERR_CHUNK_RANGE        0x10 /* mla_chunk_attention, mla_block_*, mla_tree_*: q_start not nondecreasing within [0, T], kv_len past the table, or a tree out of order */
#define MLA_ERR_PAGE_RANGE         0x20 /* mla_page_*, mla_block_keys, mla_block_scores, mla_tree_commit: a page, row or length out of range, dropped */
#define MLA_ERR_PAGE_COUNT         0x40 /* mla_page_free: a page whose count was 0 already */
#define MLA_ERR_POOL_EMPTY         0x80 /* mla_page_fork: no free page left, the entry stays -1 */

/* A cache: `data` is a device array of num_slots rows of row_bytes bytes,
 * 16-byte aligned. row_bytes is MLA_ROW_BYTES (656), or MLA_ROW_BYTES_NOPE
 * (528) for a cache of NoPE rows only: latent and scales at the same offsets,
 * no tail. A 528-byte cache takes only NoPE calls (rope_bf16 NULL, d_qk 512,
 * pe_dim 0); others return MLA_EINVAL or MLA_EUNSUPPORTED. */
typedef struct {
    void*   data;
    int64_t num_slots;
    int64_t row_bytes;
} mla_kv_cache_t;

/*
 * mla_kv_write - per-token FP8 quantise-and-scatter into packed rows.
 *
 * Defined by vLLM PR #55277 (Purpose item 1: the 656-byte row; NoPE rows zero
 * the 128-byte tail; pe_dim must be 64 or 0) and sglang PR #47013 (Summary,
 * Motivation, Modifications: rows aimed at the reserved slot are dropped; BF16
 * NaNs are kept by the quantiser, not clamped).
 *
 * For each row r in [0, n_rows) with s = slot_idx[r]:
 *   - s == reserved_slot or s < 0: the row is dropped and none of its inputs is
 *     read (its latent may hold NaN);
 *   - s >= kv.num_slots: the row is dropped and MLA_ERR_WRITE_SLOT_RANGE is set;
 *   - otherwise row s of the cache is overwritten: for each tile t,
 *       scale_t = amax_t / 448 (IEEE fp32 division; 1.0 when amax_t == 0;
 *                 amax ignores NaN),
 *       byte    = e4m3 round-to-nearest-even, saturating to +-448, of x / scale_t
 *                 (IEEE fp32 division; a NaN x gives the NaN code 0x7F),
 *     the four scales go to bytes 512..527, and bytes 528..655 receive rope row r
 *     verbatim, or zeros when rope_bf16 is NULL (a 528-byte row has no tail).
 * No other byte of the cache is touched.
 *
 * Arguments:
 *   kv            cache (device, 16-byte aligned, row_bytes 656, or 528 with
 *                 rope_bf16 NULL)
 *   slot_idx      int64 [n_rows], device
 *   latent_bf16   bf16 [n_rows, 512] row-major, device, 16-byte aligned
 *   rope_bf16     bf16 [n_rows, 64] row-major, device, 16-byte aligned; or NULL
 *                 for pe_dim = 0 (NoPE)
 *   n_rows        >= 0 (0 launches nothing)
 *   reserved_slot the slot writes must never land in (0 in every caller)
 * Precondition: no two rows of one call name the same non-reserved slot (which
 * of them would land is unspecified).
 * Ordering: the writer is launched with programmatic stream serialization: its
 * CTAs may become resident while the previous kernel on the stream finishes, and
 * they read nothing (slot indices, inputs, cache) until that kernel and its
 * memory are complete (griddepcontrol.wait). It also lets the next kernel on the
 * stream begin launching while it runs; only a kernel launched with programmatic
 * stream serialization can start early, and such a kernel must wait for its
 * predecessor before reading the cache, as mla_sparse_decode and the writer
 * itself do. Ordinary launches and copies are ordered as usual.
 * Returns MLA_OK, MLA_EINVAL or MLA_ECUDA.
 */
int mla_kv_write(mla_kv_cache_t kv, const int64_t* slot_idx, const void* latent_bf16,
                 const void* rope_bf16, int64_t n_rows, int64_t reserved_slot, void* stream);

/*
 * mla_sparse_decode_workspace_bytes - bytes of device workspace that
 * mla_sparse_decode needs for these sizes on the CURRENT device (the split of
 * the top-k list across CTAs depends on the device's SM count). 0 means no
 * workspace is needed. Returns 0 for invalid sizes as well.
 */
size_t mla_sparse_decode_workspace_bytes(int T, int H, int W);

/*
 * mla_sparse_decode - sparse top-k MLA decode over the packed FP8 cache.
 *
 * Sparse top-k MLA attention over the listed rows, written out below, with the
 * masking rules of sglang PR #47013 (Motivation: unused top-k entries must not
 * reach the result, even when slot 0 holds NaN), sglang PR #39288 ("SM120
 * sparse MLA: zero-initialise the page-split scratch", Root cause: a -1
 * candidate contributes nothing and must not gather slot 0), and vLLM PR #55277 (Purpose item 2: the index buffer
 * width W is a capacity; the active entries are bounded by the -1 padding;
 * Purpose item 1 and "Relation to #53969": NoPE decode reads no tail).
 *
 * For each token t < T and head h < H, with J = { j : 0 < topk_idx[t,j] <
 * kv.num_slots } (-1 or any negative, the reserved slot 0, and out-of-range
 * indices are absent: never dereferenced, contributing nothing; an index >=
 * num_slots also sets MLA_ERR_DECODE_INDEX_RANGE):
 *   s_j       = sm_scale * ( q[t,h,0:512] . K_j  +  [d_qk == 576] q[t,h,512:576] . rope_j )
 *   K_j[d]    = e4m3(byte_d of row) * scale[d / 128]      (V_j = K_j)
 *   out[t,h]  = sum_j softmax(s)_j V_j                     (bf16)
 *   lse[t,h]  = ln sum_j exp(s_j)                          (fp32, natural log)
 * An empty J gives out = 0 and lse = -inf; a row of J holding a NaN code gives
 * NaN out and lse for that token, whether or not its list is split. The result
 * does not depend on the order of the entries nor on what slot 0 holds
 * (bit-identical output).
 *
 * Arguments:
 *   q_bf16     bf16 [T, H, d_qk] row-major, device, 16-byte aligned
 *   T, H       tokens (>= 0; 0 launches nothing) and heads (1..128)
 *   d_qk       576 (512 latent + 64 RoPE) or 512 (NoPE: the row tail is not read)
 *   kv         the cache (16-byte aligned; row_bytes 656, or 528 with d_qk 512)
 *   topk_idx   int32 [T, W] row-major, device; W >= 0
 *   sm_scale   softmax scale applied to q . k (finite)
 *   out_bf16   bf16 [T, H, 512] row-major, device, 16-byte aligned
 *   lse        fp32 [T, H], device
 *   workspace  device scratch of at least mla_sparse_decode_workspace_bytes(T,H,W)
 *              bytes, 16-byte aligned (may be NULL when that is 0). Its contents
 *              on entry do not matter; it is clobbered.
 * The decode kernel is launched with programmatic stream serialization and waits
 * for the previous kernel on the stream, and its memory, before it reads any
 * input; behind mla_kv_write its launch overlaps the writer's last CTAs.
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED, MLA_ENOWORKSPACE or MLA_ECUDA.
 */
int mla_sparse_decode(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv,
                      const int32_t* topk_idx, int W, float sm_scale, void* out_bf16,
                      float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * mla_sparse_decode_paged - mla_sparse_decode with the top-k list given as
 * sequence positions and a block table (vLLM PR #55277, Purpose item 2: the
 * sparse attention reads its top-k entries through block tables, a page table
 * whose width is a capacity; here the kernel maps each position to a slot).
 *
 * Entry j of token t is position p = topk_pos[t,j] of the token's sequence
 * s = token_seq[t] (every token uses row 0 when token_seq is NULL). It stands for
 * the slot  block_table[s, p / page_size] * page_size + p % page_size,  and
 * the decode is then exactly mla_sparse_decode over those slots. A negative
 * position or a negative (unassigned) block-table entry is absent; a page past
 * max_pages, a sequence outside [0, n_seq) or a slot >= num_slots is absent and
 * sets MLA_ERR_DECODE_INDEX_RANGE. Slot 0 stays absent.
 *
 * Arguments as mla_sparse_decode, plus:
 *   topk_pos     int32 [T, W] positions, device
 *   block_table  int32 [n_seq, max_pages] physical page of each logical page,
 *                device, 4-byte aligned
 *   token_seq    int32 [T] block-table row of each token, device, or NULL
 *   page_size    slots per page (> 0)
 * The workspace is mla_sparse_decode_workspace_bytes(T, H, W).
 */
int mla_sparse_decode_paged(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv,
                            const int32_t* topk_pos, int W, const int32_t* block_table, int n_seq,
                            int max_pages, const int32_t* token_seq, int page_size, float sm_scale,
                            void* out_bf16, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * mla_sparse_prefill - what mla_sparse_decode computes, for batches whose
 * adjacent tokens share most of their top-k rows (a causal prefill: token i's
 * list is nearly a subset of token i+1's).
 *
 * The pages route prefill-sized batches to a dedicated kernel (sglang PR
 * #39288, Motivation: above 64 query rows the prefill kernel runs) and note
 * that the decode kernel also serves prefill today (sglang PR #47013, Speed
 * Tests). Here one CTA takes tokens 2u and 2u+1 with one group of 16 heads; the
 * rows present in both lists are copied and converted once for both tokens.
 * A row present in one list only is computed for that token only, so the result
 * of every token is exactly the decode statement of mla_sparse_decode over its
 * own list (same masking rules, bit-identical whatever slot 0 holds); only the
 * order of accumulation differs from mla_sparse_decode, so the two agree to
 * rounding, not bit for bit. A slot listed twice counts twice, as in the decode.
 *
 * Arguments as mla_sparse_decode, without the workspace; W is at most 2304
 * (MLA_EUNSUPPORTED otherwise). Batches whose adjacent tokens share few rows
 * compute correctly but gain nothing; batches of fewer than about two tokens
 * per SM leave SMs idle (no list is split): use mla_sparse_decode for those.
 * Launched with programmatic stream serialization like the decode.
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED or MLA_ECUDA.
 */
int mla_sparse_prefill(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv,
                       const int32_t* topk_idx, int W, float sm_scale, void* out_bf16, float* lse,
                       void* stream);

/*
 * mla_sparse_prefill_paged - mla_sparse_prefill with the top-k list given as
 * sequence positions and a block table, mapped exactly as in
 * mla_sparse_decode_paged (vLLM PR #55277, Purpose item 2). Arguments as
 * mla_sparse_decode_paged, without the workspace.
 */
int mla_sparse_prefill_paged(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv,
                             const int32_t* topk_pos, int W, const int32_t* block_table, int n_seq,
                             int max_pages, const int32_t* token_seq, int page_size, float sm_scale,
                             void* out_bf16, float* lse, void* stream);

/*
 * mla_gather_upconvert - gather rows of the cache and widen them to BF16
 * (vLLM PR #55277, Changes table: cp_gather_and_upconvert_fp8_kv_cache, the
 * chunked-context path; the NoPE tail is written as exact zeros).
 *
 * For i < n with s = slots[i]:
 *   out[i, d]       = the BF16 value nearest to e4m3(byte_d) * scale[d / 128]
 *                     (the exact product, rounded once, ties to even; a NaN
 *                     code gives 0x7FC0),                         d < 512
 *   out[i, 512 + k] = the RoPE value k of the row's tail (pe_dim 64), or 0
 *                     (pe_dim 0: the tail is not read),           k < 64
 * An absent slot (s <= 0) gives a row of zeros; s >= num_slots as well, and
 * sets MLA_ERR_GATHER_INDEX_RANGE.
 *
 * Arguments:
 *   kv        the cache (16-byte aligned; row_bytes 656, or 528 with pe_dim 0)
 *   slots     int32 [n], device, 4-byte aligned
 *   n         >= 0 (0 launches nothing)
 *   pe_dim    64 or 0
 *   out_bf16  bf16 [n, 576] row-major, device, 16-byte aligned
 * Returns MLA_OK, MLA_EINVAL or MLA_ECUDA.
 */
int mla_gather_upconvert(mla_kv_cache_t kv, const int32_t* slots, int64_t n, int pe_dim,
                         void* out_bf16, void* stream);

/*
 * mla_sparse_decode_noalloc - mla_sparse_decode for callers that cannot
 * allocate device memory where they call it.
 *
 * The pages have no counterpart to this entry point; it exists for users of
 * this library. mla_sparse_decode needs a caller-owned workspace whenever it
 * splits a token's top-k list across CTAs (mla_sparse_decode_workspace_bytes()
 * > 0). A caller that runs inside another framework's memory pool without an
 * allocator handle, or a process that has already committed all the device
 * memory it may use, has no way to provide one. This variant computes exactly
 * what mla_sparse_decode computes, with the same arguments minus the
 * workspace, and uses instead a fixed array of MLA_NOALLOC_SCRATCH_BYTES in the
 * library's own device memory. That array exists on every GPU that loads the
 * library's device code and stays allocated until the process exits. The call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 *
 *   - Sizes whose workspace would exceed MLA_NOALLOC_SCRATCH_BYTES are rejected
 *     with MLA_ENOWORKSPACE before anything is launched.
 *   - All calls on a device share the one array and it keeps what the last call
 *     left there: calls whose work overlaps on the GPU (other streams, or
 *     concurrently replayed graphs) race and produce wrong results. Issue them
 *     on one stream. Nothing in the array needs to start at zero.
 *   - The first call on a device looks up the array's address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 * Returns what mla_sparse_decode returns.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (64u << 20)   /* 64 MiB per device */
int mla_sparse_decode_noalloc(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv,
                              const int32_t* topk_idx, int W, float sm_scale, void* out_bf16,
                              float* lse, void* stream);

/*
 * mla_rope_t - rotary positions with one to four axes (text: one; images and video:
 * time, height, width). A host structure, read during the call.
 *
 * Pair i of the 64 rotary values is (x, y) = values (i, i + 32), or (2i, 2i + 1) when
 * `interleaved`; at position p of axis[i] it becomes
 *     scale * (x cos a - y sin a, x sin a + y cos a),   a = p * inv_freq[i]  (-a: `inverse`)
 * rounded to BF16 once. Sections of pairs per axis may be contiguous, interleaved or
 * anything else: axis[] says it pair by pair. `inverse` undoes the rotation, and
 * is its gradient: dx of y = rope(x) is the inverse rope of dy.
 */
#define MLA_ROPE_MAX_AXES  4
typedef struct {
    double  inv_freq[MLA_ROPE_DIM / 2];   /* radians per unit of position; finite */
    float   scale;                        /* of cos and sin (1 where none is wanted); finite */
    int32_t n_axes;                       /* 1 .. MLA_ROPE_MAX_AXES */
    int32_t interleaved;                  /* pairs (2i, 2i + 1), else (i, i + 32) */
    int32_t inverse;                      /* turn back */
    uint8_t axis[MLA_ROPE_DIM / 2];       /* 0 .. n_axes - 1 */
} mla_rope_t;

/*
 * mla_rope - rotates a strided view of rows x heads x 64 BF16 values.
 *
 * Positions are any int32 (angles are reduced exactly, so far positions lose nothing).
 *   x_bf16, y_bf16  first rotary value of row 0, head 0; 16-byte aligned; y may be x
 *                   with the same strides (in place), otherwise they may not overlap
 *   *_row, *_head   strides in values, multiples of 8 (unused where there is one row
 *                   or one head); x may repeat rows or heads (stride 0), y's do not overlap
 *   n_rows, n_heads >= 0 (0 launches nothing)
 *   pos             int32 [n_axes, n_rows], device; axis k at pos + k * pos_stride
 *                   (with n_axes > 1: pos_stride >= n_rows, or 0 for one row that all axes read)
 * Launched with programmatic stream serialization like the writer.
 * Returns MLA_OK, MLA_EINVAL or MLA_ECUDA.
 */
int mla_rope(const void* x_bf16, int64_t x_row, int64_t x_head, void* y_bf16, int64_t y_row, int64_t y_head,
             int64_t n_rows, int n_heads, const int32_t* pos, int64_t pos_stride, const mla_rope_t* rope,
             void* stream);

/*
 * mla_rope_kv_write - mla_kv_write with the rotary tail turned on the way, and, where
 * q is given, the rotary part of the same rows' queries turned in the same launch.
 *
 * Rows are dropped exactly as in mla_kv_write (reserved slot, negative, past the
 * cache: flagged) with none of their latent, k_pe and position read for the write. The
 * row written is the one mla_kv_write would write with rope_bf16 = mla_rope(k_pe). The
 * queries of every row are turned, those of dropped rows too.
 *
 *   kv, slot_idx, latent_bf16, n_rows, reserved_slot   as mla_kv_write; row_bytes 656
 *   k_pe_bf16     bf16 [n_rows, 64] row-major, device, 4-byte aligned
 *   pos, pos_stride, rope                              as mla_rope
 *   q_bf16, q_out_bf16 and their strides               as x and y of mla_rope, with
 *                 n_heads heads; both NULL: no queries
 * Precondition as mla_kv_write: no two rows of one call name the same non-reserved slot.
 * Returns MLA_OK, MLA_EINVAL or MLA_ECUDA.
 */
int mla_rope_kv_write(mla_kv_cache_t kv, const int64_t* slot_idx, const void* latent_bf16, const void* k_pe_bf16,
                      int64_t n_rows, int64_t reserved_slot, const int32_t* pos, int64_t pos_stride,
                      const mla_rope_t* rope, const void* q_bf16, int64_t q_row, int64_t q_head, void* q_out_bf16,
                      int64_t q_out_row, int64_t q_out_head, int n_heads, void* stream);

/*
 * mla_chunk_attention - dense attention of a chunk of new tokens over the paged cache,
 * for a ragged batch: prefill chunks, single decode tokens, drafts to verify, mixed.
 *
 * Sequence s has the tokens q_start[s] .. q_start[s+1]-1 of q and kv_len[s] positions in
 * the cache, its own new tokens included (write them first). Position p stands for the
 * slot block_table[s, p / page_size] * page_size + p % page_size. Token i of its n
 * attends the positions p <= kv_len[s] - n + i (all kv_len[s] when causal is 0) that
 * are present; a position in a page with a negative table entry, the reserved slot 0,
 * or a slot >= num_slots (flagged MLA_ERR_DECODE_INDEX_RANGE) is absent: never read. Over those
 * positions out and lse are what mla_sparse_decode computes. A token that attends nothing
 * gets out = 0 and lse = -inf. A row that holds a value that is not finite (a NaN code, a NaN
 * or infinite scale or RoPE value) makes out and lse NaN for exactly the tokens that
 * attend it; a query row that holds one gets unspecified values, and no other row does.
 * Scores are sums in fp32 of exact products, except that q values far below their row's
 * largest are rounded: below 2^-24 of it, to 2^-32 of it; in batches of many query rows per
 * sequence below 2^-13 of it, to 2^-21 of it (largest values of 2^-119 and more).
 * Values are held in f16 relative to the largest tile scale (by size; tiles of zeros do not
 * count) among the positions that up to 64 neighbouring (token, head) rows attend, whichever
 * of them: scales of at least 2^-14 of that one to half an f16 step, smaller ones to 2^-25 of it.
 * Tokens outside every sequence keep their out and lse. The result does not
 * depend on what slot 0, absent pages or positions past kv_len hold.
 *
 *   q_bf16       bf16 [T, H, d_qk] row-major, device, 16-byte aligned; d_qk 576 or 512
 *   T, H         tokens (>= 0) and heads (1..128); T * H below 2^29
 *   kv           the cache (row_bytes 656, or 528 with d_qk 512), of less than 2^31 slots
 *   q_start      int32 [n_seq + 1], device, nondecreasing within [0, T]; a sequence for
 *                which it is not is skipped and flagged MLA_ERR_CHUNK_RANGE
 *   kv_len       int32 [n_seq], device; a negative one counts as 0; positions past
 *                max_pages * page_size are absent and flagged MLA_ERR_CHUNK_RANGE
 *   block_table  int32 [n_seq, max_pages], device; max_pages * page_size below 2^31 - 4096
 *                (otherwise MLA_EUNSUPPORTED)
 *   out_bf16     bf16 [T, H, 512], device, 16-byte aligned;  lse  fp32 [T, H], device; neither
 *                overlaps an input
 *   workspace    device scratch of mla_chunk_attention_workspace_bytes(T, H, n_seq) bytes,
 *                16-byte aligned; its contents on entry do not matter. Calls that may
 *                overlap (other streams, graphs replayed at once) need their own.
 * The lengths are read on the device: a captured call serves any lengths within the
 * arrays' sizes. T, H, n_seq and max_pages * page_size decide which of two kernels runs; they agree to
 * rounding, not bit for bit, so a wider table may change an output's last bits. Launched with programmatic stream serialization like the decode.
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED, MLA_ENOWORKSPACE or MLA_ECUDA.
 */
size_t mla_chunk_attention_workspace_bytes(int T, int H, int n_seq);
int mla_chunk_attention(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* block_table, int n_seq, int max_pages, int page_size,
                        int causal, float sm_scale, void* out_bf16, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Block-sparse attention over the paged cache. A block is a page; block b of a sequence is its positions b * page_size ..
 * (b + 1) * page_size - 1, in page block_table[s, b]. Ragged batches as in mla_chunk_attention: sequence s has the
 * tokens q_start[s] .. q_start[s+1]-1 and kv_len[s] positions, its tokens' last, so its token i stands at position
 * kv_len[s] - n + i (one past the table counts as the table's last; flagged MLA_ERR_CHUNK_RANGE), and its own
 * block is the one that holds that position. A q_start that is not nondecreasing within [0, T] is flagged
 * MLA_ERR_CHUNK_RANGE, and which tokens count as being in a sequence is then unspecified. Tokens outside
 * every sequence keep what their outputs hold. Lengths are read on the device, so a captured call serves any. As calls in turn:
 *   mla_rope_kv_write, mla_block_keys, mla_block_scores, mla_block_select, mla_block_attention.
 * All are launched with programmatic stream serialization; with an empty table mla_block_keys, mla_block_scores and
 * mla_block_select write and flag nothing. max_pages * page_size is below 2^31 - 4096 (otherwise MLA_EUNSUPPORTED);
 * q_start, kv_len and block_table as in mla_chunk_attention.
 *
 * mla_block_keys - the mean key of each page that the new tokens completed:
 *   keys[p] = (sum over the rows of page p of [latent (code x scale), rope]) / rows, fp32 sums, rounded to BF16 once.
 * Sequence s completes its blocks floor((kv_len - n) / page_size) .. floor(kv_len / page_size) - 1: with n = kv_len all that are
 * complete (after pages have moved, say). The reserved slot 0 is no row: page 0 has page_size - 1. Blocks without
 * a page are skipped; a page >= num_keys or one that ends past the cache is flagged MLA_ERR_PAGE_RANGE (the first has no
 * key, the second that of its rows in the cache). A row that is not finite makes its key so, in the values concerned.
 *   kv         the cache (row_bytes 656, or 528 with d_qk 512);  d_qk  576 or 512
 *   T          the tokens that q_start counts (its last value at most)
 *   keys_bf16  bf16 [num_keys, d_qk], device, 16-byte aligned; page p's key at row p, other rows are left alone
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED or MLA_ECUDA.
 */
int mla_block_keys(mla_kv_cache_t kv, int d_qk, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                   int n_seq, int max_pages, int page_size, int T, void* keys_bf16, int num_keys, void* stream);

/*
 * mla_block_scores - how much token t wants each complete block before its own:
 *   scores[t, b] = sum over h < H of softmax over b of ( sm_scale * q[t, h] . keys[block_table[s, b]] ),
 * b < floor(position / page_size). Products are exact and summed in fp32, as are the exponentials; no
 * score is written for other blocks. A block without a page, or whose page is >= num_keys (flagged
 * MLA_ERR_PAGE_RANGE), gets -inf and no part in the softmax. A key or query row that is not finite makes the
 * scores unspecified for exactly the tokens that meet it.
 *   q_bf16     bf16 [T, H, d_qk] row-major, device, 16-byte aligned; H 1..128; T * H below 2^29
 *   keys_bf16  bf16 [num_keys, d_qk] row-major, device, 16-byte aligned
 *   scores     fp32 [T, max_pages], device
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED or MLA_ECUDA.
 */
int mla_block_scores(const void* q_bf16, int T, int H, int d_qk, const void* keys_bf16, int num_keys,
                     const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int n_seq, int max_pages,
                     int page_size, float sm_scale, float* scores, void* stream);

/*
 * mla_block_select - the blocks that each token attends: the first `sink` blocks and the last `local` up to its own
 * (its own among them), and of those between the ones with the highest scores, `width` in all. Of equal scores the
 * lower block is taken; a block between whose score is -inf or NaN is not. Row t of `blocks` receives them in
 * ascending order, then -1. A token at a negative position gets -1 throughout.
 *   scores   fp32 [T, columns], device: a column for each block of the table (without columns, as for an empty table,
 *            nothing is launched and `blocks` keeps what it holds)
 *   sink >= 0, local >= 1, sink + local <= width (otherwise MLA_EINVAL)
 *   blocks   int32 [T, width], device
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED or MLA_ECUDA.
 */
int mla_block_select(const float* scores, int T, int columns, const int32_t* q_start, const int32_t* kv_len, int n_seq,
                     int page_size, int sink, int local, int width, int32_t* blocks, void* stream);

/*
 * mla_block_attention - attention of each token over the positions up to its own of the blocks listed for it.
 * out and lse as in mla_chunk_attention over those positions (absent positions, empty rows, rows that are not finite,
 * precision: as there). A negative entry lists nothing; a block listed twice counts once; the order does not matter; a block
 * past the token's own has no position for it. A block >= max_pages is absent and flagged
 * MLA_ERR_DECODE_INDEX_RANGE, as is a page past the cache.
 *   blocks       int32 [T, width], device, as mla_block_select writes them
 *   workspace    device scratch of mla_block_attention_workspace_bytes(T, H, width) bytes, 16-byte aligned; as there
 *   others       as mla_chunk_attention. min(width, max_pages) * page_size * (tokens in 64 query rows) is below 2^31 - 4096
 *                (otherwise MLA_EUNSUPPORTED)
 * The sizes decide which of two kernels runs, and how lists are cut; results agree to rounding.
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED, MLA_ENOWORKSPACE or MLA_ECUDA.
 */
size_t mla_block_attention_workspace_bytes(int T, int H, int width);
int mla_block_attention(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv, const int32_t* blocks, int width,
                        const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int n_seq,
                        int max_pages, int page_size, float sm_scale, void* out_bf16, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Drafted trees. The n tokens of a sequence are drafted ones whose rows are the last n of its kv_len positions,
 * in an order in which parents come first. As calls in turn: mla_tree_mask (the positions that their rotary parts
 * are turned by), mla_rope_kv_write, mla_tree_attention, and once a path is accepted mla_tree_commit. Lengths are read
 * on the device; launched with programmatic stream serialization.
 *
 * mla_tree_mask - for token i of a sequence, parent[q_start[s] + i] is the index within the sequence of the
 * token before it (negative: it follows the context). Row t of `mask` receives a bit for the token itself and each of
 * its ancestors (bit j % 32 of word j / 32: token j), positions[t] (may be NULL) kv_len - n + its depth: the number of its
 * ancestors. A parent that does not come before its child counts as none, and a token j >= 32 * mask_words
 * has no bit; both are flagged MLA_ERR_CHUNK_RANGE. (With mask_words 0 only positions are made.)
 *   parent, positions  int32 [T], device;  mask  uint32 [T, mask_words], device
 * Returns MLA_OK, MLA_EINVAL or MLA_ECUDA.
 */
int mla_tree_mask(const int32_t* parent, int T, const int32_t* q_start, const int32_t* kv_len, int n_seq, uint32_t* mask,
                  int mask_words, int32_t* positions, void* stream);

/*
 * mla_tree_attention - mla_chunk_attention with a mask among the new tokens: a token attends every position below
 * kv_len - n and, of the others, position kv_len - n + j if bit j of its row of `mask` is set (any mask: also
 * one with later tokens, or empty; a token j >= 32 * mask_words is attended by none). All else as mla_chunk_attention,
 * its workspace (mla_chunk_attention_workspace_bytes) included.
 *   mask      uint32 [T, mask_words], device, 4-byte aligned
 */
int mla_tree_attention(const void* q_bf16, int T, int H, int d_qk, mla_kv_cache_t kv, const int32_t* q_start,
                       const int32_t* kv_len, const int32_t* block_table, int n_seq, int max_pages, int page_size,
                       const uint32_t* mask, int mask_words, float sm_scale, void* out_bf16, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * mla_tree_commit - moves the rows of the accepted tokens path[s, 0 .. path_len[s]-1] (indices within the sequence,
 * ascending) to positions kv_len - n, kv_len - n + 1, ..; kv_len_out[s] (may be NULL, or kv_len itself)
 * becomes kv_len - n + path_len. A path is cut before an entry that is not above the one before it or not
 * one of the tokens, and to its max_path entries; a sequence with fewer positions than tokens, or more than the
 * table, keeps its rows and length; both are flagged MLA_ERR_CHUNK_RANGE. A row whose position, old or new, has no
 * page, is the reserved slot or lies past the cache is not moved and flagged MLA_ERR_PAGE_RANGE.
 * Precondition: no two sequences share the pages of their drafted tokens.
 *   path      int32 [n_seq, max_path], device;  path_len, kv_len_out  int32 [n_seq], device
 * Returns MLA_OK, MLA_EINVAL, MLA_EUNSUPPORTED or MLA_ECUDA.
 */
int mla_tree_commit(mla_kv_cache_t kv, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int n_seq,
                    int max_pages, int page_size, const int32_t* path, const int32_t* path_len, int max_path,
                    int32_t* kv_len_out, void* stream);

/*
 * Pages of a cache. Page p is the slots p * page_size .. (p + 1) * page_size - 1; pages
 * are counted in `refcount` (int32 [num_pages], device): how many block-table rows
 * hold each, 0 for a free page. Page 0 contains the reserved slot: it is never handed
 * out, freed, moved or counted. num_pages is at most num_slots / page_size. Block
 * tables are int32 [n_seq, max_pages], -1 where there is no page. All results are
 * independent of the order in which CTAs run. Range violations are dropped and flagged
 * (MLA_ERR_PAGE_RANGE). Launched with programmatic stream serialization.
 *
 * mla_page_copy - page src[i] of src_kv to page dst[i] of dst_kv, i < n (int32, device);
 * the caches may be one. A negative src or a dst <= 0 is skipped. Precondition: no
 * page is a dst twice, and within one cache no dst is also a src.
 */
int mla_page_copy(mla_kv_cache_t dst_kv, mla_kv_cache_t src_kv, int page_size, const int32_t* dst, const int32_t* src,
                  int64_t n, void* stream);

/*
 * mla_page_free - rows[i] (int32 [n], device) of the table let go of their pages: each
 * count drops by one (one that was 0 stays 0 and is flagged MLA_ERR_PAGE_COUNT) and the
 * row becomes -1. A negative row is skipped; a row listed twice is freed once.
 */
int mla_page_free(int32_t* refcount, int num_pages, int32_t* block_table, int n_seq, int max_pages,
                  const int32_t* rows, int n, void* stream);

/*
 * mla_page_fork - row child[i] of the table becomes a copy of row parent[i] as far as
 * its first lens[i] positions, i < n (int32, device): whole pages are shared (their
 * counts rise by one), a last page that is not full is copied, its rows up to
 * lens[i], to a free page; the row's other entries become -1. Free pages are taken in
 * ascending order, fork by fork; when none is left the entry stays -1 (the rows are then
 * absent for the child) and MLA_ERR_POOL_EMPTY is set. The child's row is overwritten:
 * free it first if it holds pages. A negative parent or child skips the fork; parent ==
 * child or a length past the table is dropped and flagged. A parent may be forked
 * many times in a call. A last page that is not full and is page 0 or none of the pool's
 * (flagged) is not copied: the entry stays -1. Preconditions: every page that a parent holds is counted, no
 * child is listed twice, and none is a parent of the same call.
 */
int mla_page_fork(mla_kv_cache_t kv, int page_size, int32_t* refcount, int num_pages, int32_t* block_table, int n_seq,
                  int max_pages, const int32_t* parent, const int32_t* child, const int32_t* lens, int n,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * mla_page_compact - moves the live pages (count > 0) to pages 1 .. live: a live page
 * above that range goes to the vacant page of the same rank (both in ascending order),
 * the others stay. refcount_out and table_out receive the counts and the table that go
 * with it (they may be refcount and block_table themselves); an entry that names a free page
 * becomes -1. page_map (int32 [num_pages], may be NULL) receives where each page went: its
 * new index, -1 for a free page, 0 for page 0.
 */
int mla_page_compact(mla_kv_cache_t kv, int page_size, const int32_t* refcount, int32_t* refcount_out, int num_pages,
                     const int32_t* block_table, int32_t* table_out, int n_seq, int max_pages, int32_t* page_map,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device scratch (16-byte aligned) for mla_page_fork of up to n_forks forks, and
 * for mla_page_compact, of a pool of num_pages pages. */
size_t mla_page_workspace_bytes(int num_pages, int n_forks);

/*
 * mla_get_error - read and clear the device error word of the current device
 * (MLA_ERR_* bits accumulated by every launch since the last read). Blocks
 * until the device is idle. Returns MLA_OK or MLA_ECUDA; *host_code receives
 * the bits (host pointer, not NULL).
 */
int mla_get_error(int32_t* host_code);

/* Human-readable name of a return code (static string). */
const char* mla_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* MLASPARSE_H */
