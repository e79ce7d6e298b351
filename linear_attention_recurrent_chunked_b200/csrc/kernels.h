// Internal launchers of the library's kernels (host side). Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

template <typename T, int D>
cudaError_t launch_decode_step(const T *q, const T *k, const T *v, const float *g, const float *beta, float *S,
                               int B, int H, T *o, cudaStream_t st, bool raw = false);

template <typename T, int D>
cudaError_t launch_seq_scan(const T *q, const T *k, const T *v, const float *g, const float *beta, const float *S0,
                            const int32_t *cu, int N, int T_tot, int H, T *o, float *S_T, cudaStream_t st);

template <typename T, int D>
cudaError_t launch_chunk_simt(const T *q, const T *k, const T *v, const float *g, const float *beta, const float *S0,
                              const int32_t *cu, int N, int T_tot, int H, T *o, float *S_T, const uint32_t *err,
                              cudaStream_t st, bool raw = false);

// Tensor-core chunked forward, bf16 inputs, dk = dv = 128. Launches the
// validation / plan, the optional transition pass and the output pass;
// *stage names the launch that failed when an error is returned. The
// workspace holds the error word, the segment offsets and the per-segment
// transition slots (chunk_tc_workspace bytes for the preferred plan; a
// smaller workspace selects a coarser segmentation or none).
cudaError_t launch_chunk_tc(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v, const float *g,
                            const float *beta, const float *S0, const int32_t *cu, int N, int T_tot, int H,
                            __nv_bfloat16 *o, float *S_T, void *workspace, size_t ws_bytes, cudaStream_t st,
                            const char **stage);
int chunk_tc_seg_chunks(int N, int T_tot, int H);
size_t chunk_tc_workspace(int N, int T_tot, int H, int seg_chunks);

// Pipelined tensor-core chunked forward (same contract as launch_chunk_tc):
// plan, the parallel prep pass (decay scalars and UT solve of every chunk),
// the transition pass with its links (seg_chunks > 0 only) and the output
// pass. Needs chunk_ws_workspace(N, T_tot, H, seg_chunks) bytes of workspace.
// raw: q, k are unnormalised and g, beta hold the gate logits a, b (g = -softplus(a),
// beta = sigmoid(b)); the normalisation and gates are applied inside the passes.
cudaError_t launch_chunk_ws(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v, const float *g,
                            const float *beta, const float *S0, const int32_t *cu, int N, int T_tot, int H,
                            __nv_bfloat16 *o, float *S_T, void *workspace, int seg_chunks, cudaStream_t st,
                            const char **stage, bool raw = false);
int chunk_ws_seg_chunks(int N, int T_tot, int H, bool varlen);  // varlen: cu_seqlens given
size_t chunk_ws_workspace(int N, int T_tot, int H, int seg_chunks);

// Input projection with int8 weights (W8A16 on the tensor cores): y = x (diag(scale) w)^T split
// into q, k, v (bf16) and the gate logits a, b (fp32). x [T][D] bf16 (D % 64 == 0), w [N][D] int8,
// N = H (2 dk + dv) + 2 H; err is the error word (reset here).
cudaError_t launch_proj_w8(const __nv_bfloat16 *x, const int8_t *w, const float *scale, int T, int D, int H, int dk,
                           int dv, __nv_bfloat16 *q, __nv_bfloat16 *k, __nv_bfloat16 *v, float *a, float *b,
                           uint32_t *err, cudaStream_t st, const char **stage);

// Causal attention (bf16, d = 128) over packed sequences: o_t = softmax_j<=t(scale q_t . k_j) v_j per
// head; q, k, v, o [T_tot][H][128]; cu (device, N+1 offsets) or NULL (N equal sequences);
// max_len = the longest sequence's length (bounds the grid); err = error word.
cudaError_t launch_attn_fwd(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                            const int32_t *cu, int N, int T_tot, int H, int max_len, float scale, __nv_bfloat16 *o,
                            uint32_t *err, cudaStream_t st, const char **stage);

// Norms of queries and keys per head, the rotation, and the write into the cache's pages (see
// gdn_qk_norm_rope): q, k, v rows of a token contiguous, tokens `*_stride` elements apart.
struct NormRope {
    const void *q, *k, *v;  // v used with slots only
    int64_t q_stride, k_stride, v_stride;
    const float *wq, *wk;  // [d], or NULL: ones
    float eps;
    const int32_t *positions;  // [T]
    int T, Hq, Hkv, rot;
    double base;
    void *q_out, *k_out;        // k_out may be NULL
    void *k_cache, *v_cache;    // [num_pages][Hkv][page_size][d], used with slots only
    const int32_t *slots;       // [T] or NULL
    int num_pages, page_size;   // page_size a power of two
    uint32_t *err;
};
cudaError_t launch_norm_rope(const NormRope &a, int d, bool bf16, cudaStream_t st);

// Causal attention with grouped heads over packed prompts (see gdn_attn_prefill), and the part of
// gdn_attn_decode over the prefix that a batch shares. The fields after `err` are the latter's; for it
// q is [B][Hq][d] with T_tot = B, and k, v are the cache.
constexpr int kPromptCtas = 296;  // CTAs that the GPU holds at once: two per SM
struct AttnPrefill {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    const int32_t *cu;
    int N, T_tot, max_len;
    int Hq, Hkv, G;
    float scale_log2;  // scale * log2(e)
    __nv_bfloat16 *o;
    uint32_t *err;
    const int32_t *pages;
    int num_pages, page_log, prefix_len, splits;
    float *part_o;    // [splits][B][Hq][d] unnormalised
    float2 *part_ml;  // [splits][B][Hq] reference maximum (log2 units) and sum
    uint64_t wait_ns;  // set by the launcher, as all below: how long a wait may last
    int withhold;      // (tests) the tile of the ring that the first CTA does not load, or 0
    int P, blocks;    // positions per query tile, query tiles of the longest sequence
    bool dense;       // blocks numbered sequence by sequence
};
int64_t attn_prefill_tiles(int T_tot, int N, int P);  // most query tiles that N sequences of T_tot tokens can have
cudaError_t launch_attn_prefill(AttnPrefill a, int d, cudaStream_t st, const char **stage);

// The same kernel without the mask over a cached prefix that a batch shares: partial results per split.
cudaError_t launch_attn_prefix(const AttnPrefill &a, int d, cudaStream_t st, const char **stage);

// Attention of one token per sequence over the paged cache (see gdn_attn_decode).
constexpr int kDecodeCtas = 148;  // runs that the own keys are cut into: one per SM
struct AttnDecode {
    const __nv_bfloat16 *q, *k_cache, *v_cache;
    const int32_t *table, *lens;  // [B][max_pages], [B]
    const int32_t *prefix_pages;
    int B, Hq, Hkv, G, max_pages, num_pages, page_log, prefix_len, splits;
    float scale_log2;
    __nv_bfloat16 *o;
    uint32_t *err;
    // pieces, G rows each: two slots per CTA, then (with a prefix) one per (sequence, key head)
    float *slot_o;
    float2 *slot_ml;
    float *part_o;  // the prefix kernel's, per split
    float2 *part_ml;
    uint32_t *bad;  // [kDecodeCtas] the error bits of each CTA
    int rows;       // set by the launcher, as all below: query heads that a CTA of the combine kernel takes
    int withhold;   // (tests) not 0: the first CTA's warps do not load the second step of their runs
    uint64_t wait_ns;  // how long a wait may last
};
int attn_decode_splits(int B, int Hq, int Hkv, int prefix_len);
size_t attn_decode_slots(int B, int Hq, int Hkv, int prefix_len);  // rows of d floats
cudaError_t launch_attn_decode(AttnDecode a, int d, cudaStream_t st, const char **stage);

// Failure injection for tests (set by gdn_debug_inject; off by default): the pipelined path's
// first segment of head 0 withholds its end-state flag, and waits for flags give up after
// flag_wait_ns (0 = the normal bound) instead of hanging; or the grouped-head attention kernels' first
// CTA withholds a load (tile 2, the keys of its second step, or 3, their values; 0 = none) and all of their
// waits give up after wait_ns (0 = the normal bound).
struct Inject {
    bool withhold_first_link;
    uint64_t flag_wait_ns;
    int withhold_tile;
    uint64_t wait_ns;
};
Inject inject_settings();

// Kernel timing hooks (no-ops unless gdn_profile_enable(1)): an event pair
// around the launches between prof_start and prof_stop, recorded on st.
void *prof_start(const char *name, cudaStream_t st);
void prof_stop(void *handle);
// Diagnostic: T = (I + A)^{-1} for one strictly lower 64 x 64 fp32 matrix (row-major, device).
cudaError_t launch_diag_ut_solve(const float *A, float *T, cudaStream_t st);

// Writes the workspace error word: ERRBIT_SEQLENS if cu_seqlens (device, N+1
// entries) is not 0 = c0 <= ... <= cN = T_tot, else 0. With cu == NULL it
// just clears the word.
cudaError_t launch_validate_seqlens(const int32_t *cu, int N, int T_tot, uint32_t *err, cudaStream_t st);

}  // namespace gdn
