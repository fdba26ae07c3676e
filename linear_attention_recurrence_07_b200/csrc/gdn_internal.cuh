// Internal declarations shared by the kernels and the C-ABI layer of libgdn.so.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

constexpr int kHeadDim = 128;   // dk == dv == 128: the head size of the model (section 2.1)
constexpr int kChunk = 64;      // tokens per chunk of the chunkwise form

// Kernel arguments of the chunked prefill (plain pointers; shapes validated by the caller).
struct ChunkArgs {
    const void *q, *k, *v;
    const float *alpha, *beta, *S0;
    void *o;
    float *S_final;
    int B, T, Hqk, Hv;
    // Packed sequences: B sequences at token rows cu_seqlens[b] .. cu_seqlens[b+1]
    // of token arrays with one batch row of T tokens; null for [B, T, ...] arrays.
    const int *cu_seqlens = nullptr;
};

struct DecodeArgs {
    const void *q, *k, *v;
    const float *alpha, *beta, *S;
    void *o;
    float *S_new;
    int B, Hqk, Hv;
    int ntok = 1;                // tokens per sequence
    float *S_steps = nullptr;    // state after each token, or null
    const int *slots = nullptr;  // pool index of each sequence's state, or null
    int n_slots = 0;
};

// Launchers: enqueue on `stream`, return the launch's cudaError_t.
cudaError_t launch_decode(const DecodeArgs &a, gdn_dtype dtype, cudaStream_t stream);
cudaError_t launch_chunk_simt(const ChunkArgs &a, gdn_dtype dtype, cudaStream_t stream);
cudaError_t launch_chunk_tc(const ChunkArgs &a, cudaStream_t stream);
bool chunk_tc_available();
// Segment-parallel prefill (bf16, tensor cores): each sequence in up to `segments`
// pieces; workspace of chunk_tc_split_workspace bytes (0: no split needed).
size_t chunk_tc_split_workspace(int B, int T, int Hv, int segments);
cudaError_t launch_chunk_tc_split(const ChunkArgs &a, int segments, void *workspace,
                                  cudaStream_t stream);
// Scratch gdn_chunk_fwd_split uses for these arguments (0: it will not split).
size_t split_scratch_needed(int B, int T, int Hv, int dk, int dv, int segments, gdn_dtype dtype);
// Backward pass (gdn_bwd.cu): gradients of q, k, v, alpha, beta, S0.
struct BwdLaunch {
    const void *q, *k, *v, *dO;
    const float *alpha, *beta, *S0, *dS_final;
    float *dq, *dk, *dv, *dalpha, *dbeta, *dS0;
    float *work;
    int B, T, Hqk, Hv;
};
size_t bwd_workspace(int B, int T, int Hv);
cudaError_t launch_bwd(const BwdLaunch &L, gdn_dtype dtype, cudaStream_t stream);
// Chunkwise backward (gdn_bwd_chunk.cu, bf16 inputs): prep, forward state chain,
// gradient chain and per-chunk gradients; workspace of bwd_chunk_workspace bytes.
size_t bwd_chunk_workspace(int B, int T, int Hv);
cudaError_t launch_bwd_chunk(const BwdLaunch &L, cudaStream_t stream);

// Pipelined prefill (gdn_chunk_pipe.cu): prep CTAs stream each chunk's WY operands
// to state-carrying chain CTAs through a ring in the workspace (cooperative launch).
int chunk_pipe_chain_ctas(int B, int Hqk, int Hv, int sms, int req);
size_t chunk_pipe_workspace(int B, int Hqk, int Hv);
cudaError_t launch_chunk_pipe(const ChunkArgs &a, int chain_ctas, long long wait_limit,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream);
// Read and clear a kernel file's device error word (bit 0: a bounded wait gave up).
cudaError_t chunk_pipe_take_error(unsigned *out);
cudaError_t chunk_tc_take_error(unsigned *out);
cudaError_t split_take_error(unsigned *out);

// ---- linear attention with a constant decay per head (gdn_decay.cu, gdn_decay_tc.cu)
// One walk over the tokens of every (sequence, V head), forwards or backwards (rev),
// with operands x, y, z of 128 columns each and the state H (128 x 128, row = y's
// dimension, column = z's), which always includes the decay to the next token:
//   forwards:  o_t = H^T x_t + sum_{s <= t} lambda^{t-s} (x_t . y_s) z_s  (H at each chunk's start)
//   backwards: the same with the tokens in reverse order.
// Prefill is (x, y, z) = (q, k, v); the gradients are the same walk with
//   dq: (dO, v, k) forwards,  dk: (v, dO, q) and dv: (k, q, dO) backwards.
struct DecayWalk {
    const void *x, *y, *z;
    int hx, hy, hz;                  // heads of each operand: V head h reads head h / (Hv / heads)
    void *o = nullptr;               // [B, T, Hv, 128] of the operands' type, or fp32 (o_f32)
    bool o_f32 = false;
    const float *decay;
    const float *init = nullptr;     // [B, Hv, 128, 128] or null (zeros)
    bool init_trans = false;         // init is stored transposed (row = z's dimension)
    bool init_decays = false;        // init still lacks one decay (H = lambda init)
    float *fin = nullptr;            // end state, or null
    bool fin_back = false;           // end state without the decay to the next token
    int B, T, Hv;
    bool rev = false;
    const int *cu_seqlens = nullptr; // packed sequences (see ChunkArgs), forwards only
    // Segments (dense only): nseg > 1 pieces of seg_chunks chunks behind the first head_chunks.  A
    // first launch walks those, and writes seg [B, nseg, Hv, 128, 128]: entry 0 the state behind
    // them, entry g the state that segment g - 1 adds on its own (tensor cores: times the
    // head's power of two); the second launch starts segment g from the decayed sum of 0 .. g.
    int nseg = 1, seg_chunks = 0, head_chunks = 0;
    float *seg = nullptr;
};
// Up to three walks of the same B, T, Hv and segments, side by side in one launch (two with
// segments): a gradient's three walks fill the device where one would not.
constexpr int kMaxWalks = 3;
struct DecayWalks {
    DecayWalk w[kMaxWalks];
    int n;
    bool wide;      // CUDA cores: one CTA per head instead of four
    int wait_tries; // tensor cores: tries, of up to kWaitTryMicros each, before a wait gives up
};
constexpr int kWaitTryMicros = 20;
cudaError_t launch_decay_walks_simt(const DecayWalks &d, cudaStream_t stream);
cudaError_t launch_decay_walks_tc(const DecayWalks &d, cudaStream_t stream);   // bf16 operands
cudaError_t decay_tc_take_error(unsigned *out);
// out_a, out_b [rows, Hqk, 128] = sums over each QK head's V heads of part_a, part_b [rows, Hv, 128]
cudaError_t launch_head_sums(const float *part_a, const float *part_b, void *out_a, void *out_b, long long rows,
                             int Hqk, int Hv, gdn_dtype dtype, cudaStream_t stream);

struct DecayDecodeArgs {
    const void *q, *k, *v;
    const float *decay, *S;
    void *o;
    float *S_new;
    int B, Hqk, Hv;
    const int *slots = nullptr;
    int n_slots = 0;
};
cudaError_t launch_decay_decode(const DecayDecodeArgs &a, gdn_dtype dtype, cudaStream_t stream);

// ---- draft trees (gdn_tree.cu): alpha/beta (delta rule) or decay (then alpha, beta null)
struct TreeArgs {
    const void *q, *k, *v;
    const float *alpha, *beta, *decay;
    const int *parents, *accepted, *slots;
    const float *pool;
    float *pool_out;                 // commit
    void *o;                         // verification
    int B, n, n_slots, Hqk, Hv;
};
constexpr int kMaxTreeNodes = 64;
cudaError_t launch_tree(const TreeArgs &a, gdn_dtype dtype, cudaStream_t stream);
cudaError_t launch_tree_commit(const TreeArgs &a, gdn_dtype dtype, cudaStream_t stream);

// ---- 8-bit state cache (gdn_state_cache.cu)
struct StateCacheArgs {
    const float *pool_in;
    float *pool_out;
    const int *slots, *cache_slots;
    void *codes;
    float *scales;
    int N, n_slots, n_cache, Hv;
};
cudaError_t launch_state_store(const StateCacheArgs &a, gdn_code code, cudaStream_t stream);
cudaError_t launch_state_load(const StateCacheArgs &a, gdn_code code, cudaStream_t stream);

// Status of a launch for the C entries (remembers the error for gdn_last_cuda_error).
gdn_status launch_status(cudaError_t err);

// sst: null, or where the first segments write S_start(1)^T in bf16 (see TcParams).
cudaError_t launch_chunk_tc_segments(const ChunkArgs &a, int seg_len, int nseg, float *segD,
                                     float *segM, __nv_bfloat16 *R, __nv_bfloat16 *sst,
                                     cudaStream_t stream);

// Element conversions used by the kernels.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// log(alpha) with the documented clamp, so alpha == 0 stays finite.
__device__ __forceinline__ float clamped_log(float alpha) {
    return fmaxf(logf(alpha), -87.0f);
}

// A head's decay with the same clamp; negative or NaN: NaN, which the head's results show.
__device__ __forceinline__ float clamped_decay(float lam) {
    return lam >= 0.f ? fmaxf(lam, 1.6458114e-38f) : __int_as_float(0x7fc00000);
}

}  // namespace gdn
