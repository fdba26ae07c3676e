// C ABI of the constant-decay linear attention, the draft trees and the 8-bit state
// cache: argument checks and dispatch.  See include/gdn.h.
#include "gdn_internal.cuh"

namespace {

using gdn::DecayWalk;
using gdn::launch_status;

bool misaligned(const void *p, uintptr_t to) { return p && (reinterpret_cast<uintptr_t>(p) & (to - 1)); }

gdn_status check_sizes(int Hqk, int Hv, int dk, int dv)
{
    if (Hqk <= 0 || Hv <= 0 || dk <= 0 || dv <= 0) return GDN_ERR_INVALID_ARG;
    if (Hv % Hqk != 0 || dk != gdn::kHeadDim || dv != gdn::kHeadDim) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
bool is_dtype(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    return sms;
}

// Microseconds that a wait inside a tensor-core walk may take (0: the default); see
// gdn_set_decay_wait_limit.
thread_local long long g_wait_limit = 0;
constexpr long long kDefaultWait = 2000000;

constexpr size_t kStateBytes = (size_t)gdn::kHeadDim * gdn::kHeadDim * sizeof(float);
constexpr int kMaxDecaySegments = 16;

// fp32: whether a CTA takes a whole head (half the arithmetic) or 32 of its columns (four
// times the CTAs).  heads x segments, narrow against wide: 30 28 / 57 us, 64 43 / 59 us,
// 96 (T = 64) 47 / 34 us, 96 (T = 100) 48 / 51 us, 120 73 / 61 us.
constexpr int kWideHeads = 96;
bool wide_walk(const DecayWalk &w, int walks)
{
    const int nchunks = (w.T + gdn::kChunk - 1) / gdn::kChunk;
    const long long heads = (long long)w.B * w.Hv * walks;
    const int most = w.cu_seqlens ? 1 : nchunks < kMaxDecaySegments ? nchunks : kMaxDecaySegments;
    return heads * most >= kWideHeads;
}

// Segments of `walks` dense walks that run side by side: as many as fill the device with
// one CTA (fp32, narrow: one head's four half-SM CTAs) per walk, head and segment.  The launch
// that computes their start states has one such CTA to spare, the last segment's, and walks
// the head of the sequence with it: as much of a segment as takes the time of a state alone
// (bf16: 85% of a chunk's, which D and the state take; fp32: 25%, of its arithmetic).  48 heads,
// T=4096, three segments of 17 chunks behind 13: 58 us, of 22 each: 65; parts of 45% 61, 60% 59,
// 100% 61 us.  bf16: segments of
// at least four chunks, because that launch reads y and z once more and starts anew; the fp32
// kernel is bound by its arithmetic, so one chunk is enough.
void choose_segments(DecayWalk &w, int walks, gdn_dtype dtype)
{
    const int least = dtype == GDN_F32 ? 1 : 4;
    const int nchunks = (w.T + gdn::kChunk - 1) / gdn::kChunk;
    const long long units = (long long)w.B * w.Hv * walks * (dtype == GDN_F32 && !wide_walk(w, walks) ? 2 : 1);
    long long n = sm_count() / units;
    if (n > kMaxDecaySegments) n = kMaxDecaySegments;
    w.nseg = 1;
    w.seg_chunks = nchunks;
    w.head_chunks = 0;
    if (n < 2 || nchunks <= least) return;
    // the shortest segments of which n and a head of `part` percent of one cover the sequence
    const long long part = dtype == GDN_F32 ? 25 : 85;
    int per = (int)((100LL * nchunks + 100 * n + part - 1) / (100 * n + part));
    if (per < least) per = least;
    const int head = nchunks - n * per > 0 ? (int)(nchunks - n * per) : 0;
    const int nseg = (nchunks - head + per - 1) / per;
    if (nseg < 2) return;
    w.nseg = nseg;
    w.seg_chunks = per;
    w.head_chunks = head;
}
size_t segment_bytes(const DecayWalk &w)
{
    return w.nseg > 1 ? (size_t)w.B * w.nseg * w.Hv * kStateBytes : 0;
}

gdn_status run_walks(gdn::DecayWalks &d, gdn_dtype dtype, cudaStream_t s)
{
    const long long tries = (g_wait_limit > 0 ? g_wait_limit : kDefaultWait) / gdn::kWaitTryMicros;
    d.wait_tries = (int)(tries < 0x7fffffff ? tries : 0x7fffffff);
    if (dtype == GDN_F32) return launch_status(gdn::launch_decay_walks_simt(d, s));
    if (!gdn::chunk_tc_available()) return GDN_ERR_UNSUPPORTED;
    return launch_status(gdn::launch_decay_walks_tc(d, s));
}

// T == 0: the state passes through.
gdn_status pass_state(float *dst, const float *src, int B, int Hv, cudaStream_t s)
{
    if (!dst || dst == src) return GDN_OK;
    const size_t bytes = (size_t)B * Hv * kStateBytes;
    return launch_status(src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(dst, 0, bytes, s));
}

gdn_status fwd_common(const void *q, const void *k, const void *v, const float *decay, const float *S0, void *o,
                      float *S_final, const int *cu, int B, int T, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype,
                      void *workspace, size_t workspace_bytes, void *stream)
{
    if (B < 0 || T < 0 || !is_dtype(dtype)) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_sizes(Hqk, Hv, dk, dv);
    if (st != GDN_OK) return st;
    if (B > 65535 || Hv > 65535) return GDN_ERR_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    const void *ptrs[] = {q, k, v, decay, S0, o, S_final};
    for (const void *p : ptrs)
        if (misaligned(p, 16)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return pass_state(S_final, S0, B, Hv, s);
    if (!q || !k || !v || !decay || !o) return GDN_ERR_INVALID_ARG;
    gdn::DecayWalks d{};
    d.n = 1;
    DecayWalk &w = d.w[0];
    w.x = q; w.y = k; w.z = v;
    w.hx = w.hy = Hqk; w.hz = Hv;
    w.o = o;
    w.decay = decay;
    w.init = S0;
    w.init_decays = true;
    w.fin = S_final;
    w.fin_back = true;
    w.B = B; w.T = T; w.Hv = Hv;
    w.cu_seqlens = cu;
    w.nseg = 1;
    w.seg_chunks = (T + gdn::kChunk - 1) / gdn::kChunk;
    if (!cu) {
        choose_segments(w, 1, dtype);
        const size_t need = segment_bytes(w);
        if (need > 0) {
            if (!workspace || workspace_bytes < need || misaligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
            w.seg = static_cast<float *>(workspace);
        }
    }
    d.wide = wide_walk(w, 1);
    return run_walks(d, dtype, s);
}

gdn_status check_token_op(int B, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype, long long ctas_per_head)
{
    if (B < 0 || !is_dtype(dtype)) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_sizes(Hqk, Hv, dk, dv);
    if (st != GDN_OK) return st;
    return (long long)B * Hv * ctas_per_head > 0x7fffffffLL ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn_status decode_common(const void *q, const void *k, const void *v, const float *decay, const float *S, void *o,
                         float *S_new, const int *slots, int B, int n_slots, int Hqk, int Hv, int dk, int dv,
                         gdn_dtype dtype, void *stream)
{
    gdn_status st = check_token_op(B, Hqk, Hv, dk, dv, dtype, 4);
    if (st != GDN_OK) return st;
    if (B == 0) return GDN_OK;
    const bool states = n_slots > 0 || !slots;
    if (!q || !k || !v || !decay || !o || (states && (!S || !S_new))) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, decay, S, o, S_new};
    for (const void *p : ptrs)
        if (misaligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (misaligned(slots, 4)) return GDN_ERR_INVALID_ARG;
    gdn::DecayDecodeArgs a{q, k, v, decay, S, o, S_new, B, Hqk, Hv, slots, n_slots};
    return launch_status(gdn::launch_decay_decode(a, dtype, static_cast<cudaStream_t>(stream)));
}

// q, o null for the commit, accepted null for the verification; alpha and beta, or decay.
gdn_status tree_common(gdn::TreeArgs a, bool commit, int dk, int dv, gdn_dtype dtype, void *stream)
{
    gdn_status st = check_token_op(a.B, a.Hqk, a.Hv, dk, dv, dtype, 4);
    if (st != GDN_OK) return st;
    if (a.n < 1 || a.n_slots < 0) return GDN_ERR_INVALID_ARG;
    if (a.n > gdn::kMaxTreeNodes) return GDN_ERR_UNSUPPORTED;
    if (a.B == 0) return GDN_OK;
    if (!a.k || !a.v || !a.parents || (commit ? !a.accepted : (!a.q || !a.o))) return GDN_ERR_INVALID_ARG;
    if (a.n_slots > 0 && !(commit ? a.pool_out : a.pool)) return GDN_ERR_INVALID_ARG;
    if (!a.slots && a.n_slots < a.B) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {a.q, a.k, a.v, a.alpha, a.beta, a.decay, a.pool, a.pool_out, a.o};
    for (const void *p : ptrs)
        if (misaligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (misaligned(a.parents, 4) || misaligned(a.accepted, 4) || misaligned(a.slots, 4)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_status(commit ? gdn::launch_tree_commit(a, dtype, s) : gdn::launch_tree(a, dtype, s));
}

gdn_status check_cache(const void *pool, const int *slots, const void *codes, const float *scales,
                       const int *cache_slots, int N, int n_slots, int n_cache, int Hv, int dk, int dv, gdn_code code)
{
    if (N < 0 || n_slots < 0 || n_cache < 0 || (code != GDN_CODE_INT8 && code != GDN_CODE_E4M3)) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_sizes(1, Hv, dk, dv);
    if (st != GDN_OK) return st;
    if ((long long)N * Hv * 4 > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    if (!slots || !cache_slots || (n_slots > 0 && !pool) || (n_cache > 0 && (!codes || !scales))) return GDN_ERR_INVALID_ARG;
    if (misaligned(pool, 16) || misaligned(codes, 16) || misaligned(scales, 16) || misaligned(slots, 4) ||
        misaligned(cache_slots, 4))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_set_decay_wait_limit(long long microseconds)
{
    if (microseconds < 0) return GDN_ERR_INVALID_ARG;
    g_wait_limit = microseconds;
    return GDN_OK;
}

long long gdn_get_decay_wait_limit(void) { return g_wait_limit; }

size_t gdn_decay_fwd_workspace(int B, int T, int Hv, int dk, int dv, gdn_dtype dtype)
{
    if (B <= 0 || T <= 0 || Hv <= 0 || dk != gdn::kHeadDim || dv != gdn::kHeadDim || !is_dtype(dtype)) return 0;
    DecayWalk w{};
    w.B = B; w.T = T; w.Hv = Hv;
    choose_segments(w, 1, dtype);
    return segment_bytes(w);
}

gdn_status gdn_decay_fwd(const void *q, const void *k, const void *v, const float *decay, const float *S0, void *o,
                         float *S_final, int B, int T, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    return fwd_common(q, k, v, decay, S0, o, S_final, nullptr, B, T, Hqk, Hv, dk, dv, dtype, workspace,
                      workspace_bytes, stream);
}

gdn_status gdn_decay_fwd_varlen(const void *q, const void *k, const void *v, const float *decay, const float *S0,
                                void *o, float *S_final, const int *cu_seqlens, int N, int T_total, int Hqk, int Hv,
                                int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (N > 0 && T_total > 0 && (!cu_seqlens || misaligned(cu_seqlens, 4))) return GDN_ERR_INVALID_ARG;
    return fwd_common(q, k, v, decay, S0, o, S_final, cu_seqlens, N, T_total, Hqk, Hv, dk, dv, dtype, nullptr, 0, stream);
}

gdn_status gdn_decay_decode_step(const void *q, const void *k, const void *v, const float *decay, const float *S,
                                 void *o, float *S_new, int B, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype,
                                 void *stream)
{
    return decode_common(q, k, v, decay, S, o, S_new, nullptr, B, 0, Hqk, Hv, dk, dv, dtype, stream);
}

gdn_status gdn_decay_decode_step_slots(const void *q, const void *k, const void *v, const float *decay,
                                       float *state_pool, const int *slots, void *o, int B, int n_slots, int Hqk,
                                       int Hv, int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (n_slots < 0 || (B > 0 && !slots)) return GDN_ERR_INVALID_ARG;
    return decode_common(q, k, v, decay, state_pool, o, state_pool, slots, B, n_slots, Hqk, Hv, dk, dv, dtype, stream);
}

size_t gdn_decay_bwd_workspace(int B, int T, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype)
{
    if (B <= 0 || T <= 0 || Hqk <= 0 || Hv <= 0 || Hv % Hqk || dk != gdn::kHeadDim || dv != gdn::kHeadDim ||
        !is_dtype(dtype))
        return 0;
    DecayWalk w{};
    w.B = B; w.T = T; w.Hv = Hv;
    choose_segments(w, 3, dtype);
    const size_t rows = Hv == Hqk ? 0 : (size_t)B * T * Hv * gdn::kHeadDim * sizeof(float);
    return 3 * segment_bytes(w) + 2 * rows;
}

gdn_status gdn_decay_bwd(const void *q, const void *k, const void *v, const float *decay, const float *S0,
                         const void *dO, const float *dS_final, void *dq, void *dk, void *dv, float *dS0, int B, int T,
                         int Hqk, int Hv, int dk_, int dv_, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    if (B < 0 || T < 0 || !is_dtype(dtype)) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_sizes(Hqk, Hv, dk_, dv_);
    if (st != GDN_OK) return st;
    if (B > 65535 || Hv > 65535) return GDN_ERR_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    const void *ptrs[] = {q, k, v, decay, S0, dO, dS_final, dq, dk, dv, dS0};
    for (const void *p : ptrs)
        if (misaligned(p, 16)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return pass_state(dS0, dS_final, B, Hv, s);
    if (!q || !k || !v || !decay || !dO || !dq || !dk || !dv) return GDN_ERR_INVALID_ARG;

    DecayWalk w{};
    w.decay = decay;
    w.B = B; w.T = T; w.Hv = Hv;
    choose_segments(w, 3, dtype);
    const size_t seg = segment_bytes(w);
    const bool shared = Hv != Hqk;
    const size_t need = gdn_decay_bwd_workspace(B, T, Hqk, Hv, dk_, dv_, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 256))) return GDN_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    // shared QK heads: one fp32 row per token and V head for each of dq and dk, summed afterwards
    const long long tokens = (long long)B * T;
    float *rows_q = shared ? reinterpret_cast<float *>(ws + 3 * seg) : nullptr;
    float *rows_k = shared ? rows_q + (size_t)tokens * Hv * gdn::kHeadDim : nullptr;

    gdn::DecayWalks d{};
    d.n = 3;
    d.wide = wide_walk(w, 3);
    for (int i = 0; i < 3; ++i) {
        d.w[i] = w;
        d.w[i].seg = seg ? reinterpret_cast<float *>(ws + i * seg) : nullptr;
    }
    // dq_t = S_t dO_t: the walk of S^T (row = v's dimension)
    DecayWalk &wq = d.w[0];
    wq.x = dO; wq.y = v; wq.z = k;
    wq.hx = wq.hy = Hv; wq.hz = Hqk;
    wq.init = S0; wq.init_trans = true; wq.init_decays = true;
    wq.o = shared ? static_cast<void *>(rows_q) : dq;
    wq.o_f32 = shared;
    // dk_t = G_t v_t: backwards, the walk of G^T
    DecayWalk &wk = d.w[1];
    wk.rev = true;
    wk.x = v; wk.y = dO; wk.z = q;
    wk.hx = wk.hy = Hv; wk.hz = Hqk;
    wk.init = dS_final; wk.init_trans = true;
    wk.o = shared ? static_cast<void *>(rows_k) : dk;
    wk.o_f32 = shared;
    // dv_t = G_t^T k_t, and dS0 = lambda G_0
    DecayWalk &wv = d.w[2];
    wv.rev = true;
    wv.x = k; wv.y = q; wv.z = dO;
    wv.hx = wv.hy = Hqk; wv.hz = Hv;
    wv.init = dS_final;
    wv.fin = dS0;
    wv.o = dv;
    st = run_walks(d, dtype, s);
    if (st != GDN_OK || !shared) return st;
    return launch_status(gdn::launch_head_sums(rows_q, rows_k, dq, dk, tokens, Hqk, Hv, dtype, s));
}

gdn_status gdn_decode_tree(const void *q, const void *k, const void *v, const float *alpha, const float *beta,
                           const int *parents, const float *state_pool, const int *slots, void *o, int B, int n,
                           int n_slots, int Hqk, int Hv, int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (B > 0 && (!alpha || !beta)) return GDN_ERR_INVALID_ARG;
    gdn::TreeArgs a{q, k, v, alpha, beta, nullptr, parents, nullptr, slots, state_pool, nullptr, o, B, n, n_slots, Hqk, Hv};
    return tree_common(a, false, dk, dv, dtype, stream);
}

gdn_status gdn_decay_decode_tree(const void *q, const void *k, const void *v, const float *decay, const int *parents,
                                 const float *state_pool, const int *slots, void *o, int B, int n, int n_slots,
                                 int Hqk, int Hv, int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (B > 0 && !decay) return GDN_ERR_INVALID_ARG;
    gdn::TreeArgs a{q, k, v, nullptr, nullptr, decay, parents, nullptr, slots, state_pool, nullptr, o, B, n, n_slots, Hqk, Hv};
    return tree_common(a, false, dk, dv, dtype, stream);
}

gdn_status gdn_tree_commit(const void *k, const void *v, const float *alpha, const float *beta, const int *parents,
                           const int *accepted, float *state_pool, const int *slots, int B, int n, int n_slots,
                           int Hqk, int Hv, int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (B > 0 && (!alpha || !beta)) return GDN_ERR_INVALID_ARG;
    gdn::TreeArgs a{nullptr, k, v, alpha, beta, nullptr, parents, accepted, slots, nullptr, state_pool, nullptr, B, n, n_slots, Hqk, Hv};
    return tree_common(a, true, dk, dv, dtype, stream);
}

gdn_status gdn_decay_tree_commit(const void *k, const void *v, const float *decay, const int *parents,
                                 const int *accepted, float *state_pool, const int *slots, int B, int n, int n_slots,
                                 int Hqk, int Hv, int dk, int dv, gdn_dtype dtype, void *stream)
{
    if (B > 0 && !decay) return GDN_ERR_INVALID_ARG;
    gdn::TreeArgs a{nullptr, k, v, nullptr, nullptr, decay, parents, accepted, slots, nullptr, state_pool, nullptr, B, n, n_slots, Hqk, Hv};
    return tree_common(a, true, dk, dv, dtype, stream);
}

gdn_status gdn_state_store(const float *state_pool, const int *slots, void *codes, float *scales,
                           const int *cache_slots, int N, int n_slots, int n_cache, int Hv, int dk, int dv,
                           gdn_code code, void *stream)
{
    gdn_status st = check_cache(state_pool, slots, codes, scales, cache_slots, N, n_slots, n_cache, Hv, dk, dv, code);
    if (st != GDN_OK || N == 0) return st;
    gdn::StateCacheArgs a{state_pool, nullptr, slots, cache_slots, codes, scales, N, n_slots, n_cache, Hv};
    return launch_status(gdn::launch_state_store(a, code, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_state_load(const void *codes, const float *scales, const int *cache_slots, float *state_pool,
                          const int *slots, int N, int n_slots, int n_cache, int Hv, int dk, int dv, gdn_code code,
                          void *stream)
{
    gdn_status st = check_cache(state_pool, slots, codes, scales, cache_slots, N, n_slots, n_cache, Hv, dk, dv, code);
    if (st != GDN_OK || N == 0) return st;
    gdn::StateCacheArgs a{nullptr, state_pool, slots, cache_slots, const_cast<void *>(codes),
                          const_cast<float *>(scales), N, n_slots, n_cache, Hv};
    return launch_status(gdn::launch_state_load(a, code, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
