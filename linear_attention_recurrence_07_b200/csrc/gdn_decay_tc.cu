// Linear attention with a constant decay per head on the 5th-generation tensor cores
// (bf16 operands, fp32 state): the walk that prefill and all gradients share (see
// DecayWalk), chunk by chunk.
//
// Per chunk of L <= 64 tokens, H the state at its start (decayed to its first token),
// p_i = i forwards, L - 1 - i backwards:
//   G    = X Y^T                                        M=64  N=64  K=128
//   P_ij = lambda^{|i-j|} G_ij, j at or before i        (bf16)
//   OX^T = H^T X^T   (H^T in two bf16 pieces)           M=128 N=64  K=2x128
//   OI^T = Z^T P^T                                      M=128 N=64  K=64
//   O    = diag(lambda^p) OX + OI
//   D^T  = Z'^T Y, Z' = diag(lambda^{L-p}) Z in three bf16 pieces (all 24 bits)
//                                                       M=128 N=128 K=3x64
//   H^T <- lambda^L H^T + D^T                           (fp32 registers)
// Unlike the delta rule, D does not depend on the state: the chain from chunk to chunk
// is one fused multiply-add per state element.  The state therefore lives in registers
// (64 per thread over 256 threads), and only its two bf16 pieces go to the tensor core.
// Its rounding: the pieces drop 2^-17 of the state in O (a bf16 result); D enters the
// state with all its bits, small pieces first, because the tensor core truncates when
// it accumulates.  P is rounded to bf16 once, like every operand of a bf16 attention.
//
// One CTA per (sequence or segment, V head), warp-specialised:
//   warp 0      TMA producer: X, Y, Z tiles, four stages of 48 KB
//   warp 1      MMA issuer (one thread), event-driven: D, OX, OI, G as inputs get ready
//   warps 2-9   state: thread = TMEM lane (z dimension) and half of the 128 columns;
//               decays Z into its pieces (TMEM), adds D to the state, writes its pieces
//   warps 10-13 output: G -> P (shared memory), O epilogue (stmatrix, TMA store)
// Bound: 1 KiB of HBM traffic per token and head against about 1700 tensor cycles and
// 1500 issue slots per chunk and SM; the loads are four chunks ahead.
#include "tc_common.cuh"
#include "decay_common.cuh"

namespace gdn {
namespace {

constexpr int kDtThreads = 448;
constexpr int kStages = 4;
constexpr uint32_t kStageBytes = 6 * TILE;            // [X0][X1][Y0][Y1][Z0][Z1], 64 columns each

// TMEM columns
constexpr uint32_t T_D = 0;        // D^T, 128 fp32 columns
constexpr uint32_t T_H = 128;      // H^T pieces: high at 128, low at 192 (64 packed columns each)
constexpr uint32_t T_Z = 256;      // Z'^T pieces, 32 packed columns each
constexpr uint32_t T_G = 352;      // G, then OI^T (G is read before the OI MMAs are issued)
constexpr uint32_t T_OX = 416;     // OX^T
constexpr uint32_t T_COLS = 512;

constexpr uint32_t DOFF_P = kStages * kStageBytes;
constexpr uint32_t DOFF_O = DOFF_P + TILE;
constexpr uint32_t DOFF_TAB = DOFF_O + 2 * TILE;      // pw[0..64]; wtab[2][64]; gtab[2][64]
constexpr uint32_t TAB_FLOATS = 68 + 4 * 64;
constexpr uint32_t DOFF_BAR = DOFF_TAB + TAB_FLOATS * 4;
enum : int {
    D_FULL = 0,                    // x4: tiles of a stage landed
    D_EMPTY = 4,                   // x4: stage no longer read
    D_ZP = 8,                      // Z' pieces written, D of the chunk before read (8 warps)
    D_DFULL = 9,                   // D done
    D_HREADY = 10,                 // pieces of H written (8 warps)
    D_XFULL = 11,                  // OX done
    D_GFULL = 12,                  // G done
    D_PREADY = 13,                 // P written, G read (4 warps)
    D_OFULL = 14,                  // OX and OI done
    D_OFREE = 15,                  // OX and OI read (4 warps)
    D_DRAIN = 16,
    D_NBAR = 17
};
constexpr uint32_t DOFF_MISC = DOFF_BAR + D_NBAR * 8;
constexpr uint32_t D_SMEM = DOFF_MISC + 16 + 1024;
static_assert(D_SMEM <= 232448, "shared memory per CTA");
static_assert(DOFF_TAB % 16 == 0 && DOFF_BAR % 8 == 0, "alignment");

constexpr uint32_t IDD_G = idesc_bf16(64, 64, false, false);
constexpr uint32_t IDD_OX = idesc_bf16(128, 64, false, false);
constexpr uint32_t IDD_OI = idesc_bf16(128, 64, true, false);
constexpr uint32_t IDD_D = idesc_bf16(128, 128, false, true);

struct DecayCtl {
    uint64_t *bar;
    volatile int *abort_flag;
    // All lanes of the warp wait; the answer is the same for all of them.  Roles that meet at
    // a named barrier agree on it there before any of them leaves.
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        const bool got = mbar_try_wait(&bar[i], parity) || wait_loop(i, parity);
        return __all_sync(0xffffffffu, got);
    }
    __device__ __noinline__ bool wait_loop(int i, uint32_t parity) const {
        const long long t0 = clock64();
        for (;;) {
            if (mbar_try_wait_suspend(&bar[i], parity, 20000)) return true;
            if (*abort_flag) return false;
            if (clock64() - t0 > (1ll << 32)) {
                *abort_flag = 1;
                atomicOr(&g_tc_error, 1u);
                return false;
            }
        }
    }
};

// Upper 16 bits of two floats as a bf16 pair, and their exact remainders.
__device__ __forceinline__ uint32_t split_pair(float &a, float &b) {
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    a -= __uint_as_float(ua & 0xffff0000u);
    b -= __uint_as_float(ub & 0xffff0000u);
    return __byte_perm(ua, ub, 0x7632);
}

// Rows of O from the accumulators one column (token) at a time: ragged chunks of packed
// sequences, and fp32 partial rows (a warp writes 32 consecutive values of a row).
template <typename OT>
__device__ __noinline__ void store_rows(OT *dst, uint32_t t_lane, const float *gt, int rows, size_t stride) {
#pragma unroll 1
    for (int r0 = 0; r0 < C; r0 += 32) {
        float x[32], y[32];
        tmem_ld32(t_lane + T_OX + r0, x);
        tmem_ld32(t_lane + T_G + r0, y);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (r0 + e < rows) dst[(size_t)(r0 + e) * stride] = from_f32<OT>(fmaf(gt[r0 + e], x[e], y[e]));
    }
}

__global__ void __launch_bounds__(kDtThreads, 1)
decay_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_o,
                const DecayWalk w, const int state_only)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + DOFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + DOFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + DOFF_MISC + 4);
    float *pw = reinterpret_cast<float *>(sm + DOFF_TAB);   // lambda^0 .. lambda^64
    float *wtab = pw + 68, *gtab = wtab + 128;               // [0]: full chunks, [1]: the special one
    const DecayCtl ctl{bar, abort_flag};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x;
    const WalkSpan sp = walk_span(w, blockIdx.y, state_only != 0);
    const int n = sp.c1 - sp.c0;                             // chunks of this CTA
    const uint32_t sbase = smem_u32(sm);
    const size_t hstate = (size_t)kHeadDim * kHeadDim;

    // The one chunk that is not like the others: the sequence's last one, which may be ragged and
    // whose end state may be wanted undecayed.  It is the walk's last (forwards) or first (backwards).
    const int special = w.rev ? 0 : sp.nchunks - 1;
    const int tail = sp.L - (sp.nchunks - 1) * C;
    const int back = (w.fin_back && !state_only) ? 1 : 0;
    const double loglam = decay_log(w.decay[h]);

    if (tid == 0) {
        if (!state_only) { prefetch_tensormap(&tm_x); prefetch_tensormap(&tm_o); }
        prefetch_tensormap(&tm_y);
        prefetch_tensormap(&tm_z);
        for (int i = 0; i < (int)D_NBAR; ++i)
            mbar_init(&bar[i], i == D_ZP || i == D_HREADY ? 8 : i == D_PREADY || i == D_OFREE ? 4 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, T_COLS);
        tmem_relinquish();
    }
    for (int i = tid - 64; i >= 0 && i < 65 + 256; i += kDtThreads) {
        if (i < 65) {
            pw[i] = (float)decay_pow(loglam, i);
        } else {
            const int t = (i - 65) & 63, which = (i - 65) >> 6;          // w full, w special, g full, g special
            const int L = (which & 1) ? tail : C, bk = (which & 1) ? back : 0;
            int e;
            if (which < 2) e = w.rev ? t + 1 : L - t - bk;
            else e = w.rev ? L - 1 - t : t;
            (which < 2 ? wtab : gtab)[(which & 1) * 64 + t] = (float)decay_pow(loglam, max(e, 0));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ======================================================== TMA producer
        if (lane == 0) {
            const int hx = h / (w.Hv / w.hx), hy = h / (w.Hv / w.hy), hz = h / (w.Hv / w.hz);
            int c = 0;
            for (; c < n; ++c) {
                const int s = c % kStages;
                if (c >= kStages) {
                    bool got = mbar_try_wait(&bar[D_EMPTY + s], ((c / kStages) - 1) & 1) ||
                               ctl.wait_loop(D_EMPTY + s, ((c / kStages) - 1) & 1);
                    if (!got) break;
                }
                int t0;
                chunk_rows(sp, w.rev, sp.c0 + c, t0);
                unsigned char *st = sm + s * kStageBytes;
                uint64_t *full = &bar[D_FULL + s];
                mbar_arrive_expect_tx(full, state_only ? 4 * TILE : kStageBytes);
                tma_load_4d(st + 2 * TILE, &tm_y, full, 0, hy, t0, sp.bt);
                tma_load_4d(st + 3 * TILE, &tm_y, full, 64, hy, t0, sp.bt);
                tma_load_4d(st + 4 * TILE, &tm_z, full, 0, hz, t0, sp.bt);
                tma_load_4d(st + 5 * TILE, &tm_z, full, 64, hz, t0, sp.bt);
                if (!state_only) {
                    tma_load_4d(st + 0 * TILE, &tm_x, full, 0, hx, t0, sp.bt);
                    tma_load_4d(st + 1 * TILE, &tm_x, full, 64, hx, t0, sp.bt);
                }
            }
            // On an abort, copies still in flight land before the CTA's memory goes away.
            if (*abort_flag)
                for (int i = max(0, c - kStages); i < c; ++i)
                    mbar_wait(&bar[D_FULL + i % kStages], (i / kStages) & 1, 1ll << 28);
        }
    } else if (warp == 1) {
        // ======================================================== MMA issuer
        if (lane == 0) {
            int ng = 0, nd = 0, nx = 0, np = 0, ne = 0;
            if (state_only) ng = nx = np = n;
            long long idle_since = clock64();
            while (nd < n || np < n || nx < n) {
                if (*abort_flag) break;
                bool issued = false;
                if (nd < n && mbar_test(&bar[D_ZP], nd & 1)) {
                    // Z' written implies its tiles landed and D of the chunk before read
                    const uint32_t st = sbase + (nd % kStages) * kStageBytes;
                    tc_fence_after();
#pragma unroll
                    for (int pc = 2; pc >= 0; --pc)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ts(tmem + T_D, tmem + T_Z + pc * 32 + k * 8,
                                        smem_desc_sw128(st + 2 * TILE + k * 2048, TILE, 1024), IDD_D, pc < 2 || k > 0);
                    mma_commit(&bar[D_DFULL]);
                    ++nd;
                    issued = true;
                } else if (np < ng && mbar_test(&bar[D_PREADY], np & 1)) {
                    const uint32_t st = sbase + (np % kStages) * kStageBytes;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + T_G, smem_desc_sw128(st + 4 * TILE + k * 2048, TILE, 1024),
                                 smem_desc_sw128(sbase + DOFF_P + k * 32, 16, 1024), IDD_OI, k > 0);
                    ++np;
                    if (nx >= np) mma_commit(&bar[D_OFULL]);
                    issued = true;
                } else if (nx < n && mbar_test(&bar[D_HREADY], nx & 1) &&
                           mbar_test(&bar[D_FULL + nx % kStages], (nx / kStages) & 1) &&
                           (nx < 1 || mbar_test(&bar[D_OFREE], (nx - 1) & 1))) {
                    const uint32_t st = sbase + (nx % kStages) * kStageBytes;
                    tc_fence_after();
#pragma unroll
                    for (int pc = 1; pc >= 0; --pc)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16_ts(tmem + T_OX, tmem + T_H + pc * 64 + k * 8,
                                        smem_desc_sw128(st + (k >> 2) * TILE + (k & 3) * 32, 16, 1024), IDD_OX,
                                        pc < 1 || k > 0);
                    mma_commit(&bar[D_XFULL]);
                    ++nx;
                    if (np >= nx) mma_commit(&bar[D_OFULL]);
                    issued = true;
                } else if (ng < n && mbar_test(&bar[D_FULL + ng % kStages], (ng / kStages) & 1) &&
                           (ng < 1 || mbar_test(&bar[D_OFREE], (ng - 1) & 1)) &&
                           // rows past a packed sequence's end are zeroed before Z' is announced
                           (!w.cu_seqlens || ng < nd)) {
                    const uint32_t st = sbase + (ng % kStages) * kStageBytes;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t koff = (k >> 2) * TILE + (k & 3) * 32;
                        mma_bf16(tmem + T_G, smem_desc_sw128(st + koff, 16, 1024),
                                 smem_desc_sw128(st + 2 * TILE + koff, 16, 1024), IDD_G, k > 0);
                    }
                    mma_commit(&bar[D_GFULL]);
                    ++ng;
                    issued = true;
                }
                while (ne < nd && ne < np && ne < nx) {          // every read of the stage is issued
                    mma_commit(&bar[D_EMPTY + ne % kStages]);
                    ++ne;
                }
                if (issued) {
                    idle_since = clock64();
                } else {
                    __nanosleep(32);
                    if (clock64() - idle_since > (1ll << 32)) {
                        *abort_flag = 1;
                        atomicOr(&g_tc_error, 1u);
                        break;
                    }
                }
            }
            mma_commit(&bar[D_DRAIN]);
            mbar_wait(&bar[D_DRAIN], 0, 1ll << 30);
        }
    } else if (warp < 10) {
        // ======================================================== state
        const int q4 = warp & 3, hf = (warp - 2) >> 2;
        const int dz = q4 * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(q4 * 32) << 16);
        float H[64];                                         // H^T[dz][64 hf + e]
#pragma unroll
        for (int e = 0; e < 64; ++e) H[e] = 0.f;
        if (w.nseg > 1 && !state_only) {
            const int here = tokens_before(sp, w.rev, sp.c0);
#pragma unroll 1
            for (int g = 0; g <= sp.seg; ++g) {
                const float f = (float)decay_pow(loglam, here - tokens_before(sp, w.rev, g * w.seg_chunks));
                const float *src = w.seg + (((size_t)sp.b * w.nseg + g) * w.Hv + h) * hstate + (size_t)64 * hf * kHeadDim + dz;
#pragma unroll
                for (int e = 0; e < 64; ++e) H[e] = fmaf(f, src[(size_t)e * kHeadDim], H[e]);
            }
        } else if (w.init && (!state_only || sp.copy_init)) {
            const float f = (w.init_decays && sp.L > 0) ? pw[1] : 1.f;
            const float *src = w.init + ((size_t)sp.b * w.Hv + h) * hstate;
            if (w.init_trans) {
                const float4 *row = reinterpret_cast<const float4 *>(src + (size_t)dz * kHeadDim + 64 * hf);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 v = row[e];
                    H[4 * e] = f * v.x; H[4 * e + 1] = f * v.y; H[4 * e + 2] = f * v.z; H[4 * e + 3] = f * v.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 64; ++e) H[e] = f * src[(size_t)(64 * hf + e) * kHeadDim + dz];
            }
        }
        auto write_pieces = [&]() {
#pragma unroll
            for (int e0 = 0; e0 < 64; e0 += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float a = H[e0 + 2 * e], b = H[e0 + 2 * e + 1];
                    hi[e] = split_pair(a, b);
                    lo[e] = pack_bf16x2(a, b);
                }
                tmem_st16u(t_lane + T_H + 32 * hf + (e0 >> 1), hi);
                tmem_st16u(t_lane + T_H + 64 + 32 * hf + (e0 >> 1), lo);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_HREADY]);
        };
        // Z'^T pieces of this thread's 32 tokens, from column dz of the Z tile
        auto write_z = [&](int c) -> bool {
            const int s = c % kStages;
            if (!ctl.wait(D_FULL + s, (c / kStages) & 1)) return false;
            unsigned char *st = sm + s * kStageBytes;
            int t0;
            const int cw = sp.c0 + c, rows = chunk_rows(sp, w.rev, cw, t0);
            if (w.cu_seqlens && rows < C) {                  // the next sequence's rows: out of the products
                for (int i = tid - 64; i < (C - rows) * 4 * 8; i += 256) {
                    const int r = rows + (i >> 5), tile = (i >> 3) & 3, ch = i & 7;
                    *reinterpret_cast<uint4 *>(st + (2 + tile) * TILE + r * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            const float *wt = wtab + (cw == special ? 64 : 0) + 32 * hf;
            const unsigned char *zt = st + (4 + (dz >> 6)) * TILE;
            const uint32_t zc = (dz & 63) >> 3, zb = (dz & 7) * 2;
#pragma unroll
            for (int b0 = 0; b0 < 32; b0 += 16) {
                uint32_t p0[8], p1[8], p2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = 32 * hf + b0 + 2 * e;
                    const float2 ww = *reinterpret_cast<const float2 *>(wt + b0 + 2 * e);
                    const uint32_t ua = *reinterpret_cast<const uint16_t *>(zt + t * 128 + ((zc ^ (t & 7)) << 4) + zb);
                    const uint32_t ub = *reinterpret_cast<const uint16_t *>(zt + (t + 1) * 128 + ((zc ^ ((t + 1) & 7)) << 4) + zb);
                    float a = t < rows ? ww.x * __uint_as_float(ua << 16) : 0.f;
                    float b = t + 1 < rows ? ww.y * __uint_as_float(ub << 16) : 0.f;
                    p0[e] = split_pair(a, b);
                    p1[e] = split_pair(a, b);
                    p2[e] = split_pair(a, b);
                }
                const uint32_t col = t_lane + T_Z + 16 * hf + (b0 >> 1);
                tmem_st8u(col, p0);
                tmem_st8u(col + 32, p1);
                tmem_st8u(col + 64, p2);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_ZP]);
            return true;
        };
        bool ok = true;
        if (n > 0) {
            if (!state_only) write_pieces();
            ok = write_z(0);
        }
        const double p64 = decay_pow(loglam, C), psp = decay_pow(loglam, tail - back);
        const float fh = (float)p64, fl = (float)(p64 - (double)fh);
        const float sh = (float)psp, sl = (float)(psp - (double)sh);
        for (int c = 0; c < n && ok; ++c) {
            ok = ctl.wait(D_DFULL, c & 1);
            if (!ok) break;
            tc_fence_after();
            const bool is_special = sp.c0 + c == special;
            const float ph = is_special ? sh : fh, pl = is_special ? sl : fl;
#pragma unroll
            for (int e0 = 0; e0 < 64; e0 += 32) {
                float d[32];
                tmem_ld32(t_lane + T_D + 64 * hf + e0, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) H[e0 + e] = fmaf(ph, H[e0 + e], fmaf(pl, H[e0 + e], d[e]));
            }
            tc_fence_before();
            if (c + 1 < n) {
                if (!(ok = write_z(c + 1))) break;
                if (!state_only) {
                    if (!(ok = ctl.wait(D_XFULL, c & 1))) break;
                    tc_fence_after();
                    write_pieces();
                }
            }
        }
        float *dst = nullptr;
        if (state_only) dst = w.seg + (((size_t)sp.b * w.nseg + sp.seg) * w.Hv + h) * hstate;
        else if (w.fin && sp.c1 == sp.nchunks) dst = w.fin + ((size_t)sp.b * w.Hv + h) * hstate;
        if (ok && dst) {
#pragma unroll
            for (int e = 0; e < 64; ++e) dst[(size_t)(64 * hf + e) * kHeadDim + dz] = H[e];
        }
    } else if (!state_only) {
        // ======================================================== output
        const int q4 = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(q4 * 32) << 16);
        const bool leader = tid == 320;
        const int g = lane >> 2, t = lane & 3;
        const size_t stride = (size_t)w.Hv * kHeadDim;
        bool ok = true;
        for (int c = 0; c < n && ok; ++c) {
            // ---- G -> P: M = 64 accumulators sit in lanes 0-15 of every quarter
            if (!(ok = named_and(2, 128, ctl.wait(D_GFULL, c & 1)))) break;
            tc_fence_after();
            {
                uint32_t ra[16], rb[16];
                tmem_ld16x256b_x4(t_lane + T_G, ra);
                tmem_ld16x256b_x4(t_lane + T_G + 32, rb);
                tmem_wait_ld();
                unsigned char *pt = sm + DOFF_P;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = 16 * q4 + g + 8 * half;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t *rr = k < 4 ? ra : rb;
                        const int j = 8 * k + 2 * t, kk = k & 3;
                        const int e = w.rev ? j - i : i - j, e1 = w.rev ? e + 1 : e - 1;
                        const float a = e >= 0 ? pw[max(e, 0)] * __uint_as_float(rr[4 * kk + 2 * half]) : 0.f;
                        const float b = e1 >= 0 ? pw[max(e1, 0)] * __uint_as_float(rr[4 * kk + 2 * half + 1]) : 0.f;
                        *reinterpret_cast<uint32_t *>(pt + i * 128 + ((k ^ (i & 7)) << 4) + 4 * t) = pack_bf16x2(a, b);
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_PREADY]);
            // ---- O
            if (leader) bulk_wait_group_read0();             // the store before has read the staging tile
            if (!(ok = named_and(2, 128, ctl.wait(D_OFULL, c & 1)))) break;
            tc_fence_after();
            int t0;
            const int cw = sp.c0 + c, rows = chunk_rows(sp, w.rev, cw, t0);
            const float *gt = gtab + (cw == special ? 64 : 0);
            const size_t at = ((size_t)sp.bt * w.T + t0) * stride + (size_t)h * kHeadDim + q4 * 32 + lane;
            if (w.o_f32) {
                store_rows(static_cast<float *>(w.o) + at, t_lane, gt, rows, stride);
            } else if (rows < C && w.cu_seqlens) {
                store_rows(static_cast<__nv_bfloat16 *>(w.o) + at, t_lane, gt, rows, stride);
            } else {
                const uint32_t stage = smem_u32(sm + DOFF_O);
                const int mt = lane >> 3, mi = lane & 7;     // stored row mi of matrix mt
#pragma unroll 1
                for (int it = 0; it < 4; ++it) {             // 16-lane slab, 32-token block
                    const int slab = it >> 1, cb = it & 1;
                    uint32_t rx[16], ri[16];
                    const uint32_t ta = t_lane + ((uint32_t)(16 * slab) << 16) + 32 * cb;
                    tmem_ld16x256b_x4(ta + T_OX, rx);
                    tmem_ld16x256b_x4(ta + T_G, ri);
                    tmem_wait_ld();
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t m[4];
#pragma unroll
                        for (int mm = 0; mm < 4; ++mm) {
                            const int k = 2 * kk + (mm >> 1), gg = mm & 1;
                            const float2 gm = *reinterpret_cast<const float2 *>(gt + 32 * cb + 8 * k + 2 * t);
                            m[mm] = pack_bf16x2(
                                fmaf(gm.x, __uint_as_float(rx[4 * k + 2 * gg]), __uint_as_float(ri[4 * k + 2 * gg])),
                                fmaf(gm.y, __uint_as_float(rx[4 * k + 2 * gg + 1]), __uint_as_float(ri[4 * k + 2 * gg + 1])));
                        }
                        const int k = 2 * kk + (mt >> 1), gg = mt & 1;
                        const int orow = 32 * cb + 8 * k + mi;          // token
                        const int jst = q4 * 32 + 16 * slab + 8 * gg;   // first z of the block
                        stmatrix_x4_trans(stage + (jst >> 6) * TILE + sw128_chunk(orow, (jst & 63) >> 3),
                                          m[0], m[1], m[2], m[3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_OFREE]);
            if (!w.o_f32 && !(rows < C && w.cu_seqlens)) {
                fence_proxy_async_smem();
                named_sync(2, 128);
                if (leader) {
                    tma_store_4d(&tm_o, sm + DOFF_O, 0, h, t0, sp.bt);
                    tma_store_4d(&tm_o, sm + DOFF_O + TILE, 64, h, t0, sp.bt);
                    bulk_commit_group();
                }
            }
        }
        if (leader) bulk_wait_group0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, T_COLS);
    }
}

}  // namespace

cudaError_t decay_tc_take_error(unsigned *out)
{
    unsigned v = 0, zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_tc_error, sizeof(v));
    if (err == cudaSuccess && v) err = cudaMemcpyToSymbol(g_tc_error, &zero, sizeof(zero));
    *out = v;
    return err;
}

cudaError_t launch_decay_walk_tc(const DecayWalk &w, cudaStream_t stream)
{
    CUtensorMap tx, ty, tz, to;
    const int rows_b = w.cu_seqlens ? 1 : w.B;   // batch rows of the token arrays
    if (!make_map(&tx, w.x, rows_b, w.T, w.hx) || !make_map(&ty, w.y, rows_b, w.T, w.hy) ||
        !make_map(&tz, w.z, rows_b, w.T, w.hz))
        return cudaErrorInvalidValue;
    if (w.o_f32) to = tx;                        // not used
    else if (!make_map(&to, w.o, rows_b, w.T, w.Hv)) return cudaErrorInvalidValue;
    cudaError_t err = cudaFuncSetAttribute(decay_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)D_SMEM);
    if (err != cudaSuccess) return err;
    const dim3 grid((unsigned)w.Hv, (unsigned)(w.B * w.nseg));
    if (w.nseg > 1) {
        decay_tc_kernel<<<grid, kDtThreads, D_SMEM, stream>>>(tx, ty, tz, to, w, 1);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    decay_tc_kernel<<<grid, kDtThreads, D_SMEM, stream>>>(tx, ty, tz, to, w, 0);
    return cudaGetLastError();
}

}  // namespace gdn
