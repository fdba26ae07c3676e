// Linear attention with a constant decay per head on the 5th-generation tensor cores
// (bf16 operands, fp32 state): the walk that prefill and all gradients share (see
// DecayWalk), chunk by chunk.
//
// Per chunk of L <= 64 tokens, H the state at its start (decayed to its first token),
// p_i = i forwards, L - 1 - i backwards:
//   G    = X Y^T                                        M=64  N=64  K=128
//   P_ij = lambda^{-p_j} G_ij, j at or before i         (NP bf16 pieces)
//   O^T  = (H^T X^T + Z^T P^T) diag(lambda^p)           M=128 N=64  K=128 + NP x 64
//   D^T  = Z'^T Y, Z' = diag(lambda^{L-p}) Z in NZ bf16 pieces
//                                                       M=128 N=128 K=NZ x 64
//   H^T <- lambda^L H^T + D^T                           (fp32 registers)
// Unlike the delta rule, D does not depend on the state: the chain from chunk to chunk
// is one fused multiply-add per state element.  The state therefore lives in registers
// (64 per thread over 256 threads), and only its bf16 rounding goes to the tensor core.
//
// Roundings: H and P are rounded to bf16 where they meet X and Z, as every operand of a bf16
// product: the terms of a row average it out to about the rounding of O itself.  Sequences of
// one chunk, whose first rows have few terms and no H, get 16 bits of P in two pieces (they
// are bound by latency, and the pieces share the room of P's second buffer).  Z' has three
// pieces, all 24 bits, where an end state is wanted, two where the state only feeds O; small
// pieces are accumulated first, because the tensor core truncates.
//
// Range.  lambda^{-p_j} grows to lambda^{-63}: below lambda = 2^-(100/63) the scale is held at
// 2^100, which replaces a factor lambda^p < 2^-100 on H's share of a row by 2^-100.  Heads whose
// scales span more than 40 bits are centred: state, Z' and P carry 2^-s and the scale of O 2^s, s
// half of the span and at most 40 (powers of two, in the tables and at the walk's ends only, so
// the results' bits are the same).  Scores and sums stay finite to 2^67 (2^28 uncentred), those
// that the causal mask multiplies by zero too, and a state keeps its 24 bits down to 2^-64.
//
// One CTA per (sequence or segment, V head), warp-specialised:
//   warp 0      TMA producer: X, Y, Z tiles, four stages of 48 KB
//   warp 1      issues the D MMAs, warp 2 the G and O MMAs (one elected thread each, in order)
//   warps 4-11  state: thread = TMEM lane (z dimension) and half of the 128 columns;
//               writes the decayed pieces of Z^T to TMEM, adds D to the state, writes H
//   warps 12-15 G -> P (shared memory)
//   warps 16-19 O epilogue (stmatrix, TMA store)
//
// Measured: 16 QK / 48 V heads, B=8, T=8192: 0.67-0.69 ms, 3.3 TB/s (half of the copy
// bandwidth), 300 TF/s of the recurrence's own arithmetic; B=1, T=4096: 64 us (a head and
// three segments); gradients at 48 heads, T=4096: 129-132 us.  A chunk takes 2400 to 2700
// cycles per SM (the clock settles at 1.65 GHz under this load).  No single unit bounds it: the
// chain from D through the state's registers to the next D (pieces of Z 1100, reading D 550, H
// 280 cycles of its two warpgroups, and D itself), the tensor core 55-65% of the time (65 cycles
// per 128 x 128 x 16 MMA make 780 for D; H X 270, Z P 200, G 280), shared memory 70%.  Giving Z'
// warps of its own, Z' or O a second buffer, or Z P a place before H X was no faster: what runs
// earlier takes the tensor core from D.
// What counted on the way: no spills (setmaxnreg; 1.6 times), MMAs issued by an elected lane,
// and the size of the loops: unrolled roles of 98 KB of code waited for instructions a quarter
// of the time.
#include <type_traits>

#include "tc_common.cuh"
#include "decay_common.cuh"

namespace gdn {
namespace {

constexpr int kDtThreads = 640;
constexpr int kStages = 4;
constexpr uint32_t kStageBytes = 6 * TILE;            // [X0][X1][Y0][Y1][Z0][Z1], 64 columns each

// TMEM columns
constexpr uint32_t T_D = 0;        // D^T, 128 fp32 columns
constexpr uint32_t T_H = 128;      // H^T rounded, 64 packed columns
constexpr uint32_t T_Z = 192;      // Z'^T pieces, 32 packed columns each
constexpr uint32_t T_G = 288;      // two buffers of 64, chunk c uses c % 2
constexpr uint32_t T_O = 416;
constexpr uint32_t T_COLS = 512;

constexpr uint32_t DOFF_P = kStages * kStageBytes;    // two buffers, chunk c uses c % 2, or the two pieces
constexpr uint32_t DOFF_O = DOFF_P + 2 * TILE;
constexpr uint32_t DOFF_TAB = DOFF_O + 2 * TILE;      // powers; per token: Z weights, O scales, P scales
constexpr uint32_t TAB_PW = 0, TAB_W = 66, TAB_F = 66 + 128, TAB_C = 66 + 256, TAB_L = 66 + 3 * 128,
                   TAB_FLOATS = TAB_L + 6;     // TAB_L: lambda^L twice (two floats each), factors of start and end state
constexpr uint32_t DOFF_BAR = DOFF_TAB + TAB_FLOATS * 4;
enum : int {
    D_FULL = 0,                    // x4: tiles of a stage landed
    D_EMPTY = 4,                   // x4: stage no longer read (both issuers)
    D_ZP = 8,                      // Z' written, D of the chunk before read (8 warps)
    D_DFULL = 9,                   // D done
    D_HREADY = 10,                 // H written (8 warps)
    D_XFULL = 11,                  // H's share of O done
    D_OFREE = 12,                  // O read (4 warps)
    D_DRAIN = 13,                  // last MMAs of both issuers
    // x2, chunk c uses c % 2: P's warps run up to a chunk ahead of the MMAs, and on one barrier
    // the phase after the awaited one could have completed by the time of the wait.
    D_GFULL = 14,                  // G done
    D_PREADY = 16,                 // P written, G read (4 warps)
    D_OFULL = 18,                  // O done
    D_CUT = 20,                    // once: rows behind a packed sequence are zeros (8 warps)
    D_NBAR = 21
};
constexpr uint32_t DOFF_MISC = DOFF_BAR + D_NBAR * 8;
constexpr uint32_t D_SMEM = DOFF_MISC + 8 + 1024;
static_assert(D_SMEM <= 232448, "shared memory per CTA");
static_assert(DOFF_TAB % 16 == 0 && DOFF_BAR % 8 == 0, "alignment");

constexpr uint32_t IDD_G = idesc_bf16(64, 64, false, false);
constexpr uint32_t IDD_OX = idesc_bf16(128, 64, false, false);
constexpr uint32_t IDD_OI = idesc_bf16(128, 64, true, false);
constexpr uint32_t IDD_D = idesc_bf16(128, 128, false, true);
// Registers per thread: 640 x 96 at launch; the warpgroups without state give part of their
// share to the two that hold it (a spilled register is an L2 round trip here, because the
// shared memory leaves no L1): 40 + 2 x 160 + 2 x 56 <= 5 x 96.
constexpr int kRegsIssue = 40, kRegsState = 160, kRegsP = 56, kRegsOut = 56;
constexpr double kScaleFloor = -69.31471805599453;    // log of 2^-100
constexpr float kScaleMin = 7.8886091e-31f;           // 2^-100
constexpr double kCentred = -27.725887222397812;      // log of 2^-40

template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

struct DecayCtl {
    uint64_t *bar;
    volatile int *abort_flag;
    const DecayWalks &d;
    // One thread.  (Inlined and short: a call would not let ptxas give the roles their own
    // register counts, and the loops of all roles share the instruction cache; a limit in clocks
    // cost 4% of a long prefill.)  The second of two launches may count against its limit what the
    // first has left, at most the walk of a segment.
    __device__ __forceinline__ bool wait_one(int i, uint32_t parity) const {
        bool got = mbar_try_wait(&bar[i], parity);
#pragma unroll 1
        for (int k = d.wait_tries; !got && k > 0; --k) {
            got = mbar_try_wait_suspend(&bar[i], parity, kWaitTryMicros * 1000);
            if (*abort_flag) k = 0;
        }
        if (!got) *abort_flag = 1;
        return got;
    }
    // All lanes of the warp wait; the answer is the same for all of them.  Roles that meet at
    // a named barrier agree on it there before any of them leaves.
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        return __all_sync(0xffffffffu, wait_one(i, parity));
    }
};

// Two floats rounded to a bf16 pair.
__device__ __forceinline__ uint32_t round_pair(uint64_t v) {
    float a, b;
    unpack2(v, a, b);
    return pack_bf16x2(a, b);
}
// The rounded pair, and in v what it leaves over (exact: at most 16 bits of an fp32).
__device__ __forceinline__ uint32_t split_pair(uint64_t &v) {
    const uint32_t p = round_pair(v);
    v = sub2(v, pack2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)));
    return p;
}

// Kernel argument: the walks and their tensor maps (x, y, z, o).
struct TcWalks {
    CUtensorMap maps[kMaxWalks][4];
    DecayWalks d;
};

// Rows of O from the accumulators one column (token) at a time: ragged chunks of packed
// sequences, whose rows past the end belong to others.
__device__ __forceinline__ void store_rows(__nv_bfloat16 *dst, uint32_t t_lane, const float *gt, int rows, size_t stride) {
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
        float x[8];
        tmem_ld8(t_lane + T_O + r0, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r0 + e < rows) dst[(size_t)(r0 + e) * stride] = __float2bfloat16_rn(gt[r0 + e] * x[e]);
    }
}

// FIRST: the first launch of a segmented walk.  NZ, NP: pieces of Z' and of P; NP = 0: two for
// sequences of one chunk, else one.
template <bool FIRST, int NZ, int NP>
__global__ void __launch_bounds__(kDtThreads, 1)
decay_tc_kernel(const __grid_constant__ TcWalks p)
{
    const DecayWalk &w = p.d.w[blockIdx.z];
    const CUtensorMap &tm_x = p.maps[blockIdx.z][0], &tm_y = p.maps[blockIdx.z][1], &tm_z = p.maps[blockIdx.z][2],
                      &tm_o = p.maps[blockIdx.z][3];
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + DOFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + DOFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + DOFF_MISC + 4);
    float *tab = reinterpret_cast<float *>(sm + DOFF_TAB);
    float *seg_decay = reinterpret_cast<float *>(sm + DOFF_O);       // read before any O
    const DecayCtl ctl{bar, abort_flag, p.d};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x;
    const WalkSpan sp = walk_span(w, blockIdx.y, FIRST);
    const bool state_only = FIRST && sp.state_only;
    const int n = sp.c1 - sp.c0;                             // chunks of this CTA
    const bool fine = NP == 2 || (NP == 0 && sp.nchunks == 1);   // P in two pieces
    if (FIRST) let_next_launch_start();
    const uint32_t sbase = smem_u32(sm);
    const size_t hstate = (size_t)kHeadDim * kHeadDim;

    // The one chunk that is not like the others: the sequence's last one, which may be ragged and
    // whose end state may be wanted undecayed.  It is the walk's last (forwards) or first (backwards).
    const int special = w.rev ? 0 : sp.nchunks - 1;
    const int tail = sp.L - (sp.nchunks - 1) * C;
    const int back = (w.fin_back && !FIRST) ? 1 : 0;

    // The first stages' tiles, in flight while the rest is set up (only this thread waits on D_EMPTY).
    auto load_stage = [&](int c) {
        const int s = c % kStages;
        int t0;
        chunk_rows(sp, w.rev, sp.c0 + c, t0);
        unsigned char *st = sm + s * kStageBytes;
        uint64_t *full = &bar[D_FULL + s];
        const int hx = h / (w.Hv / w.hx), hy = h / (w.Hv / w.hy), hz = h / (w.Hv / w.hz);
        mbar_arrive_expect_tx(full, state_only ? 4 * TILE : kStageBytes);
        tma_load_4d(st + 2 * TILE, &tm_y, full, 0, hy, t0, sp.bt);
        tma_load_4d(st + 3 * TILE, &tm_y, full, 64, hy, t0, sp.bt);
        tma_load_4d(st + 4 * TILE, &tm_z, full, 0, hz, t0, sp.bt);
        tma_load_4d(st + 5 * TILE, &tm_z, full, 64, hz, t0, sp.bt);
        if (!state_only) {
            tma_load_4d(st + 0 * TILE, &tm_x, full, 0, hx, t0, sp.bt);
            tma_load_4d(st + 1 * TILE, &tm_x, full, 64, hx, t0, sp.bt);
        }
    };
    if (tid == 0) {
        for (int i = 0; i < (int)D_NBAR; ++i)
            mbar_init(&bar[i], i == D_ZP || i == D_HREADY || i == D_CUT ? 8 : i == D_PREADY || i == D_PREADY + 1 || i == D_OFREE ? 4
                               : ((i >= D_EMPTY && i < D_EMPTY + kStages) || i == D_DRAIN) && !state_only ? 2 : 1);
        *abort_flag = 0;
        fence_mbar_init();
#pragma unroll 1
        for (int c = 0; c < min(n, kStages); ++c) load_stage(c);
        if (!state_only) prefetch_tensormap(&tm_o);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, T_COLS);
        tmem_relinquish();
    }
    if (warp == 2 || warp == 3 || warp >= 12) {
        // tables: [0] of each pair for full chunks, [1] for the special one
        const double loglam = decay_log(w.decay[h]);
        const double span = 63.0 * loglam;                   // log of lambda^63
        const bool strong = span < kScaleFloor;              // below the scales' floor
        // 2^s, s half of the span
        const int s = span < kCentred ? min(40, (int)(span * -0.72134752044448170)) : 0;
        const double up = __hiloint2double((1023 + s) << 20, 0), down = __hiloint2double((1023 - s) << 20, 0);
        const int ti = warp < 4 ? tid - 64 : tid - 320;      // 0 .. 319
        for (int i = ti; i < 65 + 3 * 128; i += 320) {
            double e, centre = 1.0;
            uint32_t at;
            if (i < 65) {
                e = i;
                at = TAB_PW + i;
            } else {
                const int t = (i - 65) & 63, which = (i - 65) >> 6;      // w, w', f, f', c, c'
                const int L = (which & 1) ? tail : C, bk = (which & 1) ? back : 0;
                const int p = w.rev ? L - 1 - t : t;                     // tokens since the chunk's start
                e = which < 2 ? max(L - p - bk, 0) : which < 4 ? p : -p;
                at = TAB_W + (i - 65);
                if (strong && which >= 2 && which < 4) e = fmin(e, kScaleFloor / loglam);
                centre = which >= 2 && which < 4 ? up : down;
            }
            tab[at] = (float)(centre * decay_pow(loglam, e));
        }
        // threads with one entry of the tables
        if (ti >= 288 && ti < 304) { // decay of a segment's start state up to this segment
            const int g = ti - 288, here = tokens_before(sp, w.rev, sp.c0);
            if (w.nseg > 1 && g <= sp.seg)
                seg_decay[g] = (float)decay_pow(loglam, here - tokens_before(sp, w.rev, segment_start(w, g)));
        } else if (ti >= 304 && ti < 306) {    // lambda^L of full chunks and of the special one, in two floats
            const int last = ti - 304;
            const double p = decay_pow(loglam, last ? tail - back : C);
            tab[TAB_L + 2 * last] = (float)p;
            tab[TAB_L + 2 * last + 1] = (float)(p - (double)(float)p);
            // the walk's ends: segments' states stay centred, and with no tokens the state passes as it is
            tab[TAB_L + 4 + last] = sp.L == 0 ? 1.f : last ? (FIRST ? 1.f : (float)up) : (float)((w.init_decays ? decay_pow(loglam, 1.0) : 1.0) * down);
        }
    }
    tc_fence_before();
    // Every role meets the others at this barrier once, after its register count is set (every
    // warpgroup changes it, whether or not it has work below: the state's increase waits for the
    // others' decrease) and, for the state, after its loads are issued.
    auto all_set = [&]() -> uint32_t {
        named_sync(3, kDtThreads);
        tc_fence_after();
        return *tmem_slot;
    };

    if (warp < 4) {
        regs_dec<kRegsIssue>();
        const uint32_t tmem = all_set();
        if (warp == 0 && lane == 0) {
            // ==================================================== TMA producer
            int c = min(n, kStages);
            for (; c < n; ++c) {
                if (!ctl.wait_one(D_EMPTY + c % kStages, ((c / kStages) - 1) & 1)) break;
                load_stage(c);
            }
            // Copies in flight land before the CTA's memory goes away.  (Another role may give up after
            // the last copy is issued, so this does not ask whether one has.)
#pragma unroll 1
            for (int i = max(0, c - kStages); i < c; ++i)
                mbar_wait(&bar[D_FULL + i % kStages], (i / kStages) & 1, 1ll << 28);
        }
        if (warp == 1) {
            // ==================================================== MMA issuer: D
            for (int c = 0; c < n; ++c) {
                // Z' written: its tiles have landed and D of the chunk before has been read
                if (!ctl.wait(D_ZP, c & 1)) break;
                const uint32_t st = sbase + (c % kStages) * kStageBytes;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t yd = smem_desc_sw128(st + 2 * TILE, TILE, 1024);
#pragma unroll 1
                    for (int pc = NZ - 1; pc >= 0; --pc)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ts(tmem + T_D, tmem + T_Z + pc * 32 + k * 8, yd + k * (2048 >> 4), IDD_D,
                                        pc < NZ - 1 || k > 0);
                    mma_commit(&bar[D_DFULL]);
                    mma_commit(&bar[D_EMPTY + c % kStages]);
                }
                __syncwarp();
            }
            if (elect_one()) {
                mma_commit(&bar[D_DRAIN]);
                mbar_wait(&bar[D_DRAIN], 0, 1ll << 30);
            }
            __syncwarp();
        }
        if (!state_only && warp == 2) {
            // ==================================================== MMA issuer: G and O
            // Short loops: this code and the other roles' share the instruction cache.
            auto issue_g = [&](int c) -> bool {
                const int s = c % kStages;
                if (!ctl.wait(D_FULL + s, (c / kStages) & 1)) return false;
                // not on D_ZP, which can still be a phase short of the one before this chunk's
                if (w.cu_seqlens && sp.c0 + c == special && tail < C && !ctl.wait(D_CUT, 0)) return false;
                tc_fence_after();                            // G of two chunks before has been read
                if (elect_one()) {
                    const uint64_t xd = smem_desc_sw128(sbase + s * kStageBytes, 16, 1024);
#pragma unroll 1
                    for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t at = xd + hk * (TILE >> 4) + k * 2;
                            mma_bf16(tmem + T_G + 64 * (c & 1), at, at + (2 * TILE >> 4), IDD_G, hk > 0 || k > 0);
                        }
                    mma_commit(&bar[D_GFULL + (c & 1)]);
                }
                __syncwarp();
                return true;
            };
            bool ok = n > 0 && issue_g(0);
            for (int c = 0; c < n && ok; ++c) {
                const int s = c % kStages;
                // G one chunk ahead of P; its buffer was read before P of chunk c - 1 was written
                if (c + 1 < n && !(ok = issue_g(c + 1))) break;
                if (!ctl.wait(D_HREADY, c & 1)) break;
                if (c > 0 && !ctl.wait(D_OFREE, (c - 1) & 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t xd = smem_desc_sw128(sbase + s * kStageBytes, 16, 1024);
#pragma unroll 1
                    for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ts(tmem + T_O, tmem + T_H + hk * 32 + k * 8, xd + hk * (TILE >> 4) + k * 2, IDD_OX,
                                        hk > 0 || k > 0);
                    mma_commit(&bar[D_XFULL]);
                }
                __syncwarp();
                if (!ctl.wait(D_PREADY + (c & 1), (c >> 1) & 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t zd = smem_desc_sw128(sbase + s * kStageBytes + 4 * TILE, TILE, 1024);
                    const uint64_t pd = smem_desc_sw128(sbase + DOFF_P + (c & 1) * TILE, 16, 1024);
#pragma unroll 1
                    for (int pc = fine ? 1 : 0; pc >= 0; --pc)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + T_O, zd + k * (2048 >> 4), pd + pc * (TILE >> 4) + k * 2, IDD_OI, true);
                    mma_commit(&bar[D_OFULL + (c & 1)]);
                    mma_commit(&bar[D_EMPTY + s]);
                }
                __syncwarp();
            }
            if (elect_one()) {
                mma_commit(&bar[D_DRAIN]);
                mbar_wait(&bar[D_DRAIN], 0, 1ll << 30);
            }
            __syncwarp();
        }
    } else if (warp < 12) {
        // ======================================================== state
        regs_inc<kRegsState>();
        const int q4 = warp & 3, part = (warp - 4) >> 2;
        const int dz = q4 * 32 + lane;
        uint64_t H[32];                                      // H^T[dz][64 part + 2 e], +1
#pragma unroll
        for (int e = 0; e < 32; ++e) H[e] = 0;
        const bool has_init = w.init && (FIRST ? !state_only : w.nseg == 1);
        if (has_init) {
            const float *src = w.init + ((size_t)sp.b * w.Hv + h) * hstate;
            if (w.init_trans) {
                const float4 *row = reinterpret_cast<const float4 *>(src + (size_t)dz * kHeadDim + 64 * part);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 v = row[e];
                    H[2 * e] = pack2(v.x, v.y);
                    H[2 * e + 1] = pack2(v.z, v.w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float *at = src + (size_t)(64 * part + 2 * e) * kHeadDim + dz;
                    H[e] = pack2(at[0], at[kHeadDim]);
                }
            }
        }
        const uint32_t tmem = all_set(), t_lane = tmem + ((uint32_t)(q4 * 32) << 16);
        if (has_init && tab[TAB_L + 4] != 1.f) {
            const float f = tab[TAB_L + 4];
#pragma unroll
            for (int e = 0; e < 32; ++e) H[e] = mul2(pack2(f, f), H[e]);
        }
        if (w.nseg > 1 && !FIRST) {
            wait_for_launch_before();
#pragma unroll 1
            for (int g = 0; g <= sp.seg; ++g) {
                const float f = seg_decay[g];
                const float *src = w.seg + (((size_t)sp.b * w.nseg + g) * w.Hv + h) * hstate + (size_t)64 * part * kHeadDim + dz;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    H[e] = fma2(pack2(f, f), pack2(src[(size_t)(2 * e) * kHeadDim], src[(size_t)(2 * e + 1) * kHeadDim]), H[e]);
            }
        }
        auto write_h = [&]() {
            uint32_t hp[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) hp[e] = round_pair(H[e]);
            tmem_st32u(t_lane + T_H + 32 * part, hp);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_HREADY]);
        };
        // The decayed pieces of this warp's block of Z^T (32 lanes x 32 tokens) in registers (until
        // D of the chunk before is done).  zp[.][8 l + 4 k + 2 m + r]: lanes 16 l + 8 r + lane / 4,
        // tokens 16 k + 8 m + 2 (lane % 4), +1 of the block.
        uint32_t zp[NZ][16];
        // ldmatrix rows: lane i gives token 8 (i / 16) + i % 8 of an 8-column group (i / 8) % 2;
        // the second 16 lanes' group differs in bit 1 of the chunk index, 32 in the address
        const uint32_t z_at = sbase + (4 + (q4 >> 1)) * TILE +
                              sw128_chunk(32 * part + 8 * (lane >> 4) + (lane & 7), 4 * (q4 & 1) + ((lane >> 3) & 1));
        const int my_token = 32 * part + 2 * (lane & 3);
        auto make_z = [&](int c) -> bool {
            const int s = c % kStages;
            if (!ctl.wait(D_FULL + s, (c / kStages) & 1)) return false;
            const bool sp_c = sp.c0 + c == special;
            const int rows = sp_c ? tail : C;
            if (w.cu_seqlens && rows < C) {
                // rows of the next sequence out of the products: Y together, of Z the block read below
                unsigned char *y = sm + s * kStageBytes + 2 * TILE;
                for (int i = tid - 128; i < (C - rows) * 2 * 8; i += 256)
                    *reinterpret_cast<uint4 *>(y + ((i >> 3) & 1) * TILE + (rows + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                unsigned char *z = sm + s * kStageBytes + (4 + (q4 >> 1)) * TILE;
                if (32 * part + lane >= rows)
#pragma unroll 1
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4 *>(z + sw128_chunk(32 * part + lane, 4 * (q4 & 1) + k)) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[D_CUT]);
            }
            const float *wt = tab + TAB_W + (sp_c ? 64 : 0) + my_token;
            const uint32_t at = z_at + s * kStageBytes;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 w0 = *reinterpret_cast<const float2 *>(wt + 16 * k), w1 = *reinterpret_cast<const float2 *>(wt + 16 * k + 8);
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    uint32_t z[4];
                    ldmatrix_x4_trans(z, (at ^ (32 * l)) + 2048 * k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t ww = e < 2 ? pack2(w0.x, w0.y) : pack2(w1.x, w1.y);
                        uint64_t v = mul2(ww, pack2(__uint_as_float(z[e] << 16), __uint_as_float(z[e] & 0xffff0000u)));
                        const int x = 8 * l + 4 * k + e;
                        zp[0][x] = split_pair(v);
                        if (NZ == 3) zp[1][x] = split_pair(v);
                        zp[NZ - 1][x] = round_pair(v);
                    }
                }
            }
            return true;
        };
        auto store_z = [&]() {
#pragma unroll
            for (int pc = 0; pc < NZ; ++pc)
#pragma unroll
                for (int l = 0; l < 2; ++l)
                    tmem_st16x128b_x4(t_lane + ((uint32_t)(16 * l) << 16) + T_Z + 32 * pc + 16 * part, zp[pc] + 8 * l);
        };
        auto announce_z = [&]() {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_ZP]);
        };
        bool ok = true;
        if (n > 0 && (ok = make_z(0))) {
            store_z();
            announce_z();
            if (!state_only) write_h();
        }
        for (int c = 0; c < n && ok; ++c) {
            if (c + 1 < n && !(ok = make_z(c + 1))) break;   // while D of this chunk runs
            if (!(ok = ctl.wait(D_DFULL, c & 1))) break;
            tc_fence_after();
            if (c + 1 < n) store_z();
            const bool is_special = sp.c0 + c == special;
            const float2 pf = *reinterpret_cast<const float2 *>(tab + TAB_L + (is_special ? 2 : 0));
            const uint64_t ph = pack2(pf.x, pf.x), pl = pack2(pf.y, pf.y);
            {
                float d[64];
                tmem_ld32(t_lane + T_D + 64 * part, d);
                tmem_ld32(t_lane + T_D + 64 * part + 32, d + 32);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) H[e] = fma2(ph, H[e], fma2(pl, H[e], pack2(d[2 * e], d[2 * e + 1])));
            }
            if (c + 1 < n) {
                announce_z();
                if (!state_only) {
                    if (!(ok = ctl.wait(D_XFULL, c & 1))) break;
                    tc_fence_after();
                    write_h();
                }
            }
        }
        if (tab[TAB_L + 5] != 1.f) {
            const float f = tab[TAB_L + 5];
#pragma unroll
            for (int e = 0; e < 32; ++e) H[e] = mul2(pack2(f, f), H[e]);
        }
        float *dst = nullptr;
        if (FIRST) dst = w.seg + (((size_t)sp.b * w.nseg + sp.seg) * w.Hv + h) * hstate;
        else if (w.fin && sp.c1 == sp.nchunks) dst = w.fin + ((size_t)sp.b * w.Hv + h) * hstate;
        if (ok && dst) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                float a, b;
                unpack2(H[e], a, b);
                float *at = dst + (size_t)(64 * part + 2 * e) * kHeadDim + dz;
                at[0] = a;
                at[kHeadDim] = b;
            }
        }
    } else if (warp < 16) {
        // ======================================================== P
        regs_dec<kRegsP>();
        const int q4 = warp & 3;
        const uint32_t tmem = all_set();
        const uint32_t t_lane = tmem + ((uint32_t)(q4 * 32) << 16);
        const int g = lane >> 2, t = lane & 3, i0 = 16 * q4 + g;         // rows i0, i0 + 8
        unsigned char *pt = sm + DOFF_P + i0 * 128 + 4 * t;
        // Blocks of 8 columns past this warp's 16 rows are zeros for good; the two on the diagonal
        // are multiplied by a mask.  sgn (i - j) = tokens from j to i in walking order.
        const int sgn = w.rev ? -1 : 1;
        uint64_t mask[2][2];                                 // [block][half of the rows]
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int e = sgn * (g + 8 * half - 8 * d - 2 * t);
                mask[d][half] = pack2(e >= 0 ? 1.f : 0.f, e - sgn >= 0 ? 1.f : 0.f);
            }
        if (!state_only) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    *reinterpret_cast<uint32_t *>(pt + half * 1024 + ((k ^ g) << 4)) = 0u;           // both buffers,
                    *reinterpret_cast<uint32_t *>(pt + half * 1024 + ((k ^ g) << 4) + TILE) = 0u;    // or pieces
                }
        }
        auto wait_p = [&](int c) -> bool {
            // M = 64 accumulators sit in lanes 0-15 of every quarter
            if (!ctl.wait(D_GFULL + (c & 1), (c >> 1) & 1)) return false;
            // the MMAs of two chunks before have read this buffer
            if (c > 1 && !ctl.wait(D_OFULL + (c & 1), ((c >> 1) - 1) & 1)) return false;
            tc_fence_after();
            return true;
        };
        auto store_p = [&](auto two, int c, int k, int half, uint64_t v) {
            unsigned char *at = pt + half * 1024 + ((k ^ g) << 4);       // (i0 + 8 half) & 7 = g
            if constexpr (decltype(two)::value) {            // c = 0: the pieces fill both buffers
                *reinterpret_cast<uint32_t *>(at) = split_pair(v);
                *reinterpret_cast<uint32_t *>(at + TILE) = round_pair(v);
            } else {
                *reinterpret_cast<uint32_t *>(at + (c & 1) * TILE) = round_pair(v);
            }
        };
        auto announce_p = [&](int c) {
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[D_PREADY + (c & 1)]);                  // and G is read
        };
        // code of its own for each kind, so that the short loop stays short
        auto rows_of_p = [&](auto two) {
            if (tab[TAB_PW + 63] >= kScaleMin) {
                for (int c = 0; c < n && !state_only; ++c) {
                    if (!wait_p(c)) break;
                    const float *ct = tab + TAB_C + (sp.c0 + c == special ? 64 : 0) + 2 * t;
                    const int bn = w.rev ? 4 : q4 + 1;
                    int b = w.rev ? q4 : 0;                      // 16 columns
                    uint32_t next[8];
                    tmem_ld16x256b_x2(t_lane + T_G + 64 * (c & 1) + 16 * b, next);
#pragma unroll 1
                    for (; b < bn; ++b) {
                        uint32_t r[8];
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 8; ++x) r[x] = next[x];
                        if (b + 1 < bn) tmem_ld16x256b_x2(t_lane + T_G + 64 * (c & 1) + 16 * (b + 1), next);
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            const float2 sc = *reinterpret_cast<const float2 *>(ct + 16 * b + 8 * d);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint64_t v = mul2(pack2(sc.x, sc.y), pack2(__uint_as_float(r[4 * d + 2 * half]), __uint_as_float(r[4 * d + 2 * half + 1])));
                                if (b == q4) v = mul2(v, mask[d][half]);
                                store_p(two, c, 2 * b + d, half, v);
                            }
                        }
                    }
                    announce_p(c);
                }
            } else {
                for (int c = 0; c < n && !state_only; ++c) {
                    if (!wait_p(c)) break;
                    const float *ft = tab + TAB_F + (sp.c0 + c == special ? 64 : 0);
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        uint32_t r[4];
                        tmem_ld16x256b_x1(t_lane + T_G + 64 * (c & 1) + 8 * k, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int e = sgn * (i0 + 8 * half - 8 * k - 2 * t), e1 = e - sgn;
                            const float f = 1.f / ft[i0 + 8 * half];
                            store_p(two, c, k, half, pack2(e >= 0 ? f * tab[TAB_PW + e] * __uint_as_float(r[2 * half]) : 0.f,
                                                   e1 >= 0 ? f * tab[TAB_PW + e1] * __uint_as_float(r[2 * half + 1]) : 0.f));
                        }
                    }
                    announce_p(c);
                }
            }
        };
        if (NP != 1 && fine) rows_of_p(std::true_type{});
        else rows_of_p(std::false_type{});
    } else {
        // ======================================================== O
        regs_dec<kRegsOut>();
        const int q4 = warp & 3;
        const uint32_t tmem = all_set();
        const uint32_t t_lane = tmem + ((uint32_t)(q4 * 32) << 16);
        const bool leader = tid == 512;
        const int t = lane & 3;
        // stmatrix rows: lane i gives token 8 (i / 16) + i % 8 of the 8-column group (i / 8) % 2; the
        // second 16 lanes' group differs in bit 1 of the chunk index, 32 in the address
        const uint32_t o_at = sbase + DOFF_O + (q4 >> 1) * TILE +
                              sw128_chunk(8 * (lane >> 4) + (lane & 7), 4 * (q4 & 1) + ((lane >> 3) & 1));
        const size_t stride = (size_t)w.Hv * kHeadDim;
        for (int c = 0; c < n && !state_only; ++c) {
            const int cw = sp.c0 + c;
            const float *ft = tab + TAB_F + (cw == special ? 64 : 0);
            int t0;
            const int rows = chunk_rows(sp, w.rev, cw, t0);
            if (leader) bulk_wait_group_read0();             // the store before has read the staging tile
            if (!named_and(2, 128, ctl.wait(D_OFULL + (c & 1), (c >> 1) & 1))) break;
            tc_fence_after();
            if (rows < C && w.cu_seqlens) {
                store_rows(static_cast<__nv_bfloat16 *>(w.o) + ((size_t)sp.bt * w.T + t0) * stride + (size_t)h * kHeadDim +
                               q4 * 32 + lane, t_lane, ft, rows, stride);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[D_OFREE]);
                continue;
            }
            if (w.o_f32) {
                // fp32 rows (dense): 32 tokens x 128 values fill the staging tile; the second half is
                // out of TMEM before it waits for the store of the first
                float *tile = reinterpret_cast<float *>(sm + DOFF_O) + q4 * 32 + lane;
#pragma unroll 1
                for (int cb = 0; cb < 2; ++cb) {
                    float x[32];
                    tmem_ld32(t_lane + T_O + 32 * cb, x);
                    tmem_wait_ld();
                    if (cb == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[D_OFREE]);
                        if (leader) bulk_wait_group_read0();
                        named_sync(2, 128);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 f = *reinterpret_cast<const float2 *>(ft + 32 * cb + e);
                        tile[e * kHeadDim] = f.x * x[e];
                        tile[(e + 1) * kHeadDim] = f.y * x[e + 1];
                    }
                    fence_proxy_async_smem();
                    named_sync(2, 128);
                    if (leader) {
                        tma_store_4d(&tm_o, sm + DOFF_O, 0, h, t0 + 32 * cb, sp.bt);
                        bulk_commit_group();
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int cb = 0; cb < 2; ++cb) {                 // 32 tokens
                float2 f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = *reinterpret_cast<const float2 *>(ft + 32 * cb + 8 * k + 2 * t);
#pragma unroll
                for (int slab = 0; slab < 2; ++slab) {       // 16 lanes
                    uint32_t r[16];
                    tmem_ld16x256b_x4(t_lane + ((uint32_t)(16 * slab) << 16) + T_O + 32 * cb, r);
                    tmem_wait_ld();
                    if (cb == 1 && slab == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[D_OFREE]);
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t m[4];
#pragma unroll
                        for (int mm = 0; mm < 4; ++mm) {
                            const int k = 2 * kk + (mm >> 1);
                            const uint32_t *v = r + 4 * k + 2 * (mm & 1);
                            m[mm] = round_pair(mul2(pack2(f[k].x, f[k].y), pack2(__uint_as_float(v[0]), __uint_as_float(v[1]))));
                        }
                        stmatrix_x4_trans((o_at ^ (32 * slab)) + 4096 * cb + 2048 * kk, m[0], m[1], m[2], m[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            named_sync(2, 128);
            if (leader) {
                tma_store_4d(&tm_o, sm + DOFF_O, 0, h, t0, sp.bt);
                tma_store_4d(&tm_o, sm + DOFF_O + TILE, 64, h, t0, sp.bt);
                bulk_commit_group();
            }
        }
        if (leader) bulk_wait_group0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, T_COLS);
        if (lane == 0 && *abort_flag) atomicOr(&g_tc_error, 1u);
    }
}

// Map over a [B, T, H, 128] fp32 tensor; box = 128 x 1 head x 32 tokens x 1, rows as they are.
bool make_map_f32(CUtensorMap *map, const void *base, int B, int T, int H)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * 4, (cuuint64_t)H * kHeadDim * 4, (cuuint64_t)T * H * kHeadDim * 4};
    const cuuint32_t box[4] = {(cuuint32_t)kHeadDim, 1, 32, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FIRST, int NZ, int NP>
cudaError_t launch_tc(const TcWalks &p, cudaStream_t stream)
{
    cudaError_t err = cudaFuncSetAttribute(decay_tc_kernel<FIRST, NZ, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)D_SMEM);
    if (err != cudaSuccess) return err;
    const DecayWalk &w = p.d.w[0];
    const dim3 grid((unsigned)w.Hv, (unsigned)(w.B * w.nseg), (unsigned)p.d.n);
    if (!FIRST && w.nseg > 1) return launch_after(decay_tc_kernel<FIRST, NZ, NP>, grid, kDtThreads, (int)D_SMEM, stream, p);
    decay_tc_kernel<FIRST, NZ, NP><<<grid, kDtThreads, D_SMEM, stream>>>(p);
    return cudaGetLastError();
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

cudaError_t launch_decay_walks_tc(const DecayWalks &d, cudaStream_t stream)
{
    TcWalks p;
    p.d = d;
    bool ends = false;                           // an end state is wanted: its increments with all 24 bits
    for (int i = 0; i < d.n; ++i) {
        const DecayWalk &w = d.w[i];
        const int rows_b = w.cu_seqlens ? 1 : w.B;   // batch rows of the token arrays
        if (!make_map(&p.maps[i][0], w.x, rows_b, w.T, w.hx) || !make_map(&p.maps[i][1], w.y, rows_b, w.T, w.hy) ||
            !make_map(&p.maps[i][2], w.z, rows_b, w.T, w.hz))
            return cudaErrorInvalidValue;
        if (!(w.o_f32 ? make_map_f32(&p.maps[i][3], w.o, rows_b, w.T, w.Hv) : make_map(&p.maps[i][3], w.o, rows_b, w.T, w.Hv)))
            return cudaErrorInvalidValue;
        ends = ends || w.fin;
    }
    const DecayWalk &w = d.w[0];
    cudaError_t err = cudaSuccess;
    if (w.nseg > 1) err = ends ? launch_tc<true, 3, 1>(p, stream) : launch_tc<true, 2, 1>(p, stream);
    if (err != cudaSuccess) return err;
    // packed calls with more than a chunk of tokens hold sequences of both kinds
    if (w.cu_seqlens && w.T > C) return ends ? launch_tc<false, 3, 0>(p, stream) : launch_tc<false, 2, 0>(p, stream);
    if (w.T <= C) return ends ? launch_tc<false, 3, 2>(p, stream) : launch_tc<false, 2, 2>(p, stream);
    return ends ? launch_tc<false, 3, 1>(p, stream) : launch_tc<false, 2, 1>(p, stream);
}

}  // namespace gdn
