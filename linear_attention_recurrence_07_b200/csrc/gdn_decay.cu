// Linear attention with a constant decay per head, chunk by chunk on CUDA cores in
// fp32 (the path of fp32 inputs; see DecayWalk for the walk that prefill and all
// gradients share).
//
// Per chunk of L <= 64 tokens, with H the state at its start (decayed to its first
// token), p_i = i forwards and L - 1 - i backwards (tokens since the start):
//   P_ij = lambda^{|i - j|} x_i . y_j   for j at or before i in the walk, else 0
//   o_i  = lambda^{p_i} H^T x_i + sum_j P_ij z_j
//   H   <- lambda^L H + sum_j lambda^{L - p_j} y_j z_j^T
// (a prefill's last chunk uses one power less throughout, so that S_final is not
// decayed past its last token).  The powers come from a table computed in 64 bits,
// and lambda^L enters the state as a sum of two floats: its rounding would add up
// over hundreds of chunks of a slowly decaying head.
//
// Two forms.  Wide: a CTA owns a whole head (128 columns of the state and output), 8 x 4
// and 8 x 8 register tiles, the next chunk's rows on their way into registers during the
// sums.  Narrow: 32 columns, two CTAs per SM; the score tile is computed four times, but
// short prompts of few heads still spread over the device.
//
// Bound by fp32 arithmetic: 2.9 M multiply-adds per chunk and head (wide: scores 0.5, H's share
// 1.05, P z 0.3, the state's update 1.05), 22,800 cycles of an SM or 12 us; measured 24 us (144
// heads, one CTA on each SM), of which shared-memory operands and the phases' barriers take the
// rest.  48 heads, T=512: 119 us; gradients of B=2, T=206: 207 us (narrow: 369).
#include "decay_common.cuh"

namespace gdn {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kLdX = kHeadDim + 4;           // padded rows
constexpr int kLdP = kChunk + 4;

template <int DZ>                            // columns of the state per CTA
struct SimtSmem {
    static constexpr int kLdZ = DZ + 4;
    float x[kChunk][kLdX], y[kChunk][kLdX];
    float z[kChunk][kLdZ];
    float H[kHeadDim][kLdZ];
    float P[kChunk][kLdP];
    float pw[kChunk + 1];                    // lambda^0 .. lambda^64
    float seg[16];                           // decay of each segment's state up to this one
    float2 step[2];                          // lambda^L as two floats: full chunks, the sequence's last
};

template <int DZ>
__global__ void __launch_bounds__(kSimtThreads)
decay_walk_kernel(const __grid_constant__ DecayWalks d, bool first)
{
    constexpr int kZSlices = kHeadDim / DZ;
    const DecayWalk &w = d.w[blockIdx.z];
    extern __shared__ __align__(16) unsigned char raw[];
    SimtSmem<DZ> &sm = *reinterpret_cast<SimtSmem<DZ> *>(raw);
    const int tid = threadIdx.x;
    const int h = blockIdx.x / kZSlices, z0 = (blockIdx.x - h * kZSlices) * DZ;
    const WalkSpan sp = walk_span(w, blockIdx.y, first);
    const bool state_only = sp.state_only;
    if (first) let_next_launch_start();
    const size_t st = (size_t)kHeadDim * kHeadDim;
    const int tail = sp.L - (sp.nchunks - 1) * kChunk, special = w.rev ? 0 : sp.nchunks - 1;
    const int last_back = w.fin_back && !first;     // the end state is wanted undecayed

    if (tid < kChunk + 1 + 16 + 2) {
        const double loglam = decay_log(w.decay[h]);
        if (tid <= kChunk) {
            sm.pw[tid] = (float)decay_pow(loglam, tid);
        } else if (tid <= kChunk + 16) {
            const int g = tid - kChunk - 1, here = tokens_before(sp, w.rev, sp.c0);
            if (w.nseg > 1 && !first && g <= sp.seg)
                sm.seg[g] = (float)decay_pow(loglam, here - tokens_before(sp, w.rev, segment_start(w, g)));
        } else {
            const int last = tid - kChunk - 17;
            const double p = decay_pow(loglam, last ? tail - last_back : kChunk);
            sm.step[last] = make_float2((float)p, (float)(p - (double)(float)p));
        }
    }
    __syncthreads();
    // ---- start state
    if (w.nseg > 1 && !first) {
        wait_for_launch_before();
        for (int i = tid; i < kHeadDim * (DZ / 4); i += kSimtThreads) {
            const int d = i / (DZ / 4), c = (i % (DZ / 4)) * 4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int g = 0; g <= sp.seg; ++g) {          // entry g holds the walk up to segment g's start
                const float f = sm.seg[g];
                const float4 v = *reinterpret_cast<const float4 *>(
                    w.seg + (((size_t)sp.b * w.nseg + g) * w.Hv + h) * st + (size_t)d * kHeadDim + z0 + c);
                a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y);
                a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
            }
            *reinterpret_cast<float4 *>(&sm.H[d][c]) = a;
        }
    } else {
        const float *src = (w.init && !state_only) ? w.init + ((size_t)sp.b * w.Hv + h) * st : nullptr;
        const float f = (w.init_decays && sp.L > 0) ? sm.pw[1] : 1.f;
        for (int i = tid; i < kHeadDim * DZ; i += kSimtThreads) {
            const int d = w.init_trans ? (i & (kHeadDim - 1)) : i / DZ;
            const int c = w.init_trans ? i / kHeadDim : i % DZ;
            const size_t at = w.init_trans ? (size_t)(z0 + c) * kHeadDim + d : (size_t)d * kHeadDim + z0 + c;
            sm.H[d][c] = src ? f * src[at] : 0.f;
        }
    }
    __syncthreads();

    const float *x = static_cast<const float *>(w.x), *y = static_cast<const float *>(w.y), *z = static_cast<const float *>(w.z);
    float *o = static_cast<float *>(w.o);
    const int xh = h / (w.Hv / w.hx), yh = h / (w.Hv / w.hy), zh = h / (w.Hv / w.hz);
    const int ti = tid >> 4, tj = tid & 15;      // 16 x 16 threads
    // a chunk's rows: 8 float4 of x and of y and DZ / 16 of z per thread, zeros past the end
    constexpr int kZ4 = DZ / 16;
    float4 px[8], py[8], pz[kZ4];
    auto fetch = [&](int c) {
        int t0;
        const int L = chunk_rows(sp, w.rev, c, t0);
        const size_t tok = (size_t)sp.bt * w.T + t0;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int r = (tid >> 5) + 8 * m, d = (tid & 31) * 4;
            px[m] = py[m] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < L) {
                if (!state_only) px[m] = *reinterpret_cast<const float4 *>(x + ((tok + r) * w.hx + xh) * kHeadDim + d);
                py[m] = *reinterpret_cast<const float4 *>(y + ((tok + r) * w.hy + yh) * kHeadDim + d);
            }
        }
#pragma unroll
        for (int m = 0; m < kZ4; ++m) {
            const int i = tid + m * kSimtThreads, r = i / (DZ / 4), d = (i % (DZ / 4)) * 4;
            pz[m] = r < L ? *reinterpret_cast<const float4 *>(z + ((tok + r) * w.hz + zh) * kHeadDim + z0 + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    if (DZ == 128 && sp.c0 < sp.c1) fetch(sp.c0);
    for (int c = sp.c0; c < sp.c1; ++c) {
        int t0;
        const int L = chunk_rows(sp, w.rev, c, t0);
        const size_t tok = (size_t)sp.bt * w.T + t0;
        if (DZ != 128) fetch(c);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            *reinterpret_cast<float4 *>(&sm.x[(tid >> 5) + 8 * m][(tid & 31) * 4]) = px[m];
            *reinterpret_cast<float4 *>(&sm.y[(tid >> 5) + 8 * m][(tid & 31) * 4]) = py[m];
        }
#pragma unroll
        for (int m = 0; m < kZ4; ++m) {
            const int i = tid + m * kSimtThreads;
            *reinterpret_cast<float4 *>(&sm.z[i / (DZ / 4)][(i % (DZ / 4)) * 4]) = pz[m];
        }
        __syncthreads();
        if (DZ == 128 && c + 1 < sp.c1) fetch(c + 1);
        if (!state_only) {
            // ---- P: rows ti + 16 a, columns tj + 16 b
            float p[4][4] = {};
            for (int d = 0; d < kHeadDim; d += 4) {
                float4 xv[4], yv[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    xv[a] = *reinterpret_cast<const float4 *>(&sm.x[ti + 16 * a][d]);
                    yv[a] = *reinterpret_cast<const float4 *>(&sm.y[tj + 16 * a][d]);
                }
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        p[a][b] = fmaf(xv[a].x, yv[b].x, p[a][b]);
                        p[a][b] = fmaf(xv[a].y, yv[b].y, p[a][b]);
                        p[a][b] = fmaf(xv[a].z, yv[b].z, p[a][b]);
                        p[a][b] = fmaf(xv[a].w, yv[b].w, p[a][b]);
                    }
            }
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int i = ti + 16 * a, j = tj + 16 * b;
                    const int e = w.rev ? j - i : i - j;
                    sm.P[i][j] = e >= 0 ? sm.pw[max(e, 0)] * p[a][b] : 0.f;
                }
            __syncthreads();
            if constexpr (DZ == 128) {
            // ---- o: warp = 8 rows, lane = four columns
            const int r = tid >> 5, cc = (tid & 31) * 4;
            float acc[8][4] = {};
            for (int d = 0; d < kHeadDim; d += 4) {
                float4 hv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[e] = *reinterpret_cast<const float4 *>(&sm.H[d + e][cc]);
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    const float4 xv = *reinterpret_cast<const float4 *>(&sm.x[8 * r + a][d]);
                    const float xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[a][0] = fmaf(xx[e], hv[e].x, acc[a][0]); acc[a][1] = fmaf(xx[e], hv[e].y, acc[a][1]);
                        acc[a][2] = fmaf(xx[e], hv[e].z, acc[a][2]); acc[a][3] = fmaf(xx[e], hv[e].w, acc[a][3]);
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                const int i = 8 * r + a;
                const float f = sm.pw[w.rev ? max(L - 1 - i, 0) : i];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[a][e] *= f;
            }
            // columns of P that some of the 8 rows can see; rows past L of z are zeros
            const int j0 = w.rev ? 8 * r : 0, j1 = w.rev ? L : min(L, 8 * r + 8);
            for (int j = j0; j < j1; j += 4) {
                float4 zv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) zv[e] = *reinterpret_cast<const float4 *>(&sm.z[j + e][cc]);
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    const float4 pv = *reinterpret_cast<const float4 *>(&sm.P[8 * r + a][j]);
                    const float pp[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[a][0] = fmaf(pp[e], zv[e].x, acc[a][0]); acc[a][1] = fmaf(pp[e], zv[e].y, acc[a][1]);
                        acc[a][2] = fmaf(pp[e], zv[e].z, acc[a][2]); acc[a][3] = fmaf(pp[e], zv[e].w, acc[a][3]);
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < 8; ++a)
                if (8 * r + a < L)
                    *reinterpret_cast<float4 *>(o + ((tok + 8 * r + a) * w.Hv + h) * kHeadDim + cc) =
                        make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
            } else {
            // ---- o: rows 4 r .., four columns; the two halves of the block take half of d and of j
            const int part = tid >> 7, r = (tid & 127) >> 3, cc = (tid & 7) * 4;
            float acc[4][4] = {}, dia[4][4] = {};
            for (int d = 64 * part; d < 64 * part + 64; d += 4) {
                float4 hv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[e] = *reinterpret_cast<const float4 *>(&sm.H[d + e][cc]);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float4 xv = *reinterpret_cast<const float4 *>(&sm.x[4 * r + a][d]);
                    const float xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[a][0] = fmaf(xx[e], hv[e].x, acc[a][0]); acc[a][1] = fmaf(xx[e], hv[e].y, acc[a][1]);
                        acc[a][2] = fmaf(xx[e], hv[e].z, acc[a][2]); acc[a][3] = fmaf(xx[e], hv[e].w, acc[a][3]);
                    }
                }
            }
            for (int j = 4 * part; j < L; j += 8) {              // rows past L of z are zeros
                float4 zv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) zv[e] = *reinterpret_cast<const float4 *>(&sm.z[j + e][cc]);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float4 pv = *reinterpret_cast<const float4 *>(&sm.P[4 * r + a][j]);
                    const float pp[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dia[a][0] = fmaf(pp[e], zv[e].x, dia[a][0]); dia[a][1] = fmaf(pp[e], zv[e].y, dia[a][1]);
                        dia[a][2] = fmaf(pp[e], zv[e].z, dia[a][2]); dia[a][3] = fmaf(pp[e], zv[e].w, dia[a][3]);
                    }
                }
            }
            __syncthreads();                                     // P and x have been read
            float *half = &sm.P[0][0] + (tid & 127) * 16;        // 128 x 16 floats of P's room
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int i = 4 * r + a;
                const float f = sm.pw[w.rev ? max(L - 1 - i, 0) : i];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[a][e] = fmaf(f, acc[a][e], dia[a][e]);
                if (part) *reinterpret_cast<float4 *>(half + 4 * a) = make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
            }
            __syncthreads();
            if (!part) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int i = 4 * r + a;
                    if (i >= L) continue;
                    const float4 o4 = *reinterpret_cast<const float4 *>(half + 4 * a);
                    *reinterpret_cast<float4 *>(o + ((tok + i) * w.Hv + h) * kHeadDim + z0 + cc) =
                        make_float4(acc[a][0] + o4.x, acc[a][1] + o4.y, acc[a][2] + o4.z, acc[a][3] + o4.w);
                }
            }
            }
            __syncthreads();
        }
        // ---- H: rows d0 .., columns c0 .. (wide: and c0 + 64 ..)
        {
            constexpr int RD = DZ == 128 ? 8 : 4, CZ = DZ == 128 ? 2 : 1;
            const int back = last_back && c == special ? 1 : 0;
            const float2 step = sm.step[c == special];
            const int d0 = (DZ == 128 ? tid >> 4 : tid >> 3) * RD, c0 = (DZ == 128 ? tid & 15 : tid & 7) * 4;
            float acc[RD][4 * CZ] = {};
            for (int j = 0; j < L; ++j) {
                const float f = sm.pw[(w.rev ? j + 1 : L - j) - back];
                float yy[RD];
#pragma unroll
                for (int e = 0; e < RD; e += 4) {
                    const float4 yv = *reinterpret_cast<const float4 *>(&sm.y[j][d0 + e]);
                    yy[e] = f * yv.x; yy[e + 1] = f * yv.y; yy[e + 2] = f * yv.z; yy[e + 3] = f * yv.w;
                }
#pragma unroll
                for (int q = 0; q < CZ; ++q) {
                    const float4 zv = *reinterpret_cast<const float4 *>(&sm.z[j][c0 + 64 * q]);
#pragma unroll
                    for (int a = 0; a < RD; ++a) {
                        float *t = &acc[a][4 * q];
                        t[0] = fmaf(yy[a], zv.x, t[0]); t[1] = fmaf(yy[a], zv.y, t[1]);
                        t[2] = fmaf(yy[a], zv.z, t[2]); t[3] = fmaf(yy[a], zv.w, t[3]);
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < RD; ++a)
#pragma unroll
                for (int q = 0; q < CZ; ++q) {
                    float4 &hv = *reinterpret_cast<float4 *>(&sm.H[d0 + a][c0 + 64 * q]);
                    const float *t = &acc[a][4 * q];
                    hv = make_float4(fmaf(step.x, hv.x, fmaf(step.y, hv.x, t[0])), fmaf(step.x, hv.y, fmaf(step.y, hv.y, t[1])),
                                     fmaf(step.x, hv.z, fmaf(step.y, hv.z, t[2])), fmaf(step.x, hv.w, fmaf(step.y, hv.w, t[3])));
                }
        }
        __syncthreads();
    }
    // ---- end state
    float *dst = nullptr;
    if (first) dst = w.seg + (((size_t)sp.b * w.nseg + sp.seg) * w.Hv + h) * st;
    else if (w.fin && sp.c1 == sp.nchunks) dst = w.fin + ((size_t)sp.b * w.Hv + h) * st;
    if (dst)
        for (int i = tid; i < kHeadDim * (DZ / 4); i += kSimtThreads) {
            const int d = i / (DZ / 4), cc = (i % (DZ / 4)) * 4;
            *reinterpret_cast<float4 *>(dst + (size_t)d * kHeadDim + z0 + cc) =
                *reinterpret_cast<const float4 *>(&sm.H[d][cc]);
        }
}

template <int DZ>
cudaError_t launch_form(const DecayWalks &d, cudaStream_t stream)
{
    const int smem = (int)sizeof(SimtSmem<DZ>);
    cudaError_t err = cudaFuncSetAttribute(decay_walk_kernel<DZ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    const DecayWalk &w = d.w[0];
    const dim3 grid((unsigned)w.Hv * (kHeadDim / DZ), (unsigned)(w.B * w.nseg), (unsigned)d.n);
    if (w.nseg > 1) {
        decay_walk_kernel<DZ><<<grid, kSimtThreads, smem, stream>>>(d, true);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
        return launch_after(decay_walk_kernel<DZ>, grid, kSimtThreads, smem, stream, d, false);
    }
    decay_walk_kernel<DZ><<<grid, kSimtThreads, smem, stream>>>(d, false);
    return cudaGetLastError();
}

// One thread per four columns of an output row; blockIdx.y picks the array.
template <typename T>
__global__ void __launch_bounds__(256)
head_sum_kernel(const float *__restrict__ part_a, const float *__restrict__ part_b, T *__restrict__ out_a,
                T *__restrict__ out_b, long long n4, int G)
{
    const float *part = blockIdx.y ? part_b : part_a;
    T *out = blockIdx.y ? out_b : out_a;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256) {
        const long long row = i >> 5;                    // token * Hqk + head
        const int d = (int)(i & 31) * 4;
        const float *p = part + row * G * kHeadDim + d;  // V heads of a QK head are contiguous
        float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
        for (int g = 1; g < G; ++g) {
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p + (size_t)g * kHeadDim));
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        T *dst = out + row * kHeadDim + d;
        if constexpr (sizeof(T) == 2) {
            __nv_bfloat162 v[2] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w)};
            *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(v);
        } else {
            *reinterpret_cast<float4 *>(dst) = a;
        }
    }
}

}  // namespace

cudaError_t launch_decay_walks_simt(const DecayWalks &d, cudaStream_t stream)
{
    return d.wide ? launch_form<128>(d, stream) : launch_form<32>(d, stream);
}

cudaError_t launch_head_sums(const float *part_a, const float *part_b, void *out_a, void *out_b, long long rows,
                             int Hqk, int Hv, gdn_dtype dtype, cudaStream_t stream)
{
    const long long n4 = rows * Hqk * (kHeadDim / 4);
    const dim3 grid((unsigned)((n4 + 255) / 256 < 148 * 8 ? (n4 + 255) / 256 : 148 * 8), 2);
    if (dtype == GDN_BF16)
        head_sum_kernel<<<grid, 256, 0, stream>>>(part_a, part_b, (__nv_bfloat16 *)out_a, (__nv_bfloat16 *)out_b, n4, Hv / Hqk);
    else
        head_sum_kernel<<<grid, 256, 0, stream>>>(part_a, part_b, (float *)out_a, (float *)out_b, n4, Hv / Hqk);
    return cudaGetLastError();
}

}  // namespace gdn
