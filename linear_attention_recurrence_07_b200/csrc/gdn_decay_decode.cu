// Decode of linear attention with a constant decay per head: one token for every
// (sequence, V head), S' = lambda S + k v^T, o = S'^T q.
//
// The state is the whole cost: read once, written once, an HBM stream.  One CTA
// owns 32 columns of one state (a row's piece is one 128-byte line): 16 KiB, so
// that even a few sequences spread over all SMs.  Thread (row group, lane of 8)
// holds eight float4; the products with q are summed over the 16 row groups
// through shared memory.  B=256, 48 heads: 243 us, 6.65 TB/s, the copy bandwidth.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kCols = 32;                                // state columns per CTA
constexpr int kSlices = kHeadDim / kCols;
constexpr int kDecThreads = 128;
constexpr int kGroups = kDecThreads / (kCols / 4);       // 16 row groups
constexpr int kRowsPerThread = kHeadDim / kGroups;       // 8

template <typename T>
__global__ void __launch_bounds__(kDecThreads)
decay_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                    const float *__restrict__ decay, const float *S, T *__restrict__ o, float *S_new,
                    const int *__restrict__ slots, int n_slots, int Hqk, int Hv)
{
    const unsigned bh = blockIdx.x / kSlices;            // b * Hv + h
    const int c0 = (int)(blockIdx.x - bh * kSlices) * kCols;
    const int b = (int)(bh / (unsigned)Hv), h = (int)(bh - (unsigned)b * Hv);
    const int hq = h / (Hv / Hqk);
    const int tid = threadIdx.x, l8 = tid & 7, g = tid >> 3;
    __shared__ float sk[kHeadDim], sq[kHeadDim];
    __shared__ float4 part[kGroups / 4][kCols / 4];

    size_t state = bh;
    if (slots) {
        const int sl = slots[b];
        if (sl < 0 || sl >= n_slots) return;             // padding entry
        state = (size_t)sl * Hv + h;
    }
    const size_t base = state * (kHeadDim * kHeadDim / 4) + c0 / 4 + l8;   // in float4
    const float4 *S4 = reinterpret_cast<const float4 *>(S) + base;
    float4 s[kRowsPerThread];
#pragma unroll
    for (int m = 0; m < kRowsPerThread; ++m) s[m] = __ldcs(S4 + (g + kGroups * m) * (kHeadDim / 4));
    const size_t qk = ((size_t)b * Hqk + hq) * kHeadDim + tid;
    sk[tid] = to_f32(k[qk]);
    sq[tid] = to_f32(q[qk]);
    const float lam = clamped_decay(decay[h]);
    const size_t vo = (size_t)bh * kHeadDim + c0 + 4 * l8;
    const float v0 = to_f32(v[vo]), v1 = to_f32(v[vo + 1]), v2 = to_f32(v[vo + 2]), v3 = to_f32(v[vo + 3]);
    __syncthreads();
    float4 *D4 = reinterpret_cast<float4 *>(S_new) + base;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < kRowsPerThread; ++m) {
        const int row = g + kGroups * m;
        const float ki = sk[row], qi = sq[row];
        s[m].x = fmaf(lam, s[m].x, ki * v0);
        s[m].y = fmaf(lam, s[m].y, ki * v1);
        s[m].z = fmaf(lam, s[m].z, ki * v2);
        s[m].w = fmaf(lam, s[m].w, ki * v3);
        __stcs(D4 + row * (kHeadDim / 4), s[m]);
        r.x = fmaf(s[m].x, qi, r.x);
        r.y = fmaf(s[m].y, qi, r.y);
        r.z = fmaf(s[m].z, qi, r.z);
        r.w = fmaf(s[m].w, qi, r.w);
    }
#pragma unroll
    for (int off = 8; off < 32; off <<= 1) {             // the four row groups of a warp
        r.x += __shfl_xor_sync(0xffffffffu, r.x, off);
        r.y += __shfl_xor_sync(0xffffffffu, r.y, off);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, off);
        r.w += __shfl_xor_sync(0xffffffffu, r.w, off);
    }
    if ((tid & 31) < 8) part[tid >> 5][l8] = r;
    __syncthreads();
    if (tid < kCols) {
        const float *p = reinterpret_cast<const float *>(part);
        o[(size_t)bh * kHeadDim + c0 + tid] =
            from_f32<T>((p[tid] + p[kCols + tid]) + (p[2 * kCols + tid] + p[3 * kCols + tid]));
    }
}

template <typename T>
void launch_typed(const DecayDecodeArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((size_t)a.B * a.Hv * kSlices);
    decay_decode_kernel<T><<<grid, kDecThreads, 0, stream>>>((const T *)a.q, (const T *)a.k, (const T *)a.v, a.decay,
                                                             a.S, (T *)a.o, a.S_new, a.slots, a.n_slots, a.Hqk, a.Hv);
}

}  // namespace

cudaError_t launch_decay_decode(const DecayDecodeArgs &a, gdn_dtype dtype, cudaStream_t stream)
{
    if (dtype == GDN_BF16) launch_typed<__nv_bfloat16>(a, stream);
    else launch_typed<float>(a, stream);
    return cudaGetLastError();
}

}  // namespace gdn
