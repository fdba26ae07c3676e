// Trees of drafted tokens over a pool of recurrent states: outputs of every node in
// one pass over each state (verification), and the update of the states along the
// accepted path (commit).  Gated delta rule, or decay rule (u = v).
//
// Verification.  With path(i) the nodes from the root to i, Gam_ij the product of
// the gates after j down to i (j on path(i)) and root_i the product along all of
// path(i), the recurrence along every path at once is the chunk form with "earlier
// token" replaced by "ancestor":
//   u_i = beta_i (v_i - root_i S^T k_i - sum_{j strict ancestor} Gam_ij (k_i . k_j) u_j)
//   o_i = root_i S^T q_i + sum_{j on path(i)} Gam_ij (q_i . k_j) u_j
// K S and Q S are warp MMAs on bf16 pieces of S (two pieces for bf16 inputs: 14 to 16
// bits, against the 8 of the output; three, all 24 bits, for fp32 inputs, whose rows are
// cut in three as well).  A state is 64 KiB and n is at most 64 rows, so the products
// are short next to the state's load, and M = 2n rows do not fill a 128-row tcgen05
// tile: fragments come straight from the fp32 state in shared memory, which saves
// the pass that would lay the pieces out for it.
//
// A CTA owns 64 columns of one head's state (two to five CTAs per SM, so that one's load
// runs under another's sums).  The sums over ancestors go level by level: a node has one
// ancestor on every level above it, so at level L every deeper node takes one term from
// the row its ancestor has just finished, into registers, and the nodes of the next level
// are finished.  A bushy tree costs its depth, not its size; non-ancestors are never read,
// so that what is not finite stays below its node.
//
// Measured, 48 heads: 128 sequences of 8 nodes 108 us (3.9 TB/s, 60% of the copy bandwidth),
// 32 of 30 nodes 67 us, 16 of 48 nodes 60 us.  Shared memory holds five (16 nodes) to two (64)
// CTAs per SM.  Small trees are bound by the way of a CTA from the load to the levels; large ones
// by instructions (24 thousand per CTA of 48 nodes, two thirds of the issue slots).
// Commit, 128 sequences of 7 nodes: 164 us, 4.9 TB/s.
#include "gdn_internal.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kTreeCols = 64;            // columns of the state per CTA
constexpr int kTreeSlices = kHeadDim / kTreeCols;
// Columns of S, and of U and QS, in shared memory: no padding (room for one more CTA per SM with
// up to 32 nodes), blocks of 8 and of 16 exchanged by row so that a fragment's rows meet other banks.
__device__ __forceinline__ int s_col(int row, int c) { return c ^ (((row >> 1) & 3) << 3); }
__device__ __forceinline__ int r_col(int row, int c) { return c ^ ((row & 1) << 4); }
constexpr int kLdK = kHeadDim + 8;       // bf16 per row of K and Q
constexpr float kLog2Clamp = -87.0f * 1.4426950408889634f;

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p)) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The bf16 pieces of a pair: the upper 16 bits of what the pieces before left over
// (exact remainders: three pieces are all 24 bits).
__device__ __forceinline__ uint32_t take_piece(float &a, float &b) {
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    a -= __uint_as_float(ua & 0xffff0000u);
    b -= __uint_as_float(ub & 0xffff0000u);
    return __byte_perm(ua, ub, 0x7632);
}

__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(a.x << 16);
    x[1] = __uint_as_float(a.x & 0xffff0000u);
    x[2] = __uint_as_float(a.y << 16);
    x[3] = __uint_as_float(a.y & 0xffff0000u);
}

template <typename T> struct TreeTypes;
template <> struct TreeTypes<__nv_bfloat16> { static constexpr int kPlanes = 1, kPieces = 2; };
template <> struct TreeTypes<float> { static constexpr int kPlanes = 3, kPieces = 3; };

template <typename T, int N>
struct TreeSmem {
    static constexpr int kPlanes = TreeTypes<T>::kPlanes;
    union {
        float S[kHeadDim][kTreeCols];
        struct { float U[N][kTreeCols], QS[N][kTreeCols]; } r;     // after the products with S
    };
    __nv_bfloat16 kq[kPlanes][2][N][kLdK];               // k rows, q rows
    // [node][level of its ancestor], rows of 1, 2, .. N entries (a third CTA per SM at N = 48)
    static constexpr int kTri = N * (N + 1) / 2;
    float A[kTri], P[kTri];
    double b[N];                                         // log2 of root_i
    float2 b2[N];                                        // the same as a sum of two floats
    unsigned long long mask[N];                          // path(i), bit j; 0 for padding
    float beta[N], root[N];
    int jump[N];
    unsigned char list[(kTri + 3) / 4 * 4];              // path(i) in node order: [node][level]
    unsigned char len[N];
    int levels;
};

// Warps per CTA: four for small trees (of which more CTAs fit on an SM), eight for large ones.
template <int N> struct TreeWarps { static constexpr int kWarps = N <= 16 ? 4 : 8; };

// CTAs per SM that shared memory (227 KB) allows: registers are held to that.
template <typename T, int N> constexpr int tree_ctas() { return 227 * 1024 / ((int)sizeof(TreeSmem<T, N>) + 1024); }
static_assert(tree_ctas<__nv_bfloat16, 16>() == 5 && tree_ctas<__nv_bfloat16, 32>() == 4 &&
              tree_ctas<__nv_bfloat16, 48>() == 3 && tree_ctas<__nv_bfloat16, 64>() == 2, "CTAs per SM");

template <typename T, bool DELTA, int N>
__global__ void __launch_bounds__(TreeWarps<N>::kWarps * 32, tree_ctas<T, N>())
tree_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
            const float *__restrict__ alpha, const float *__restrict__ beta, const float *__restrict__ decay,
            const int *__restrict__ parents, const float *__restrict__ pool, const int *__restrict__ slots,
            T *__restrict__ o, int n, int n_slots, int Hqk, int Hv)
{
    using Sm = TreeSmem<T, N>;
    constexpr int kPlanes = Sm::kPlanes, kPieces = TreeTypes<T>::kPieces, MT = N / 16;
    constexpr int W = TreeWarps<N>::kWarps, kTreeThreads = W * 32;
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const unsigned bh = blockIdx.x / kTreeSlices;
    const int c0 = (int)(blockIdx.x - bh * kTreeSlices) * kTreeCols;
    const int b = (int)(bh / (unsigned)Hv), h = (int)(bh - (unsigned)b * Hv), hq = h / (Hv / Hqk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // ---- what does not wait for the slot: k and q rows (bf16: straight to shared memory; rows
    //      past n are zeros), the tree and its gates, v of this thread's rows and columns
    if constexpr (kPlanes == 1) {
        for (int i = tid; i < 2 * N * 16; i += kTreeThreads) {
            const int which = i / (N * 16), r = (i / 16) % N, d = (i % 16) * 8;
            void *dst = &sm.kq[0][which][r][d];
            if (r < n) cp_async16(dst, (which ? q : k) + (((size_t)b * n + r) * Hqk + hq) * kHeadDim + d);
            else *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    constexpr int kPer = (N + 31) / 32;
    int p[kPer];
    float ga[kPer], be[kPer];
    if (warp == 0) {
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int i = lane + 32 * x;
            p[x] = -2; ga[x] = 1.f; be[x] = 0.f;
            if (i < n) {
                const size_t at = ((size_t)b * n + i) * Hv + h;
                p[x] = parents[(size_t)b * n + i];
                ga[x] = DELTA ? alpha[at] : decay[h];
                if (DELTA) be[x] = beta[at];
            }
        }
    }
    const int slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= n_slots) {
        cp_async_wait_all();
        return;
    }
    const float *S = pool + ((size_t)slot * Hv + h) * (kHeadDim * kHeadDim) + c0;
#pragma unroll
    for (int m = 0; m < 2048 / kTreeThreads; ++m) {
        const int row = (tid >> 4) + (kTreeThreads / 16) * m, c = (tid & 15) * 4;
        cp_async16(&sm.S[row][s_col(row, c)], S + row * kHeadDim + c);
    }
    // warps by columns of S, and with eight of them by row set (0: k, 1: q)
    constexpr int RW = W == 8 ? 1 : 2;                   // row sets per warp
    const int role = W == 8 ? warp >> 2 : 0, cw = 16 * (warp & 3);
    const int g = lane >> 2, t = lane & 3;
    float vv[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = mt * 16 + g + 8 * half;
#pragma unroll
            for (int e = 0; e < 4; ++e) vv[mt][half][e] = 0.f;
            if (i < n && (W == 4 || role == 0)) load4(v + (((size_t)b * n + i) * Hv + h) * kHeadDim + c0 + cw + 4 * t, vv[mt][half]);
        }
    if (warp == 0) {
        // ---- paths and gates by pointer jumping: after round r, mask and b cover 2^r steps.
        //      jump: next node up, -1 past the root, -2 padding.
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int i = lane + 32 * x;
            if (i < N) {
                sm.jump[i] = p[x] < -1 || p[x] >= i ? -2 : p[x];
                sm.mask[i] = 1ull << i;
                const float l = log2f(ga[x]);
                sm.b[i] = (double)(DELTA ? fmaxf(l, kLog2Clamp) : l < kLog2Clamp ? kLog2Clamp : l);   // a bad decay stays NaN
                sm.beta[i] = be[x];
            }
        }
        __syncwarp();
#pragma unroll 1
        for (int step = 1; step < N; step <<= 1) {
            unsigned long long m2[kPer];
            double b2[kPer];
            int j2[kPer];
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int i = lane + 32 * x;
                m2[x] = 0; b2[x] = 0.0; j2[x] = -1;
                if (i < N) {
                    const int j = sm.jump[i];
                    j2[x] = j;
                    if (j >= 0) { m2[x] = sm.mask[j]; b2[x] = sm.b[j]; j2[x] = sm.jump[j]; }
                }
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int i = lane + 32 * x;
                if (i < N) { sm.mask[i] |= m2[x]; sm.b[i] += b2[x]; sm.jump[i] = j2[x]; }
            }
            if (!__any_sync(0xffffffffu, j2[0] >= 0 || j2[kPer - 1] >= 0)) step = N;    // every path has ended
            __syncwarp();
        }
        int most = 0;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int i = lane + 32 * x;
            if (i < N) {
                const unsigned long long m = sm.jump[i] == -1 ? sm.mask[i] : 0ull;   // -2 reached: padding
                const double bi = sm.b[i];
                const float hi = (float)bi;
                sm.mask[i] = m;
                sm.b2[i] = make_float2(hi, (float)(bi - (double)hi));
                sm.root[i] = exp2f(hi);
                const int c = __popcll(m);
                sm.len[i] = (unsigned char)c;
                most = max(most, c);
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) sm.levels = most;
    } else {
        for (int i = tid - 32; i < (int)sizeof(sm.list) / 4; i += kTreeThreads - 32) reinterpret_cast<uint32_t *>(sm.list)[i] = 0u;
        if constexpr (kPlanes > 1) {
            for (int i = tid - 32; i < 2 * N * (kHeadDim / 4); i += kTreeThreads - 32) {
                const int which = i / (N * (kHeadDim / 4)), r = (i / (kHeadDim / 4)) % N, d = (i % (kHeadDim / 4)) * 4;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < n) f = *reinterpret_cast<const float4 *>((which ? q : k) + (((size_t)b * n + r) * Hqk + hq) * kHeadDim + d);
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) {
                    const uint32_t lo = take_piece(f.x, f.y), hi = take_piece(f.z, f.w);
                    *reinterpret_cast<uint2 *>(&sm.kq[pl][which][r][d]) = make_uint2(lo, hi);
                }
            }
        }
    }
    cp_async_wait_all();
    __syncthreads();

    const int lrow = lane & 15, lcol = (lane >> 4) * 8;  // ldmatrix addresses
    // ---- grams with k -> coefficients of the path sums, j <= i only
    const int gr = warp / (W / 2), gc = warp % (W / 2);  // row set and share of the columns
    if (DELTA || gr == 1) {
#pragma unroll 1
        for (int nt = gc; nt < N / 8; nt += W / 2) {
            uint32_t kb[kPlanes][kHeadDim / 16][2];          // this tile's 8 rows of k
#pragma unroll
            for (int pb = 0; pb < kPlanes; ++pb)
#pragma unroll
                for (int ks = 0; ks < kHeadDim / 16; ++ks) {
                    const __nv_bfloat16 *kr = &sm.kq[pb][0][nt * 8 + g][ks * 16 + 2 * t];
                    kb[pb][ks][0] = *reinterpret_cast<const uint32_t *>(kr);
                    kb[pb][ks][1] = *reinterpret_cast<const uint32_t *>(kr + 8);
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt < nt / 2) continue;
                float acc[2][4] = {};                        // even and odd ks: half the chain
#pragma unroll
                for (int sum = kPlanes - 1; sum >= 0; --sum)
#pragma unroll
                    for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
                            uint32_t a[4];
                            ldmatrix_x4(a, &sm.kq[pa][gr][mt * 16 + lrow][ks * 16 + lcol]);
                            mma16816(acc[ks & 1], a, kb[sum - pa][ks][0], kb[sum - pa][ks][1]);
                        }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = mt * 16 + g + half * 8, j0 = nt * 8 + 2 * t;
                    const unsigned long long m = sm.mask[i];
                    const uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32);
                    // path bits below j0, and of j0 and j0 + 1 (of the same word: j0 is even)
                    const uint32_t word = j0 < 32 ? lo : hi, bits = word >> (j0 & 31);
                    int at = i * (i + 1) / 2 + __popc(word & ((1u << (j0 & 31)) - 1u)) + (j0 < 32 ? 0 : __popc(lo));
                    const float2 bi = sm.b2[i];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if ((bits >> e) & 1u) {
                            const int j = j0 + e;
                            const float2 bj = sm.b2[j];
                            const float x = exp2f((bi.x - bj.x) + (bi.y - bj.y)) * (acc[0][2 * half + e] + acc[1][2 * half + e]);
                            if (gr == 0) {
                                if (j < i) sm.A[at] = sm.beta[i] * x;
                            } else {
                                sm.P[at] = x;
                                sm.list[at] = (unsigned char)j;
                            }
                            ++at;
                        }
                    }
                }
            }
        }
    }
    // ---- rows of k and of q times S: this warp's 16 columns (each piece of S is cut once), thread
    //      (g, t) the columns 2g, 2g+1 of B.  fp32 inputs: the tensor core truncates as it accumulates,
    //      so each 16 rows of S are summed from zero, small pieces first, and added in fp32.
    float acc[RW][MT][2][4];
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][mt][j][e] = 0.f;
    // the decay rule needs no k S
    if (DELTA || W == 4 || role == 1)
#pragma unroll 1
    for (int ks = 0; ks < kHeadDim / 16; ++ks) {
        const float *sr = &sm.S[ks * 16 + 2 * t][s_col(2 * t, cw + 2 * g)];      // rows 2t + 1, + 8, + 9 alike
        float2 s0 = *reinterpret_cast<const float2 *>(sr), s1 = *reinterpret_cast<const float2 *>(sr + kTreeCols);
        float2 s2 = *reinterpret_cast<const float2 *>(sr + 8 * kTreeCols), s3 = *reinterpret_cast<const float2 *>(sr + 9 * kTreeCols);
        uint32_t bp[kPieces][2][2];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            bp[p][0][0] = take_piece(s0.x, s1.x); bp[p][0][1] = take_piece(s2.x, s3.x);
            bp[p][1][0] = take_piece(s0.y, s1.y); bp[p][1][1] = take_piece(s2.y, s3.y);
        }
#pragma unroll
        for (int r = DELTA || RW == 1 ? 0 : 1; r < RW; ++r)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (kPlanes == 1) {
                    uint32_t a[4];
                    ldmatrix_x4(a, &sm.kq[0][role + r][mt * 16 + lrow][ks * 16 + lcol]);
#pragma unroll
                    for (int p = kPieces - 1; p >= 0; --p)
#pragma unroll
                        for (int j = 0; j < 2; ++j) mma16816(acc[r][mt][j], a, bp[p][j][0], bp[p][j][1]);
                } else {
                    float d[2][4] = {};
#pragma unroll
                    for (int sum = kPieces - 1; sum >= 0; --sum)         // orders of size, small first
#pragma unroll
                        for (int pa = sum; pa >= 0; --pa) {
                            uint32_t a[4];
                            ldmatrix_x4(a, &sm.kq[pa][role + r][mt * 16 + lrow][ks * 16 + lcol]);
#pragma unroll
                            for (int j = 0; j < 2; ++j) mma16816(d[j], a, bp[sum - pa][j][0], bp[sum - pa][j][1]);
                        }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][mt][j][e] += d[j][e];
                }
            }
    }
    __syncthreads();                                     // S read; A and P written
    // ---- accumulators: rows g, g + 8 of each tile, columns cw + 4t .. + 3
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = mt * 16 + g + 8 * half, c = cw + 4 * t;
            if (W == 4 || role == 0) {
                const float f = sm.root[i], be_i = sm.beta[i];
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = DELTA ? be_i * (vv[mt][half][e] - f * acc[0][mt][e & 1][2 * half + (e >> 1)]) : vv[mt][half][e];
                *reinterpret_cast<float4 *>(&sm.r.U[i][r_col(i, c)]) = make_float4(x[0], x[1], x[2], x[3]);
            }
            if (W == 4 || role == 1) {
                const float(&y)[2][4] = acc[RW - 1][mt];
                *reinterpret_cast<float4 *>(&sm.r.QS[i][r_col(i, c)]) = make_float4(y[0][2 * half], y[1][2 * half], y[0][2 * half + 1], y[1][2 * half + 1]);
            }
        }
    __syncthreads();
    // ---- levels: warp w of W owns nodes w, w + W, ..., lane l columns 2l, 2l + 1
    constexpr int kOwn = N / W;
    float2 u[kOwn], out[kOwn];
    int len[kOwn];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
        const int i = warp + W * x;
        len[x] = sm.len[i];
        const float2 r = *reinterpret_cast<const float2 *>(&sm.r.QS[i][r_col(i, 2 * lane)]);
        out[x] = make_float2(sm.root[i] * r.x, sm.root[i] * r.y);
        u[x] = *reinterpret_cast<const float2 *>(&sm.r.U[i][r_col(i, 2 * lane)]);
    }
    const int levels = sm.levels;
#pragma unroll 1
    for (int L = 0; L < levels; ++L) {
        if (DELTA && L > 0) {                            // the nodes of this level are finished
#pragma unroll
            for (int x = 0; x < kOwn; ++x)
                if (len[x] == L + 1) *reinterpret_cast<float2 *>(&sm.r.U[warp + W * x][r_col(warp + W * x, 2 * lane)]) = u[x];
            __syncthreads();
        }
        // loads outside the conditions, so that all rows are on their way at once
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
            const int i = warp + W * x;
            const int at = i * (i + 1) / 2 + L;              // in the arrays for every L < N, a row's or not
            const int j = sm.list[at];
            const float2 w = *reinterpret_cast<const float2 *>(&sm.r.U[j][r_col(j, 2 * lane)]);
            const float p = sm.P[at];
            const bool on = len[x] > L;
            if (on) { out[x].x = fmaf(p, w.x, out[x].x); out[x].y = fmaf(p, w.y, out[x].y); }
            if (DELTA) {
                const float a = sm.A[at];
                const bool deeper = len[x] > L + 1;
                if (deeper) { u[x].x = fmaf(-a, w.x, u[x].x); u[x].y = fmaf(-a, w.y, u[x].y); }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
        const int i = warp + W * x;
        if (len[x] == 0) continue;                       // padding: the row stays as it was
        T *dst = o + (((size_t)b * n + i) * Hv + h) * kHeadDim + c0 + 2 * lane;
        if constexpr (kPlanes == 1) *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(out[x].x, out[x].y);
        else *reinterpret_cast<float2 *>(dst) = out[x];
    }
}

template <typename T, bool DELTA, int N>
cudaError_t launch_tree_n(const TreeArgs &a, cudaStream_t stream)
{
    const int smem = (int)sizeof(TreeSmem<T, N>);
    cudaError_t err = cudaFuncSetAttribute(tree_kernel<T, DELTA, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    tree_kernel<T, DELTA, N><<<(unsigned)((size_t)a.B * a.Hv * kTreeSlices), TreeWarps<N>::kWarps * 32, smem, stream>>>(
        (const T *)a.q, (const T *)a.k, (const T *)a.v, a.alpha, a.beta, a.decay, a.parents, a.pool, a.slots, (T *)a.o,
        a.n, a.n_slots, a.Hqk, a.Hv);
    return cudaGetLastError();
}

template <typename T, bool DELTA>
cudaError_t launch_tree_typed(const TreeArgs &a, cudaStream_t stream)
{
    if (a.n <= 16) return launch_tree_n<T, DELTA, 16>(a, stream);
    if (a.n <= 32) return launch_tree_n<T, DELTA, 32>(a, stream);
    if (a.n <= 48) return launch_tree_n<T, DELTA, 48>(a, stream);
    return launch_tree_n<T, DELTA, 64>(a, stream);
}

// ------------------------------------------------------------------ commit
// One CTA owns 32 columns of one state (a row's piece is one 128-byte line), in registers,
// read and written once: thread (row group, lane of 8) holds eight float4, as in the decay
// decode.  The path's nodes are taken four at a time: their products with the state share
// one pass over the registers and one reduction, the delta rule inside the four is a 4 x 4
// substitution per column, and one pass applies the four writes.
constexpr int kGroup = 4;
constexpr int kComCols = 32;
constexpr int kComSlices = kHeadDim / kComCols;
constexpr int kComThreads = 128;
constexpr int kComGroups = kComThreads / (kComCols / 4);     // 16 row groups
constexpr int kComRows = kHeadDim / kComGroups;              // 8

template <typename T, bool DELTA>
__global__ void __launch_bounds__(kComThreads, 8)
commit_kernel(const T *__restrict__ k, const T *__restrict__ v, const float *__restrict__ alpha,
              const float *__restrict__ beta, const float *__restrict__ decay, const int *__restrict__ parents,
              const int *__restrict__ accepted, float *pool, const int *__restrict__ slots, int n, int n_slots,
              int Hqk, int Hv)
{
    __shared__ int path[kMaxTreeNodes], par[kMaxTreeNodes];
    __shared__ int path_len;
    __shared__ float sk[kGroup][kHeadDim];
    __shared__ float4 part[kComThreads / 32][kGroup][kComCols / 4];
    __shared__ __align__(16) float su[kGroup][kComCols];     // read as float4
    __shared__ float skk[kGroup][kGroup];
    const unsigned bh = blockIdx.x / kComSlices;
    const int c0 = (int)(blockIdx.x - bh * kComSlices) * kComCols;
    const int b = (int)(bh / (unsigned)Hv), h = (int)(bh - (unsigned)b * Hv), hq = h / (Hv / Hqk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l8 = tid & 7, rg = tid >> 3;
    const int my_parent = tid < n ? parents[(size_t)b * n + tid] : 0;
    const int slot = slots ? slots[b] : b, leaf = accepted[b];
    if (slot < 0 || slot >= n_slots || leaf < 0 || leaf >= n) return;
    if (tid < n) par[tid] = my_parent;
    float4 *S4 = reinterpret_cast<float4 *>(pool + ((size_t)slot * Hv + h) * (kHeadDim * kHeadDim) + c0) + l8;
    uint64_t s[kComRows][2];                             // pairs of columns
#pragma unroll
    for (int m = 0; m < kComRows; ++m) {
        const float4 x = __ldcs(S4 + (rg + kComGroups * m) * (kHeadDim / 4));
        s[m][0] = pack2(x.x, x.y);
        s[m][1] = pack2(x.z, x.w);
    }
    __syncthreads();
    if (tid == 0) {
        int len = 0, i = leaf;
        while (i >= 0) {                                 // parents are smaller: at most n steps
            path[len++] = i;
            const int p = par[i];
            i = (p < -1 || p >= i) ? -2 : p;
        }
        path_len = i == -1 ? len : 0;                    // -2: below a padding node
    }
    __syncthreads();
    const int len = path_len;
    if (len == 0) return;
    // one group's inputs: element tid of each k, the gates, and what the substitution of this
    // thread's column needs (root first; missing nodes get k = 0, gate 1 and no write)
    float nk[kGroup], na[kGroup], nv[kGroup], nb[kGroup];
    auto fetch = [&](int d0) {
        const int m = min(kGroup, len - d0);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            const size_t node = (size_t)b * n + path[len - 1 - d0 - min(j, m - 1)];
            nk[j] = j < m ? to_f32(k[(node * Hqk + hq) * kHeadDim + tid]) : 0.f;
            na[j] = j >= m ? 1.f : DELTA ? fmaxf(alpha[node * Hv + h], 1.6458114e-38f) : clamped_decay(decay[h]);
            nv[j] = nb[j] = 0.f;
            if (tid < kComCols) {
                nv[j] = to_f32(v[(node * Hv + h) * kHeadDim + c0 + tid]);
                if (DELTA) nb[j] = beta[node * Hv + h];
            }
        }
    };
    fetch(0);
    for (int d0 = 0; d0 < len; d0 += kGroup) {
        const int m = min(kGroup, len - d0);
        float a[kGroup], vv[kGroup], be[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            sk[j][tid] = nk[j];
            a[j] = na[j]; vv[j] = nv[j]; be[j] = nb[j];
        }
        if (d0 + kGroup < len) fetch(d0 + kGroup);       // while this group is worked on
        __syncthreads();
        if (DELTA) {
            for (int pr = warp; pr < 6; pr += kComThreads / 32) {        // k_i . k_j, i > j
                const int i = pr < 1 ? 1 : pr < 3 ? 2 : 3, j = pr - (i * (i - 1)) / 2;
                float x = 0.f;
#pragma unroll
                for (int d = 0; d < 4; ++d) x = fmaf(sk[i][lane + 32 * d], sk[j][lane + 32 * d], x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if (lane == 0) skk[i][j] = x;
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (j >= m) break;
                uint64_t p0 = 0, p1 = 0;
#pragma unroll
                for (int r = 0; r < kComRows; ++r) {
                    const float ki = sk[j][rg + kComGroups * r];
                    p0 = fma2(s[r][0], pack2(ki, ki), p0);
                    p1 = fma2(s[r][1], pack2(ki, ki), p1);
                }
                float4 pp;
                unpack2(p0, pp.x, pp.y);
                unpack2(p1, pp.z, pp.w);
#pragma unroll
                for (int off = 8; off < 32; off <<= 1) {                 // the four row groups of a warp
                    pp.x += __shfl_xor_sync(0xffffffffu, pp.x, off);
                    pp.y += __shfl_xor_sync(0xffffffffu, pp.y, off);
                    pp.z += __shfl_xor_sync(0xffffffffu, pp.z, off);
                    pp.w += __shfl_xor_sync(0xffffffffu, pp.w, off);
                }
                if (lane < 8) part[warp][j][l8] = pp;
            }
            __syncthreads();
        }
        if (tid < kComCols) {
            float u[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                u[j] = 0.f;
                if (j < m) {
                    u[j] = vv[j];
                    if (DELTA) {
                        float p = 0.f;
#pragma unroll
                        for (int w = 0; w < kComThreads / 32; ++w) p += reinterpret_cast<const float *>(&part[w][j][0])[tid];
#pragma unroll
                        for (int i = 0; i < j; ++i) p = fmaf(a[i], p, skk[j][i] * u[i]);   // S after node i, times k_j
                        u[j] = be[j] * (u[j] - a[j] * p);
                    }
                }
            }
            // the writes as they stand after the group: each decayed by the gates behind it
            float behind = 1.f;
#pragma unroll
            for (int j = kGroup - 1; j >= 0; --j) {
                su[j][tid] = behind * u[j];
                behind *= a[j];
            }
        }
        const float all = (a[0] * a[1]) * (a[2] * a[3]);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kComRows; ++r) {
            s[r][0] = mul2(pack2(all, all), s[r][0]);
            s[r][1] = mul2(pack2(all, all), s[r][1]);
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            if (j >= m) break;
            const float4 u4 = *reinterpret_cast<const float4 *>(&su[j][4 * l8]);
#pragma unroll
            for (int r = 0; r < kComRows; ++r) {
                const float ki = sk[j][rg + kComGroups * r];
                s[r][0] = fma2(pack2(ki, ki), pack2(u4.x, u4.y), s[r][0]);
                s[r][1] = fma2(pack2(ki, ki), pack2(u4.z, u4.w), s[r][1]);
            }
        }
        __syncthreads();                                 // sk, su, part are written again
    }
#pragma unroll
    for (int m = 0; m < kComRows; ++m) {
        float4 x;
        unpack2(s[m][0], x.x, x.y);
        unpack2(s[m][1], x.z, x.w);
        __stcs(S4 + (rg + kComGroups * m) * (kHeadDim / 4), x);
    }
}

template <typename T, bool DELTA>
cudaError_t launch_commit_typed(const TreeArgs &a, cudaStream_t stream)
{
    commit_kernel<T, DELTA><<<(unsigned)((size_t)a.B * a.Hv * kComSlices), kComThreads, 0, stream>>>(
        (const T *)a.k, (const T *)a.v, a.alpha, a.beta, a.decay, a.parents, a.accepted, a.pool_out, a.slots, a.n,
        a.n_slots, a.Hqk, a.Hv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, gdn_dtype dtype, cudaStream_t stream)
{
    if (dtype == GDN_BF16)
        return a.decay ? launch_tree_typed<__nv_bfloat16, false>(a, stream) : launch_tree_typed<__nv_bfloat16, true>(a, stream);
    return a.decay ? launch_tree_typed<float, false>(a, stream) : launch_tree_typed<float, true>(a, stream);
}

cudaError_t launch_tree_commit(const TreeArgs &a, gdn_dtype dtype, cudaStream_t stream)
{
    if (dtype == GDN_BF16)
        return a.decay ? launch_commit_typed<__nv_bfloat16, false>(a, stream) : launch_commit_typed<__nv_bfloat16, true>(a, stream);
    return a.decay ? launch_commit_typed<float, false>(a, stream) : launch_commit_typed<float, true>(a, stream);
}

}  // namespace gdn
