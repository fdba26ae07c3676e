// Shared by the walks of the decay recurrence (CUDA cores and tensor cores): where a
// CTA's tokens, start state and end state are, and the powers of its head's decay.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {
namespace {

// lambda^e for integer e >= 0, with log lambda >= -87; computed in 64 bits, because a
// power is applied once per chunk and its relative error adds up over the chunks.  A negative or
// NaN decay stays NaN.
__device__ __forceinline__ double decay_log(float lam)
{
    const double l = log((double)lam);
    return l < -87.0 ? -87.0 : l;
}
__device__ __forceinline__ double decay_pow(double loglam, double e) { return exp(e * loglam); }

// The two launches of a segmented walk overlap: the first lets the second start as its CTAs
// leave (and may itself be gone before anything of it is read), the second sets itself up,
// loads its first rows, and waits for the first's states just before it reads them.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches the second of the two.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What one CTA of a walk does.  Chunk c of the walk (c0 <= c < c1) holds token rows
// tb + 64 m .. of batch row bt, m = c forwards and nchunks - 1 - c backwards.
struct WalkSpan {
    int bt, tb, L;         // batch row, first token row, tokens of the sequence
    int nchunks;           // chunks of the whole sequence
    int c0, c1;            // this CTA's chunks
    int b, seg;            // sequence, segment
    bool state_only;       // first launch: no output rows, the segment's state from zero
};

__device__ __forceinline__ int chunk_rows(const WalkSpan &s, bool rev, int c, int &t0)
{
    const int m = rev ? s.nchunks - 1 - c : c;
    t0 = s.tb + m * kChunk;
    return min(kChunk, s.L - m * kChunk);
}

// First chunk of segment g of the second launch.
__device__ __forceinline__ int segment_start(const DecayWalk &w, int g) { return w.head_chunks + g * w.seg_chunks; }

// y: index over sequences x segments.  first: the first launch of a segmented walk, which walks the
// head of the sequence (entry 0, from its start state) and the states of the segments but the last
// (entry g + 1: segment g).
__device__ __forceinline__ WalkSpan walk_span(const DecayWalk &w, int y, bool first)
{
    WalkSpan s;
    s.state_only = false;
    if (w.cu_seqlens) {
        const int a = min(max(w.cu_seqlens[y], 0), w.T);
        const int e = min(max(w.cu_seqlens[y + 1], a), w.T);
        s.b = y; s.seg = 0; s.bt = 0; s.tb = a; s.L = e - a;
        s.nchunks = (s.L + kChunk - 1) / kChunk;
        s.c0 = 0; s.c1 = s.nchunks;
        return s;
    }
    s.b = y / w.nseg;
    s.seg = y - s.b * w.nseg;
    s.bt = s.b; s.tb = 0; s.L = w.T;
    s.nchunks = (w.T + kChunk - 1) / kChunk;
    if (first) {
        s.state_only = s.seg > 0;
        s.c0 = s.state_only ? segment_start(w, s.seg - 1) : 0;
        s.c1 = segment_start(w, s.seg);
    } else {
        s.c0 = segment_start(w, s.seg);
        s.c1 = s.seg == w.nseg - 1 ? s.nchunks : s.c0 + w.seg_chunks;
    }
    return s;
}

// Tokens that the walk has passed before chunk c.
__device__ __forceinline__ int tokens_before(const WalkSpan &s, bool rev, int c)
{
    if (c >= s.nchunks) return s.L;
    if (!rev) return c * kChunk;
    return c == 0 ? 0 : s.L - (s.nchunks - c) * kChunk;   // backwards the ragged chunk comes first
}

}  // namespace
}  // namespace gdn
