// Logprobs and seeded sampling over rows of fp32 logits.
//
// "Mathematically equivalent is not bitwise equivalent": logprobs come from
// one log_softmax kernel pair, whichever step (prefill rescoring or decode)
// produced the logits.  A row is cut into segments of kSeg columns (a
// function of V alone); each segment's max and sum of exponentials are
// reduced in one fixed order, and the segments' partials are merged in
// segment order, so a row's logprobs are bitwise the same whatever other rows
// share the launch ("The replacement kernels are deliberately dull": no
// reduction whose order follows the batch).
//
// "The weaker guarantees, which are usually enough": a request's draw depends
// only on its own seed, its position and the column: Gumbel noise from
// MurmurHash3 (x86, 32-bit) of (position, column) under the request's seed,
// in float64, and the token is the argmax of logit / temperature + noise.
// The argmax is a total order (a NaN beats every number, ties go to the
// lowest index), so segments of a row may be searched by separate CTAs and
// combined in any order without changing the winner.  float64 is slow on
// this GPU, so every score is first computed in fp32 with a proven error
// bound; only the columns whose fp32 score lies within the bounds of their
// segment's best fp32 score can be that segment's float64 winner, and only
// they are scored in float64.  The token is the float64 argmax exactly.
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "tc_tmem.cuh"

namespace bi {

constexpr int kSeg = 4096;            // columns per segment (log_softmax and sampling)
constexpr int kSegThreads = 256;
constexpr int kPerThread = kSeg / kSegThreads;  // 16 columns per thread: j = seg * kSeg + tid + 256 k

int32_t logit_segments(int32_t V) { return (V + kSeg - 1) / kSeg; }

// ---------------------------------------------------------------------------
// log_softmax: lp_j = (x_j - m) - log(z), m = max_j x_j, z = sum_j exp(x_j - m)
// Pass 1 (one CTA per segment s): m_s = max over the segment, z_s = sum of
// exp(x_j - m_s) in a fixed order: each thread's 16 columns in ascending k,
// an xor butterfly inside each warp, the 8 warps' sums in warp order (a
// segment without a finite maximum contributes z_s = 0).  Pass 2: every CTA
// of the row merges the row's partials in segment order, m = max_s m_s,
// z = sum_s z_s * exp(m_s - m), and writes its segment's logprobs.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kSegThreads)
log_softmax_partial_kernel(const float* __restrict__ x, int32_t V, int32_t nseg, float2* __restrict__ part) {
    pdl_trigger();
    pdl_wait();
    __shared__ float red[kSegThreads / 32];
    __shared__ float bc;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int32_t seg = blockIdx.x, r = blockIdx.y;
    const float* xr = x + static_cast<int64_t>(r) * V;
    float v[kPerThread];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int32_t j = seg * kSeg + tid + kSegThreads * k;
        v[k] = j < V ? xr[j] : -INFINITY;
        mx = fmaxf(mx, v[k]);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    if (tid == 0) {
        float m = red[0];
        for (int w = 1; w < kSegThreads / 32; ++w) m = fmaxf(m, red[w]);
        bc = m;
    }
    __syncthreads();
    const float m = bc;
    float z = 0.0f;
    if (m != -INFINITY) {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const int32_t j = seg * kSeg + tid + kSegThreads * k;
            if (j < V) z = __fadd_rn(z, expf(__fsub_rn(v[k], m)));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k)
            if (isnan(v[k])) z = v[k];
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) z = __fadd_rn(z, __shfl_xor_sync(0xffffffffu, z, off));
    __syncthreads();  // red[] is reused
    if (lane == 0) red[warp] = z;
    __syncthreads();
    if (tid == 0) {
        float t = red[0];
        for (int w = 1; w < kSegThreads / 32; ++w) t = __fadd_rn(t, red[w]);
        part[static_cast<int64_t>(r) * nseg + seg] = make_float2(m, t);
    }
}

__global__ void __launch_bounds__(kSegThreads)
log_softmax_write_kernel(const float* __restrict__ x, int32_t V, int32_t nseg, const float2* __restrict__ part,
                         float* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    __shared__ float2 ml;
    const int tid = threadIdx.x;
    const int32_t seg = blockIdx.x, r = blockIdx.y;
    if (tid == 0) {
        const float2* pr = part + static_cast<int64_t>(r) * nseg;
        float m = pr[0].x;
        for (int32_t q = 1; q < nseg; ++q) m = fmaxf(m, pr[q].x);
        float z = 0.0f;
        for (int32_t q = 0; q < nseg; ++q) z = __fadd_rn(z, __fmul_rn(pr[q].y, expf(__fsub_rn(pr[q].x, m))));
        ml = make_float2(m, logf(z));
    }
    __syncthreads();
    const float m = ml.x, lz = ml.y;
    const float* xr = x + static_cast<int64_t>(r) * V;
    float* orow = out + static_cast<int64_t>(r) * V;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int32_t j = seg * kSeg + tid + kSegThreads * k;
        if (j < V) orow[j] = __fsub_rn(__fsub_rn(xr[j], m), lz);
    }
}

size_t log_softmax_ws_bytes(int32_t R, int32_t V) {
    if (R <= 0 || V <= 0) return 0;
    return static_cast<size_t>(R) * logit_segments(V) * sizeof(float2) + 256;
}

cudaError_t launch_log_softmax(const float* logits, float* out, int32_t R, int32_t V, void* ws, cudaStream_t s) {
    if (R <= 0) return cudaSuccess;
    const int32_t nseg = logit_segments(V);
    float2* part = static_cast<float2*>(ws);
    cudaError_t e = launch_pdl(log_softmax_partial_kernel, dim3(nseg, R), dim3(kSegThreads), 0, s, logits, V, nseg,
                               part);
    if (e != cudaSuccess) return e;
    return launch_pdl(log_softmax_write_kernel, dim3(nseg, R), dim3(kSegThreads), 0, s, logits, V, nseg,
                      static_cast<const float2*>(part), out);
}

// ---------------------------------------------------------------------------
// Seeded Gumbel-max sampling
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t rotl32(uint32_t v, int r) { return (v << r) | (v >> (32 - r)); }

// MurmurHash3_x86_32 of the 8-byte key le32(pos) || le32(col): two 4-byte
// blocks, no tail, length 8, then the final avalanche.
__device__ __forceinline__ uint32_t murmur3_pos_col(uint32_t pos, uint32_t col, uint32_t seed) {
    constexpr uint32_t c1 = 0xcc9e2d51u, c2 = 0x1b873593u;
    uint32_t h = seed;
    uint32_t k = pos * c1;
    k = rotl32(k, 15) * c2;
    h ^= k;
    h = rotl32(h, 13) * 5u + 0xe6546b64u;
    k = col * c1;
    k = rotl32(k, 15) * c2;
    h ^= k;
    h = rotl32(h, 13) * 5u + 0xe6546b64u;
    h ^= 8u;
    h ^= h >> 16;
    h *= 0x85ebca6bu;
    h ^= h >> 13;
    h *= 0xc2b2ae35u;
    h ^= h >> 16;
    return h;
}

// (score a, index ia) beats (b, ib) in the sampling total order.
__device__ __forceinline__ bool beats(double a, int32_t ia, double b, int32_t ib) {
    const bool an = isnan(a), bn = isnan(b);
    if (an || bn) return an && (!bn || ia < ib);
    return a > b || (a == b && ia < ib);
}

// The float64 score of column j (the definition): x_j / t + g_j, or x_j for
// a greedy row.
__device__ __forceinline__ double score64(float x, double td, bool greedy, uint32_t h) {
    if (greedy) return static_cast<double>(x);
    const double u = (static_cast<double>(h) + 0.5) * 0x1p-32;  // exact: (0, 1)
    return __dadd_rn(__ddiv_rn(static_cast<double>(x), td), -log(-log(u)));
}

// fp32 estimate of score64 and the bound on their difference.  With
// u = (h + 0.5) / 2^32: w = -log(u) from u itself when u < 1/2 (w >= ln 2),
// else from 1 - u = (2^32 - 1 - h + 0.5) / 2^32 through log1pf, so neither
// loses digits to cancellation; the arguments carry a relative error of at
// most 2^-23 (two roundings).  __logf is within 2^-21.41 absolute on [0.5, 2]
// and 3 ulp elsewhere, log1pf within 1 ulp: |w32 - w| / w < 9e-6 and
// |g32 - g| < 1e-5 over the whole range of g ([-3.14, 22.9], its ends at
// h = 0 and h = 2^32 - 1).  x * (1/t) and the sum add 3 * 2^-24 of
// |x / t| and of |s|.  delta(s) = 1e-4 + 1e-6 (|s| + 48) covers all of it
// with a margin of five or more (|x / t| <= |s| + 24).  A greedy row is exact
// in fp32 (delta = 0).
__device__ __forceinline__ float score32(float x, float rt, bool greedy, uint32_t h) {
    if (greedy) return x;
    float w;
    if (h < 0x80000000u) {
        const float u = __fmul_rn(__fadd_rn(static_cast<float>(h), 0.5f), 0x1p-32f);
        w = -__logf(u);
    } else {
        const float v = __fmul_rn(__fadd_rn(static_cast<float>(0xffffffffu - h), 0.5f), 0x1p-32f);
        w = -log1pf(-v);
    }
    return __fadd_rn(__fmul_rn(x, rt), -__logf(w));
}
__device__ __forceinline__ float score_bound(float s, bool greedy) {
    return greedy ? 0.0f : __fadd_rn(1e-4f, __fmul_rn(1e-6f, __fadd_rn(fabsf(s), 48.0f)));
}

// grid (segments, rows): the float64 winner of one segment of a row.  Every
// column's fp32 score is kept in registers; with M the segment's best fp32
// score (reached at column k), the segment's float64 winner w satisfies
// s32_w + delta_w >= s64_w >= s64_k >= M - delta(M), so only such columns
// (and any non-finite score or maximum: a NaN beats every number, an
// overflow leaves no bound) are scored in float64.  The row's winner is the
// float64 winner of its own segment, so the merge below is exact.
__global__ void __launch_bounds__(kSegThreads)
sample_segment_kernel(const float* __restrict__ x, const uint32_t* __restrict__ seeds,
                      const int32_t* __restrict__ positions, const float* __restrict__ temps, int32_t V,
                      int32_t nseg, double* __restrict__ ws_score, int32_t* __restrict__ ws_idx) {
    pdl_trigger();
    pdl_wait();
    __shared__ float red[kSegThreads / 32];
    __shared__ float s_thr;
    __shared__ double s_sc[kSegThreads / 32];
    __shared__ int32_t s_ix[kSegThreads / 32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int32_t seg = blockIdx.x, r = blockIdx.y;
    const float* xr = x + static_cast<int64_t>(r) * V;
    const float t = temps[r];
    const bool greedy = !(t > 0.0f);  // temperature 0 (or not positive): the greedy argmax of the logits
    const float rt = greedy ? 1.0f : __frcp_rn(t);
    const double td = static_cast<double>(t);
    const uint32_t seed = seeds[r], pos = static_cast<uint32_t>(positions[r]);
    float s32[kPerThread];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int32_t j = seg * kSeg + tid + kSegThreads * k;
        s32[k] = -INFINITY;
        if (j < V) {
            const uint32_t h = greedy ? 0u : murmur3_pos_col(pos, static_cast<uint32_t>(j), seed);
            s32[k] = score32(xr[j], rt, greedy, h);
            mx = fmaxf(mx, s32[k]);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    if (tid == 0) {
        float m = red[0];
        for (int w = 1; w < kSegThreads / 32; ++w) m = fmaxf(m, red[w]);
        s_thr = isfinite(m) ? __fsub_rn(m, score_bound(m, greedy)) : -INFINITY;
    }
    __syncthreads();
    const float thr = s_thr;
    double best = 0.0;
    int32_t bi = -1;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int32_t j = seg * kSeg + tid + kSegThreads * k;
        if (j < V) {
            const bool cand = !isfinite(s32[k]) || !(thr > -INFINITY) ||
                              __fadd_rn(s32[k], score_bound(s32[k], greedy)) >= thr;
            if (cand) {
                const uint32_t h = greedy ? 0u : murmur3_pos_col(pos, static_cast<uint32_t>(j), seed);
                const double sc = score64(xr[j], td, greedy, h);
                if (bi < 0 || beats(sc, j, best, bi)) {
                    best = sc;
                    bi = j;
                }
            }
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const double os = __shfl_xor_sync(0xffffffffu, best, off);
        const int32_t oi = __shfl_xor_sync(0xffffffffu, bi, off);
        if (oi >= 0 && (bi < 0 || beats(os, oi, best, bi))) {
            best = os;
            bi = oi;
        }
    }
    if (lane == 0) {
        s_sc[warp] = best;
        s_ix[warp] = bi;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kSegThreads / 32; ++w)
            if (s_ix[w] >= 0 && (bi < 0 || beats(s_sc[w], s_ix[w], best, bi))) {
                best = s_sc[w];
                bi = s_ix[w];
            }
        ws_score[static_cast<int64_t>(r) * nseg + seg] = best;
        ws_idx[static_cast<int64_t>(r) * nseg + seg] = bi;
    }
}

// grid (rows), one warp: the winner over a row's segments.
__global__ void __launch_bounds__(32)
sample_merge_kernel(const double* __restrict__ ws_score, const int32_t* __restrict__ ws_idx, int32_t nseg,
                    int32_t* __restrict__ tokens) {
    pdl_trigger();
    pdl_wait();
    const int32_t r = blockIdx.x;
    const int lane = threadIdx.x;
    double best = 0.0;
    int32_t bi = -1;
    for (int32_t sg = lane; sg < nseg; sg += 32) {
        const double sc = ws_score[static_cast<int64_t>(r) * nseg + sg];
        const int32_t ix = ws_idx[static_cast<int64_t>(r) * nseg + sg];
        if (ix >= 0 && (bi < 0 || beats(sc, ix, best, bi))) {
            best = sc;
            bi = ix;
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const double os = __shfl_xor_sync(0xffffffffu, best, off);
        const int32_t oi = __shfl_xor_sync(0xffffffffu, bi, off);
        if (oi >= 0 && (bi < 0 || beats(os, oi, best, bi))) {
            best = os;
            bi = oi;
        }
    }
    if (lane == 0) tokens[r] = bi;
}

size_t sample_ws_bytes(int32_t R, int32_t V) {
    if (R <= 0 || V <= 0) return 0;
    const size_t n = static_cast<size_t>(R) * logit_segments(V);
    return n * (sizeof(double) + sizeof(int32_t)) + 256;
}

cudaError_t launch_sample(const float* logits, const uint32_t* seeds, const int32_t* positions, const float* temps,
                          int32_t* tokens, int32_t R, int32_t V, void* ws, cudaStream_t s) {
    if (R <= 0) return cudaSuccess;
    const int32_t nseg = logit_segments(V);
    const size_t n = static_cast<size_t>(R) * nseg;
    double* ws_score = static_cast<double*>(ws);
    int32_t* ws_idx = reinterpret_cast<int32_t*>(ws_score + n);
    cudaError_t e = launch_pdl(sample_segment_kernel, dim3(nseg, R), dim3(kSegThreads), 0, s, logits, seeds,
                               positions, temps, V, nseg, ws_score, ws_idx);
    if (e != cudaSuccess) return e;
    return launch_pdl(sample_merge_kernel, dim3(R), dim3(32), 0, s, static_cast<const double*>(ws_score),
                      static_cast<const int32_t*>(ws_idx), nseg, tokens);
}

// ---------------------------------------------------------------------------
// Log probabilities of given tokens, entropy and the best alternatives
// (bi_token_logprobs): one read of the logits, no [R, V] output.
//
// Pass 1 (one CTA per segment): log_softmax_partial_kernel's maximum and sum
// in its order (so the log probabilities have its bits), t_s = sum of
// e^(x - m_s) (x - m_s) in the same order, and the segment's K best columns.
// Pass 2 (one CTA per row) merges the segments' sums in segment order
//   m = max m_s, f_s = e^(m_s - m), z = sum z_s f_s,
//   t = sum f_s (t_s + z_s (m_s - m)),   entropy = log z - t / z,
// picks the K best of the segments' lists and gathers the asked columns.
// Columns are compared by argmax_key (a total order), so lists may be built
// in any order.
//
// K best without sorting: each warp finds the ceil(K/8)-th largest of its
// lanes' maxima (a reduction per round); no column below the smallest of the
// 8 warps' values can be among the K best, because every warp holds
// ceil(K/8) columns at or above its own.  The columns at or above it
// (typically about 2K of 4096) are listed and ranked by counting; a list that
// overflows (many equal logits) is taken one column at a time.
//
// Bound by instruction issue: a column costs about 13 instructions, eight of
// them log_softmax's exponential, and a segment's reductions as much as 10
// columns of each thread.  Measured: 1001 x 50257 bf16 without alternatives 37
// us (15 for the bytes), 512 x 128256 fp32 with the 8 best 77 us (39).
// ---------------------------------------------------------------------------
constexpr int kSegWarps = kSegThreads / 32;
constexpr int kCand = 256;  // listed columns; more are taken one at a time

struct TopSmem {
    unsigned long long cand[kCand];
    unsigned long long red[kSegWarps];
    uint32_t cut[kSegWarps];
    int32_t n;
};

// The upper half of argmax_key: smaller is better.
__device__ __forceinline__ uint32_t key_hi(float v) { return static_cast<uint32_t>(argmax_key(v, 0) >> 32); }

// A key's high half that at least K of the block's keys do not exceed, or
// ~0u when there are too few; best = the smallest high half this thread has.
__device__ __forceinline__ uint32_t top_cut(TopSmem& sm, uint32_t best, int K) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    uint32_t w = ~0u;
    for (int c = 0; c < (K + kSegWarps - 1) / kSegWarps; ++c) {
        w = __reduce_min_sync(0xffffffffu, best);
        // one lane at a time, so that each round stands for a column of its own
        const unsigned at = __ballot_sync(0xffffffffu, best == w);
        if (lane == __ffs(at) - 1) best = ~0u;
    }
    if (lane == 0) sm.cut[warp] = w;
    if (threadIdx.x == 0) sm.n = 0;
    __syncthreads();
    uint32_t cut = 0u;
#pragma unroll
    for (int i = 0; i < kSegWarps; ++i) cut = max(cut, sm.cut[i]);
    return cut;
}

__device__ __forceinline__ void list_key(TopSmem& sm, unsigned long long key) {
    const int at = atomicAdd(&sm.n, 1);
    if (at < kCand) sm.cand[at] = key;
}

// After the candidates are listed: put(rank, key) for the K best keys of the
// block, ascending; keys(k) = this thread's k-th key (kArgmaxKeyNone: none).
template <typename Keys, typename Put>
__device__ __forceinline__ void top_rank(TopSmem& sm, int K, Keys&& keys, Put&& put) {
    __syncthreads();
    const int n = sm.n;
    if (n <= kCand) {
        if (static_cast<int>(threadIdx.x) < n) {
            const unsigned long long mine = sm.cand[threadIdx.x];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += sm.cand[i] < mine;
            if (rank < K) put(rank, mine);
        }
        for (int i = n + threadIdx.x; i < K; i += kSegThreads) put(i, kArgmaxKeyNone);
        return;
    }
    unsigned long long last = 0;
    for (int r = 0; r < K; ++r) {
        unsigned long long best = kArgmaxKeyNone;
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const unsigned long long x = keys(k);
            if ((r == 0 || x > last) && x < best) best = x;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o < best ? o : best;
        }
        if ((threadIdx.x & 31) == 0) sm.red[threadIdx.x / 32] = best;
        __syncthreads();
        best = sm.red[0];
#pragma unroll
        for (int i = 1; i < kSegWarps; ++i) best = sm.red[i] < best ? sm.red[i] : best;
        if (threadIdx.x == 0) put(r, best);
        last = best;
        __syncthreads();
    }
}

__device__ __forceinline__ float logit_f32(const float* p) { return *p; }
__device__ __forceinline__ float logit_f32(const uint16_t* p) { return bf16_to_f32(*p); }

// ws: parts [R, nseg] {m_s, z_s, t_s, 0}, then keys [R, nseg, K]
// kFull: the segment has all its kSeg columns (every column a test less)
template <typename IN, bool kTop, bool kFull>
__device__ __forceinline__ void logprobs_segment(const IN* __restrict__ xr, int32_t left, int32_t seg, int32_t K,
                                                 float4* __restrict__ part, unsigned long long* __restrict__ keys) {
    __shared__ __align__(16) float red[kSegWarps];
    __shared__ float red2[kSegWarps], red3[kSegWarps];
    __shared__ TopSmem top;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    auto exists = [&](int k) { return kFull || kSegThreads * k < left; };
    auto at = [&](int k) { return exists(k) ? logit_f32(xr + kSegThreads * k) : -INFINITY; };
    float v[kPerThread];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) v[k] = at(k);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) mx = fmaxf(mx, v[k]);
    const float mine = mx;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(mx) : "f"(mine));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    float m = red[0];
#pragma unroll
    for (int w = 1; w < kSegWarps; ++w) m = fmaxf(m, red[w]);
    float z = 0.0f, t = 0.0f;
    if (m != -INFINITY) {
        float2 tt = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kPerThread; k += 2) {
            const float2 d = tc::add2(make_float2(v[k], v[k + 1]), make_float2(-m, -m));
            const float2 e = make_float2(expf(d.x), expf(d.y));  // (0 for a column that does not exist)
            z = __fadd_rn(__fadd_rn(z, e.x), e.y);
            tt = tc::fma2(e, d, tt);
        }
        t = __fadd_rn(tt.x, tt.y);
        if (isnan(t)) {  // 0 * -inf: an excluded column adds nothing (a NaN among the logits stays, in z)
            t = 0.0f;
            for (int k = 0; k < kPerThread; ++k) {
                const float d = __fsub_rn(at(k), m);
                t = __fmaf_rn(expf(d), fmaxf(d, -FLT_MAX), t);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k)
            if (isnan(v[k])) z = v[k];
    }
    // (a NaN column makes this thread's sum NaN, where there is one)
    const bool odd = m == -INFINITY || isnan(z);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        z = __fadd_rn(z, __shfl_xor_sync(0xffffffffu, z, off));
        t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, off));
    }
    if (lane == 0) {
        red2[warp] = z;
        red3[warp] = t;
    }
    if constexpr (!kTop) __syncthreads();
    uint32_t cut = 0u;
    if constexpr (kTop) {
        // fmaxf passes over NaN: a thread that has one lets the cut know
        bool nan = false;
        if (odd) {
#pragma unroll
            for (int k = 0; k < kPerThread; ++k) nan |= isnan(v[k]);
        }
        cut = top_cut(top, left > 0 ? (nan ? 0u : key_hi(mine)) : ~0u, K);  // (joins the block)
    }
    if (tid == 0) {
        float zs = red2[0], ts = red3[0];
        for (int w = 1; w < kSegWarps; ++w) {
            zs = __fadd_rn(zs, red2[w]);
            ts = __fadd_rn(ts, red3[w]);
        }
        *part = make_float4(m, zs, ts, 0.0f);
    }
    if constexpr (kTop) {
        // key_hi(v) <= cut, decided on the float: its value at the cut
        const uint32_t ord = ~cut;
        const float tau = __uint_as_float((ord & 0x80000000u) ? ord & 0x7fffffffu : ~ord);
        auto list = [&](int k) { list_key(top, argmax_key(v[k], seg * kSeg + tid + kSegThreads * k)); };
        if (cut != 0u && tau > -INFINITY && !odd) {  // (neither NaN nor columns that do not exist pass the test)
            if (mine >= tau) {
#pragma unroll
                for (int k = 0; k < kPerThread; ++k)
                    if (v[k] >= tau) list(k);
            }
        } else {
            const bool any = cut == ~0u;
            for (int k = 0; k < kPerThread; ++k)
                if (exists(k) && (any || (cut == 0u ? isnan(at(k)) : !(at(k) < tau))))
                    list_key(top, argmax_key(at(k), seg * kSeg + tid + kSegThreads * k));
        }
        top_rank(
            top, K,
            [&](int k) { return exists(k) ? argmax_key(v[k], seg * kSeg + tid + kSegThreads * k) : kArgmaxKeyNone; },
            [&](int rank, unsigned long long key) { keys[rank] = key; });
    }
}

template <typename IN, bool kTop>
__global__ void __launch_bounds__(kSegThreads, 6)
token_logprobs_segment_kernel(const IN* __restrict__ x, int64_t stride, int32_t V, int32_t nseg, int32_t K,
                              float4* __restrict__ part, unsigned long long* __restrict__ keys) {
    pdl_trigger();
    pdl_wait();
    const int32_t seg = blockIdx.x;
    const int64_t r = blockIdx.y, at = r * nseg + seg;
    const IN* xr = x + r * stride + seg * kSeg + threadIdx.x;
    const int32_t left = V - seg * kSeg - static_cast<int32_t>(threadIdx.x);  // column k of the thread exists while 256 k < left
    if (V - seg * kSeg >= kSeg) logprobs_segment<IN, kTop, true>(xr, left, seg, K, part + at, keys + at * K);
    else logprobs_segment<IN, kTop, false>(xr, left, seg, K, part + at, keys + at * K);
}

// A row's m, log z and entropy from its segments' parts, in every lane of a warp.
struct RowSums {
    float m, log_z, entropy;
};
__device__ __forceinline__ RowSums row_sums(const float4* __restrict__ pr, int32_t nseg) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int32_t s = lane; s < nseg; s += 32) m = fmaxf(m, pr[s].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    // a term per lane, the sums in segment order
    float z = 0.0f, t = 0.0f;
    for (int32_t s0 = 0; s0 < nseg; s0 += 32) {
        float pz = 0.0f, pt = 0.0f;
        if (s0 + lane < nseg) {
            const float4 p = pr[s0 + lane];
            const float d = __fsub_rn(p.x, m), f = expf(d);
            pz = __fmul_rn(p.y, f);
            // a segment without a finite logit, or too far below m to weigh anything, adds nothing (d may be
            // as low as -FLT_MAX: z_s d overflows); a NaN reaches the entropy through z
            pt = p.y == 0.0f || f == 0.0f ? 0.0f : __fmul_rn(f, __fmaf_rn(p.y, d, p.z));
        }
        const int n = min(32, nseg - s0);
        for (int i = 0; i < n; ++i) {
            z = __fadd_rn(z, __shfl_sync(0xffffffffu, pz, i));
            t = __fadd_rn(t, __shfl_sync(0xffffffffu, pt, i));
        }
    }
    const float lz = logf(z);
    return RowSums{m, lz, __fsub_rn(lz, __fdiv_rn(t, z))};
}

template <typename IN>
__device__ __forceinline__ float token_logprob(const IN* __restrict__ xr, int32_t id, int32_t V, const RowSums& sums,
                                               int32_t* status) {
    if (id >= V) {
        report(status, BI_DEV_BAD_TOKEN);
        return __int_as_float(0x7fffffff);
    }
    return id < 0 ? 0.0f : __fsub_rn(__fsub_rn(logit_f32(xr + id), sums.m), sums.log_z);
}

// Pass 2 without alternatives: a warp per row.
template <typename IN>
__global__ void __launch_bounds__(kSegThreads)
token_logprobs_rows_kernel(const IN* __restrict__ x, int64_t stride, int32_t R, int32_t V, int32_t nseg,
                           const float4* __restrict__ part, const int32_t* __restrict__ tokens,
                           float* __restrict__ logprobs, float* __restrict__ entropy, int32_t P, int32_t* status) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kSegWarps + threadIdx.x / 32;
    if (r >= R) return;
    const RowSums sums = row_sums(part + r * nseg, nseg);
    if (entropy != nullptr && lane == 0) entropy[r] = sums.entropy;
    for (int32_t i = lane; i < P; i += 32)
        logprobs[r * P + i] = token_logprob(x + r * stride, tokens[r * P + i], V, sums, status);
}

// Pass 2 with alternatives: a CTA per row (each warp has the sums of its own).
template <typename IN>
__global__ void __launch_bounds__(kSegThreads)
token_logprobs_merge_kernel(const IN* __restrict__ x, int64_t stride, int32_t V, int32_t nseg,
                            const float4* __restrict__ part, const unsigned long long* __restrict__ keys,
                            const int32_t* __restrict__ tokens, float* __restrict__ logprobs,
                            float* __restrict__ entropy, int32_t* __restrict__ top_ids,
                            float* __restrict__ top_logprobs, int32_t P, int32_t K, int32_t* status) {
    pdl_trigger();
    pdl_wait();
    __shared__ TopSmem top;
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const unsigned long long* kr = keys + r * nseg * K;
    const int32_t total = nseg * K;  // <= kSeg
    unsigned long long mykeys[kPerThread];
    uint32_t best = ~0u;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        mykeys[k] = tid + kSegThreads * k < total ? kr[tid + kSegThreads * k] : kArgmaxKeyNone;
        best = min(best, static_cast<uint32_t>(mykeys[k] >> 32));
    }
    const RowSums sums = row_sums(part + r * nseg, nseg);
    if (entropy != nullptr && tid == 0) entropy[r] = sums.entropy;
    const IN* xr = x + r * stride;
    for (int32_t i = tid; i < P; i += kSegThreads)
        logprobs[r * P + i] = token_logprob(xr, tokens[r * P + i], V, sums, status);
    const uint32_t cut = top_cut(top, best, K);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
        if (mykeys[k] != kArgmaxKeyNone && static_cast<uint32_t>(mykeys[k] >> 32) <= cut) list_key(top, mykeys[k]);
    top_rank(
        top, K, [&](int k) { return mykeys[k]; },
        [&](int rank, unsigned long long key) {
            const int32_t id = static_cast<int32_t>(static_cast<uint32_t>(key));
            top_ids[r * K + rank] = id;
            top_logprobs[r * K + rank] = __fsub_rn(__fsub_rn(logit_f32(xr + id), sums.m), sums.log_z);
        });
}

size_t token_logprobs_ws_bytes(int32_t R, int32_t V, int32_t K) {
    if (R <= 0 || V <= 0 || K < 0) return 0;
    return static_cast<size_t>(R) * logit_segments(V) * (sizeof(float4) + K * sizeof(unsigned long long)) + 256;
}

template <typename IN>
static cudaError_t launch_token_logprobs_t(const IN* x, int64_t stride, const int32_t* tokens, float* logprobs,
                                           float* entropy, int32_t* top_ids, float* top_logprobs, int32_t R, int32_t V,
                                           int32_t P, int32_t K, void* ws, int32_t* status, cudaStream_t s) {
    const int32_t nseg = logit_segments(V);
    float4* parts = static_cast<float4*>(ws);
    unsigned long long* all_keys = reinterpret_cast<unsigned long long*>(parts + static_cast<int64_t>(R) * nseg);
    // the grid's y extent is 16 bits: rows go in slices of it
    for (int32_t r0 = 0; r0 < R; r0 += 65535) {
        const int32_t n = R - r0 < 65535 ? R - r0 : 65535;
        float4* part = parts + static_cast<int64_t>(r0) * nseg;
        unsigned long long* keys = all_keys + static_cast<int64_t>(r0) * nseg * K;
        const IN* xs = x + r0 * stride;
        const dim3 grid(nseg, n);
        cudaError_t e = K > 0 ? launch_pdl(token_logprobs_segment_kernel<IN, true>, grid, dim3(kSegThreads), 0, s, xs,
                                           stride, V, nseg, K, part, keys)
                              : launch_pdl(token_logprobs_segment_kernel<IN, false>, grid, dim3(kSegThreads), 0, s, xs,
                                           stride, V, nseg, K, part, keys);
        if (e != cudaSuccess) return e;
        const int32_t* tok = tokens ? tokens + static_cast<int64_t>(r0) * P : nullptr;
        float* lp = logprobs ? logprobs + static_cast<int64_t>(r0) * P : nullptr;
        float* ent = entropy ? entropy + r0 : nullptr;
        const float4* parts_r0 = part;
        if (K > 0)
            e = launch_pdl(token_logprobs_merge_kernel<IN>, dim3(n), dim3(kSegThreads), 0, s, xs, stride, V, nseg, parts_r0,
                           static_cast<const unsigned long long*>(keys), tok, lp, ent,
                           top_ids + static_cast<int64_t>(r0) * K, top_logprobs + static_cast<int64_t>(r0) * K, P, K, status);
        else
            e = launch_pdl(token_logprobs_rows_kernel<IN>, dim3((n + kSegWarps - 1) / kSegWarps), dim3(kSegThreads), 0, s, xs,
                           stride, n, V, nseg, parts_r0, tok, lp, ent, P, status);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_token_logprobs(const void* logits, bool f32, int64_t row_stride, const int32_t* tokens,
                                  float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs, int32_t R,
                                  int32_t V, int32_t P, int32_t K, void* ws, int32_t* status, cudaStream_t s) {
    if (R <= 0) return cudaSuccess;
    return f32 ? launch_token_logprobs_t(static_cast<const float*>(logits), row_stride, tokens, logprobs, entropy,
                                         top_ids, top_logprobs, R, V, P, K, ws, status, s)
               : launch_token_logprobs_t(static_cast<const uint16_t*>(logits), row_stride, tokens, logprobs, entropy,
                                         top_ids, top_logprobs, R, V, P, K, ws, status, s);
}

}  // namespace bi
