// Page tables and slot maps from request lengths (bi_build_slots), and the
// per-head norm + rotation + append that writes through such a map
// (bi_qk_norm_rope_append).
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace bi {

// ---------------------------------------------------------------------------
// bi_build_slots: two prefix sums over the requests (tokens, pages taken),
// then one binary search per token.
//
// The work is a few integers per token; what counts is latency, so it is one
// launch.  Every CTA sums the request lengths by itself (B integers twice:
// cheaper than passing sums between CTAs) and takes its share of the tokens and
// of the new page-table entries.  Entries read (pages a request already holds)
// and entries written (its new ones) never coincide, so the only order needed
// is between reading free_head everywhere and writing free_head_out: where they
// are one word the CTAs are a cluster and meet at its barrier.  Requests are
// taken kSlotThreads at a time, so B has no limit.  Measured: 64 requests, one
// token each 3.9 us (the launch); 512 requests, 131 k tokens 8.1 us as a
// grid, 22 us as a cluster.
// ---------------------------------------------------------------------------
constexpr int kSlotThreads = 1024;
constexpr int kSlotCluster = 8;

struct SlotArgs {
    const int32_t *q_len, *pos0, *free_pages, *free_head, *depth;
    int32_t *page_table, *free_head_out, *cu_q, *tok_req, *tok_pos, *slots, *status;
    int32_t B, T, max_pages, num_pages, n_free, pad;
};

struct SlotSmem {
    int64_t cu[kSlotThreads + 1];       // first token of each request of this round
    int64_t page_at[kSlotThreads + 1];  // first new page of each, counted from free_head
    int32_t pos0[kSlotThreads];
    int32_t ok[kSlotThreads];
    int64_t warp_q[32], warp_n[32];
    int64_t taken;                      // pages handed out so far
};

// Inclusive sums over the block of two values per thread.
__device__ __forceinline__ void block_scan2(SlotSmem& sm, int64_t& a, int64_t& b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sm.warp_q[warp] = a;
        sm.warp_n[warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t x = sm.warp_q[lane], y = sm.warp_n[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) {
                x += u;
                y += v;
            }
        }
        sm.warp_q[lane] = x;
        sm.warp_n[lane] = y;
    }
    __syncthreads();
    if (warp > 0) {
        a += sm.warp_q[warp - 1];
        b += sm.warp_n[warp - 1];
    }
}

// Last entry of the ascending s[0 .. n) that is <= v (s[0] <= v).
__device__ __forceinline__ int last_le(const int64_t* s, int n, int64_t v) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <bool kClustered>
__global__ void __launch_bounds__(kSlotThreads)
build_slots_kernel(SlotArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ SlotSmem sm;
    const int tid = threadIdx.x;
    const int32_t rank = blockIdx.x, ranks = gridDim.x;
    const int64_t head = a.free_head[0];
    const int64_t avail = head < 0 ? 0 : max(static_cast<int64_t>(a.n_free) - head, static_cast<int64_t>(0));
    if (tid == 0) sm.taken = 0;
    int64_t tok_base = 0, page_base = 0;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * BI_PAGE;
    for (int32_t r0 = 0; r0 < a.B; r0 += kSlotThreads) {
        const int n = min(kSlotThreads, a.B - r0);
        int64_t q = 0, fresh = 0;
        int32_t p0 = 0;
        bool ok = true;
        if (tid < n) {
            q = a.q_len[r0 + tid];
            p0 = a.pos0[r0 + tid];
            ok = q >= 0 && p0 >= 0 && p0 + q <= cap;
            if (!ok) {
                report(a.status, BI_DEV_BAD_POSITION);
                q = max(q, static_cast<int64_t>(0));
            } else if (q > 0) {
                fresh = (p0 + q + BI_PAGE - 1) / BI_PAGE - (static_cast<int64_t>(p0) + BI_PAGE - 1) / BI_PAGE;
            }
        }
        int64_t q_end = q, n_end = fresh;
        __syncthreads();  // the previous round's tables are no longer read
        block_scan2(sm, q_end, n_end);
        if (tid < n) {
            const int64_t first = page_base + n_end - fresh;
            if (fresh > 0 && first + fresh > avail) {
                report(a.status, BI_DEV_NO_PAGES);
                ok = false;
            }
            sm.cu[tid] = tok_base + q_end - q;
            sm.page_at[tid] = first;
            sm.pos0[tid] = p0;
            sm.ok[tid] = ok;
            // the requests that the list serves come first: their end is what was handed out
            if (ok && fresh > 0)
                atomicMax(reinterpret_cast<unsigned long long*>(&sm.taken), static_cast<unsigned long long>(first + fresh));
            if (rank == 0) a.cu_q[r0 + tid] = static_cast<int32_t>(min(sm.cu[tid], static_cast<int64_t>(a.T)));
            if (tid == n - 1) {
                sm.cu[n] = tok_base + q_end;
                sm.page_at[n] = page_base + n_end;
            }
        }
        __syncthreads();
        const int64_t tok_end = sm.cu[n], page_end = sm.page_at[n], step = static_cast<int64_t>(ranks) * kSlotThreads;
        for (int64_t g = page_base + rank * kSlotThreads + tid; g < page_end; g += step) {
            const int i = last_le(sm.page_at, n, g);
            if (sm.ok[i]) {
                const int32_t col = (sm.pos0[i] + BI_PAGE - 1) / BI_PAGE + static_cast<int32_t>(g - sm.page_at[i]);
                a.page_table[static_cast<int64_t>(r0 + i) * a.max_pages + col] = a.free_pages[head + g];
            }
        }
        if (tok_end > a.T && tid == 0 && rank == 0) report(a.status, BI_DEV_BAD_POSITION);
        const int64_t t_end = min(tok_end, static_cast<int64_t>(a.T));
        for (int64_t t = tok_base + rank * kSlotThreads + tid; t < t_end; t += step) {
            const int i = last_le(sm.cu, n, t);
            const int32_t off = static_cast<int32_t>(t - sm.cu[i]);
            const int32_t p0i = sm.pos0[i];
            int32_t slot = -1;
            if (sm.ok[i]) {
                const int32_t at = p0i + off, lp = at / BI_PAGE, have = (p0i + BI_PAGE - 1) / BI_PAGE;
                const int32_t page = lp < have ? a.page_table[static_cast<int64_t>(r0 + i) * a.max_pages + lp]
                                               : a.free_pages[head + sm.page_at[i] + (lp - have)];
                if (page >= 0 && page < a.num_pages) slot = page * BI_PAGE + (at & (BI_PAGE - 1));
                else report(a.status, BI_DEV_BAD_PAGE);
            }
            a.tok_req[t] = r0 + i;
            a.tok_pos[t] = static_cast<int32_t>(static_cast<uint32_t>(p0i) + static_cast<uint32_t>(a.depth ? a.depth[t] : off));
            a.slots[t] = slot;
        }
        tok_base = tok_end;
        page_base = page_end;
    }
    if (a.pad) {
        const int64_t step = static_cast<int64_t>(ranks) * kSlotThreads;
        for (int64_t t = tok_base + rank * kSlotThreads + tid; t < a.T; t += step) a.tok_req[t] = a.tok_pos[t] = a.slots[t] = -1;
    }
    __syncthreads();
    if constexpr (kClustered) ptx::cluster_sync();  // every CTA has read free_head
    if (rank == 0 && tid == 0) {
        a.cu_q[a.B] = static_cast<int32_t>(min(tok_base, static_cast<int64_t>(a.T)));
        a.free_head_out[0] = static_cast<int32_t>(head + sm.taken);
    }
}

cudaError_t launch_build_slots(const int32_t* q_len, const int32_t* pos0, int32_t* page_table,
                               const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                               int32_t* free_head_out, const int32_t* depth, int32_t* cu_q, int32_t* tok_req,
                               int32_t* tok_pos, int32_t* slots, bool pad, int32_t B, int32_t T, int32_t max_pages,
                               int32_t num_pages, int32_t* status, cudaStream_t s) {
    const SlotArgs a{q_len, pos0, free_pages, free_head, depth, page_table, free_head_out, cu_q, tok_req, tok_pos,
                     slots, status, B, T, max_pages, num_pages, n_free, pad};
    // one CTA writes what a decode step needs in one sweep; more tokens than that are shared, by as many CTAs as have
    // a sweep of their own, or by a cluster where the list's head is updated in place
    if (T <= 4 * kSlotThreads || free_head_out != free_head) {
        const int32_t sweeps = T / kSlotThreads, ctas = sweeps <= 4 ? 1 : sweeps < num_sms() ? sweeps : num_sms();
        return launch_pdl(build_slots_kernel<false>, dim3(ctas), dim3(kSlotThreads), 0, s, a);
    }
    return launch_cluster_pdl(build_slots_kernel<true>, kSlotCluster, dim3(kSlotCluster), dim3(kSlotThreads), 0, s, a);
}

// ---------------------------------------------------------------------------
// bi_qk_norm_rope_append: one pass over the projection.
//
// A head's LPH lanes hold it whole: lane l has elements [8l, 8l + 8) and their
// rotation partners Dh/2 further on, so the norm is a sum over LPH lanes and
// the rotation needs no exchange; every load and store is 16 bytes.  A CTA is
// one token; its lanes keep the token's cos and sin for all their heads.  With
// fewer tokens than SMs a token's heads go to several CTAs, each with one sweep
// of them.  Bound by HBM: each element is read once and written once.  Measured
// on 411 MB (16384 tokens, bf16, 32 + 16 heads of 128, norms): 71.6 us with 64
// threads, 5.7 TB/s; 74.1 with 128, 100 with 256, whose last sweep leaves lanes
// idle.
// ---------------------------------------------------------------------------
constexpr int kQkThreads = 64;

struct QkArgs {
    const void* qkv;
    const uint16_t *q_gamma, *k_gamma;
    const int32_t *tok_pos, *slots;
    const float *rc, *rs;
    uint16_t *q_out, *kc, *vc;
    int32_t* status;
    float eps;
    int32_t max_pos, num_pages, H, Hkv, Dh;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), x); }

template <typename IN, int LPH>
__global__ void __launch_bounds__(kQkThreads)
qk_norm_rope_append_kernel(QkArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int kGroups = kQkThreads / LPH;
    const int32_t t = blockIdx.x, half = a.Dh / 2, heads = a.H + 2 * a.Hkv;
    const int l = threadIdx.x % LPH;
    const bool on = 8 * l < half;
    const int32_t pos = a.tok_pos[t], slot = a.slots[t];
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const bool slot_ok = slot >= 0 && slot / BI_PAGE < a.num_pages;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        if (!pos_ok && (pos != -1 || slot != -1)) report(a.status, BI_DEV_BAD_POSITION);
        else if (pos_ok && !slot_ok && slot != -1) report(a.status, BI_DEV_BAD_PAGE);
    }
    float c[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        sn[i] = 0.0f;
    }
    if (pos_ok && on) {
        load8(a.rc + static_cast<int64_t>(pos) * half + 8 * l, c);
        load8(a.rs + static_cast<int64_t>(pos) * half + 8 * l, sn);
    }
    const IN* row = static_cast<const IN*>(a.qkv) + static_cast<int64_t>(t) * heads * a.Dh + 8 * l;
    for (int32_t h0 = blockIdx.y * kGroups; h0 < heads; h0 += gridDim.y * kGroups) {  // uniform: every lane takes part in the sums
        const int32_t h = h0 + threadIdx.x / LPH;
        const bool live = on && h < heads;
        float lo[8], hi[8];
        if (live) {
            load8(row + static_cast<int64_t>(h) * a.Dh, lo);
            load8(row + static_cast<int64_t>(h) * a.Dh + half, hi);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0.0f;
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(lo[i], lo[i], ss);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(hi[i], hi[i], ss);
#pragma unroll
        for (int off = LPH / 2; off >= 1; off >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
        if (!live) continue;
        if (h < a.H + a.Hkv) {
            const uint16_t* gamma = h < a.H ? a.q_gamma : a.k_gamma;
            if (gamma != nullptr) {
                const float rinv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(a.Dh)), a.eps)));
                float g[8];
                load8(gamma + 8 * l, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[i] = __fmul_rn(__fmul_rn(lo[i], rinv), g[i]);
                load8(gamma + half + 8 * l, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) hi[i] = __fmul_rn(__fmul_rn(hi[i], rinv), g[i]);
            }
            // rotate-half, each product rounded before the sum (as rope_append_kernel)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float r0 = __fsub_rn(__fmul_rn(lo[i], c[i]), __fmul_rn(hi[i], sn[i]));
                const float r1 = __fadd_rn(__fmul_rn(hi[i], c[i]), __fmul_rn(lo[i], sn[i]));
                lo[i] = r0;
                hi[i] = r1;
            }
        }
        uint16_t* dst;
        if (h < a.H) {
            dst = a.q_out + (static_cast<int64_t>(t) * a.H + h) * a.Dh;
        } else {
            if (!pos_ok || !slot_ok) continue;
            const bool is_k = h < a.H + a.Hkv;
            const int32_t g = is_k ? h - a.H : h - a.H - a.Hkv;
            dst = (is_k ? a.kc : a.vc) +
                  ((static_cast<int64_t>(slot / BI_PAGE) * a.Hkv + g) * BI_PAGE + (slot & (BI_PAGE - 1))) * a.Dh;
        }
        *reinterpret_cast<uint4*>(dst + 8 * l) = pack8(lo);
        *reinterpret_cast<uint4*>(dst + half + 8 * l) = pack8(hi);
    }
}

template <typename IN>
static cudaError_t launch_qk_t(const QkArgs& a, int32_t T, cudaStream_t s) {
    const int32_t per = a.Dh / 16;  // lanes a head needs
    auto go = [&](auto kernel, int32_t lanes) {
        const int32_t groups = kQkThreads / lanes, sweeps = (a.H + 2 * a.Hkv + groups - 1) / groups;
        const int32_t split = T >= num_sms() ? 1 : sweeps < 64 ? sweeps : 64;
        return launch_pdl(kernel, dim3(T, split), dim3(kQkThreads), 0, s, a);
    };
    if (per <= 4) return go(qk_norm_rope_append_kernel<IN, 4>, 4);
    if (per <= 8) return go(qk_norm_rope_append_kernel<IN, 8>, 8);
    return go(qk_norm_rope_append_kernel<IN, 16>, 16);
}

cudaError_t launch_qk_norm_rope_append(const void* qkv, bool f32, const bi_bf16* q_gamma, const bi_bf16* k_gamma,
                                       float eps, const int32_t* tok_pos, const int32_t* slots, const float* rc,
                                       const float* rs, int32_t max_pos, bi_bf16* q_out, bi_bf16* kc, bi_bf16* vc,
                                       int32_t num_pages, int32_t T, int32_t H, int32_t Hkv, int32_t Dh,
                                       int32_t* status, cudaStream_t s) {
    if (T <= 0) return cudaSuccess;
    const QkArgs a{qkv, q_gamma, k_gamma, tok_pos, slots, rc, rs, q_out, kc, vc, status, eps,
                   max_pos, num_pages, H, Hkv, Dh};
    return f32 ? launch_qk_t<float>(a, T, s) : launch_qk_t<uint16_t>(a, T, s);
}

}  // namespace bi
