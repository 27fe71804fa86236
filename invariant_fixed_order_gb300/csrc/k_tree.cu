// Attention of drafted nodes over the paged cache (bi_tree_attention), on the
// tcgen05 tensor cores.
//
// out = sum_j softmax_j(scale q.k_j) v_j over the positions a node attends: its
// request's context and, by the bits of its mask row, nodes of its own request.
//
// Work.  A tile is 128 (node, head) rows of one request and one KV head (128/G
// consecutive nodes x the G heads of the group; row = tensor-memory lane).  Its
// keys are cut into segments of whole steps (128 positions; segment_steps, a
// function of the request alone), and a segment is walked in half steps of 64:
//   S = Q K^T              tcgen05 128 x 64 x Dh, bf16 in, fp32 in TMEM
//   p = 2^(S c - M)        c = scale * log2 e; M, a row's reference, is its
//                          first half step's maximum and follows a later one
//                          only when that exceeds it by 2^8 (a sum stays below
//                          2^8 per key, far inside fp32; the factor 2^(M_old -
//                          M) is then applied to O and L)
//   L = L + sum p          fp32, of the unrounded p
//   O = O + P V            tcgen05 128 x Dh x 16 keys, accumulated in TMEM
// P is taken as bf16 hi + lo parts (p to 2^-16), as in the decode and prefill
// kernels: one part would be off by up to 2^-8 of each p, which over few keys is
// as much as a bf16 output's own rounding.  Outputs of either type are the same
// fp32 values, rounded once where they are bf16.  A segment's M, L and O go to
// the workspace and tree_merge_kernel folds them in ascending order,
//   M' = max(M, m), L' = L 2^(M-M') + l 2^(m-M'), O' likewise.
// All of that belongs to the request alone.  Which CTA computes a segment does
// not: the launch's segments, laid end to end, are cut into one contiguous range
// of equal work per CTA.
//
// A CTA has two lanes, each with its queries, two score buffers and O: two
// tiles of a request that read the same keys (one copy of K and V serves both),
// or two segments of a lone tile.  Roles: warps 0-3 and 4-7 the softmax of a
// lane, one thread per row; warps 8 and 10 copy pages by TMA, each half of
// every stage, K two steps ahead of V and on from run to run; warps 9 and 11
// issue a lane's products.  In a lane S (h + 2) follows P V (h) in order, so the
// scores of a half step are ready when its warps come to it, and S and P share
// columns without a wait of their own.
//
// Bound.  Lone tiles by HBM: a step's 64 KB of K and V take one SM's share of
// the copy bandwidth 1.5 us.  Pairs of tiles by the softmax warps: they take a
// half step's scores, exponentials and parts of P one after the other, while the
// tensor pipe is busy for 47 % of the cycles and DRAM for 42 (24 requests).
// Measured (32 query heads, 8 KV heads, Dh 128): 16 requests with up to 16 nodes
// over up to 8192 positions 79 us (46 for the bytes), 64 requests with 33 to 64
// nodes 390 us (188).  What remains is the ranges' unequal ends (runs are whole
// segments; 10 to 20 %), the partials, and a CTA's start and end.  P's lo part is
// 6 and 66 us of it.
//
// What the other layouts measured on the 16 / 64 requests, with P in one part
// (73 / 326 us in this one): one lane whose two warpgroups take steps in turn 78 /
// 508 us (each tile copies its keys again); O in registers, 16 warps with four
// threads to a row 96 / 538.
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "tc_tmem.cuh"

namespace bi {
namespace tree {

using namespace tc;

constexpr int kRows = 128;
constexpr int kStep = 128;                 // keys per step
constexpr int kStepPages = kStep / BI_PAGE;
constexpr int kHalf = kStep / 2;           // keys per half step: one score buffer
constexpr int kSoft = 256;                 // softmax threads: a warpgroup for each lane, one thread per row
constexpr int kSoftWarps = kSoft / 32;
constexpr int kThreads = kSoft + 128;      // warps 8 and 10 copy, warps 9 and 11 issue products (of a lane)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;              // two score buffers of 64 columns for each lane, P in place
constexpr uint32_t kColO = 4 * kHalf;      // O of each lane
constexpr int kRegion = kStep * 128;       // 64 dims of a stage (or of Q): 128 rows of 128 bytes, swizzled
constexpr float kSlack = 8.0f;             // growth of a row's maximum (log2) before its reference follows

// A run: a segment of one tile (kind 1), two segments of one tile side by side
// (kind 2), or a segment of two tiles that read the same keys (kind 3).
struct RunDesc {
    int32_t kind;                          // 0: no more runs
    int32_t g, r, p0, n, len;              // KV head, request, its context, nodes and keys
    int32_t t0[2], rows[2], j0[2], steps[2], new_q[2];  // by lane: first token, rows, first step, steps, queries change
    int64_t part[2];                       // where its partial goes
    // Steps of K (and of V) come in a sequence that both lanes follow: A0 B0 A1 B1 ..., the longer lane's rest, or
    // one sequence for both.
    __device__ __forceinline__ int32_t items() const { return kind == 2 ? steps[0] + steps[1] : steps[0]; }
};
__device__ __forceinline__ int32_t item_of(int32_t kind, int32_t lane_id, int32_t j, int32_t steps_b) {
    return kind != 2 ? j : lane_id == 0 ? j + min(j, steps_b) : 2 * j + 1;
}

// Partials, for each segment of each tile: tiles are counted over the whole
// launch by tile_id, x Hkv, x slots segments.
struct Layout {
    float2* ml;            // [.., rows] reference and sum
    float4* o;             // [.., DH / 4, rows] unnormalised O: rows side by side, so that a warp's rows are one access
    int32_t slots, rows;   // segments and rows a tile may have
};
// Tile tl of request r, which owns tokens from c0 on: distinct, and below T / NT + B.
__device__ __forceinline__ int64_t tile_id(int32_t r, int32_t c0, int32_t tl, int32_t NT) { return c0 / NT + r + tl; }

template <int DH>
struct Smem {
    static constexpr int kRegions = DH / 64;
    static constexpr int kStagesK = DH == 128 ? 3 : 5, kStagesV = DH == 128 ? 2 : 4;
    // K: per 64 dims, 128 rows of 128 bytes; V: per page and 64 dims, 16 rows of 128 bytes (both swizzled)
    uint8_t k[kStagesK][kRegions * kRegion];   // 1024-aligned (first)
    uint8_t v[kStagesV][kRegions * kRegion];
    uint8_t q[2][kRegions * kRegion];          // by lane
    // a stage's copies have landed / both lanes are done with it
    uint64_t k_full[kStagesK], k_free[kStagesK], v_full[kStagesV], v_free[kStagesV];
    // by lane (and parity of its half steps, or of the runs):
    uint64_t q_full[2], q_free[2];
    uint64_t s_full[2][2], p_full[2][2];       // scores ready / P written
    uint64_t o_prev[2], o_done[2];             // P V of a run's last half step but one / of its last done
    uint64_t v_seen[2];                        // V of a step with nodes has landed
    uint64_t o_free[2];                        // a run's O read
    uint64_t run_full[2][2];                   // P of a run's last half step written
    uint64_t rd_full[2], rd_free[2];
    uint64_t drain[2];
    uint32_t k_issued[2][kStagesK], v_issued[2][kStagesV], q_issued[2];  // fills so far (by copying warp)
    uint32_t tmem_base;
    int32_t abort;
    uint32_t bad[2][BI_TREE_MAX_NODES / 32];   // nodes whose V is not finite, by run parity
    RunDesc rd[2];
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The maximum of N scores (a NaN is passed over).
template <int N>
__device__ __forceinline__ float max_of(const uint32_t (&s)[N]) {
    float m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        m[u] = fmaxf(__uint_as_float(s[u]), __uint_as_float(s[4 + u]));
#pragma unroll
        for (int x = 8; x < N; x += 8) m[u] = max3(m[u], __uint_as_float(s[x + u]), __uint_as_float(s[x + 4 + u]));
    }
    return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// Steps per segment of a request of so many steps whose rows make `tiles` tiles
// over all KV heads.  A segment costs a partial of each of its tiles, written
// and read (66 KB at most; a step's K and V are 64 KB), and a change of run;
// what it gives is CTAs for a request with few of its own.  So a request is cut
// into about kSegRuns pieces (tiles x segments), a segment is at least 2 steps,
// and no more than kSegLong, or kSegPairs where there are tiles enough to share
// their keys in pairs: longer ones spread a batch unevenly.  The number of
// segments is bounded, which bounds the workspace.
// Measured, us, means over 60 random sets of lengths of each kind: lone requests
// of 150 to 32000 positions with 8 tiles, 16 tiles, 2 KV heads / 2 to 4 requests of
// 8000 to 32000 with 2 KV heads, 2 to 6 of 4000 to 32000 with 8 / 16 and 64 requests
// of up to 8192 with 8 tiles, 64 with 16:
//   as below        19.3 28.7 23.1 / 47.3 81.2 / 80.9 248 373
//   kSegLong 7      18.2 28.7 21.1 / 47.4 82.3 / 80.4 255 371
//   kSegLong 8      18.5 28.7 21.8 / 47.5 82.3 / 80.1 252 372
//   kSegLong 11     19.6 28.7 23.7 / 46.3 81.6 / 81.4 248 374
//   kSegRuns 40     18.8 27.6 22.7 / 47.5 81.5 / 82.0 256 386
//   kSegPairs 20    19.2 31.0 23.1 / 47.3 81.2 / 80.9 248 371
// and over 30 sets, against the like: kSegRuns 24 1 to 6 % longer for lone requests
// and 1 to 2 % for batches; kSegShort 1 within 2 %; kSegPairs 8 13 % shorter for a
// lone request of 16 tiles, 10 % longer for 64.  From 7 to 11 kSegLong trades lone
// requests for batches, a few percent either way.
constexpr int32_t kSegRuns = 32, kSegShort = 2, kSegLong = 10, kSegPairs = 16, kPairTiles = 16, kFewTiles = 8;
__host__ __device__ constexpr int32_t segments_bound(int32_t tiles) {
    return tiles >= kFewTiles ? BI_TREE_MAX_SEGMENTS / 2 : BI_TREE_MAX_SEGMENTS;
}
__host__ __device__ constexpr int32_t longest_segment(int32_t tiles) { return tiles >= kPairTiles ? kSegPairs : kSegLong; }
__host__ __device__ constexpr int32_t segment_steps(int32_t steps, int32_t tiles) {
    const int64_t even = (static_cast<int64_t>(steps) * tiles + kSegRuns - 1) / kSegRuns;
    const int32_t most = longest_segment(tiles), least = (steps + segments_bound(tiles) - 1) / segments_bound(tiles);
    const int32_t s = even < kSegShort ? kSegShort : even > most ? most : static_cast<int32_t>(even);
    return s > least ? s : least;
}
// The most segments that a request of up to so many steps has.  It has a tile for
// each KV head at least, and fewer segments with more tiles; of s steps each they
// are ceil(steps / s), where s >= 2 and either s >= steps tiles / kSegRuns or s is
// the longest.
static int32_t most_segments(int32_t steps, int32_t Hkv) {
    const int32_t runs = (kSegRuns + Hkv - 1) / Hkv, full = (steps + longest_segment(Hkv) - 1) / longest_segment(Hkv);
    const int32_t n = runs > full ? runs : full, shortest = (steps + kSegShort - 1) / kSegShort;
    const int32_t m = n < shortest ? n : shortest;
    return m < segments_bound(Hkv) ? m : segments_bound(Hkv);
}

// Work of a run, in steps of K and V: its own, and what the change of queries,
// the nodes' masks and the partials cost on top.
constexpr int kRunCost = 2;
// First step of CTA c's range of the launch's work W.
__device__ __forceinline__ int64_t range_begin(int64_t W, int32_t c, int32_t C) { return c * W / C; }

// The fold of two partials' scales; an empty partial (m = -inf) weighs 0.
struct Fold {
    float m, a, b;
};
__device__ __forceinline__ Fold fold_scales(float M, float m) {
    Fold f;
    f.m = fmaxf(M, m);
    const float z = f.m == -INFINITY ? 0.0f : f.m;
    f.a = ex2(__fsub_rn(M, z));
    f.b = ex2(__fsub_rn(m, z));
    return f;
}
__device__ __forceinline__ float fold_value(const Fold& f, float X, float x) {
    return __fadd_rn(__fmul_rn(X, f.a), __fmul_rn(x, f.b));
}
// Row's output factor: 1 / L, or 0 where nothing was attended (L is 0 then and only then; O is 0 too).
__device__ __forceinline__ float out_factor(float L) { return L == 0.0f ? 0.0f : __frcp_rn(L); }

// Which of the 32 positions from kb on a node attends, as bits: the context,
// and the nodes of its mask row (NULL: a row past the tile's last).
__device__ __forceinline__ uint32_t visible(const uint32_t* mask, int32_t kb, int32_t p0, int32_t n) {
    uint32_t bits = kb >= p0 ? 0u : (p0 - kb >= 32 ? ~0u : (1u << (p0 - kb)) - 1u);
    const int32_t rel = kb - p0;  // the node at bit 0 (negative: bit -rel is node 0)
    if (mask == nullptr || rel >= n || rel <= -32) return bits;
    uint32_t m;
    if (rel >= 0) {
        const int32_t w = rel >> 5;
        m = mask[w];
        if (rel & 31) m = __funnelshift_r(m, (w + 1) * 32 < n ? mask[w + 1] : 0u, rel & 31);
    } else {
        m = mask[0] << -rel;
    }
    const int32_t live = n - rel;  // bits below it are the request's
    if (live < 32) m &= (1u << live) - 1u;
    return bits | m;
}

// ---------------------------------------------------------------------------
// The copying warps: this CTA's range as runs, and their copies as the
// buffers come free.  Both walk the same runs; the first writes their
// descriptors and copies the queries, and each copies half the pages of every
// stage (a box takes one warp about 80 cycles to issue).  A page of K is one
// box per 64 dims, so that a step's keys lie as one operand; a page of V, 16
// keys, is the operand of one product, and one box.  Copies go out in the
// order of use, K two items ahead of V, on from one run to the next.
// ---------------------------------------------------------------------------

template <int G, int DH, bool kFirst, bool kTest>
__device__ __forceinline__ void produce(Smem<DH>& sm, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                        const CUtensorMap* tmQ, const TreeArgs& a, int32_t slots) {
    constexpr int NT = kRows / G;
    constexpr int kRegions = DH / 64, kStagesK = Smem<DH>::kStagesK, kStagesV = Smem<DH>::kStagesV;
    const int lane = threadIdx.x & 31;
    volatile int32_t* abort = &sm.abort;
    const int32_t C = gridDim.x, cta = blockIdx.x;
    bool ok = true;
    const uint64_t policy = ptx::policy_evict_normal();  // (a request's other tiles read the same pages)
    uint32_t runs = 0, base = 0, last_base = 0, q_runs[2] = {0, 0};  // runs, items, those before the last run, runs of each lane
    int64_t last_q[2] = {-1, -1};  // the tiles whose queries the lanes have
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        bool r = true;
        if (lane == 0) r = wait_bounded(bar, parity, abort);
        return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
    };

    // This warp's pages of K or V of item `at` of the CTA: first rows (a page for each group of lanes) and number.
    struct Copy {
        int32_t y, np;
    };
    Copy late0{0, 0}, late1{0, 0};  // the items whose V is still to be copied: of even and odd place in the CTA
    constexpr int kWarp = kFirst ? 0 : 1, kPages = kStepPages / 2, kFrom = kWarp * kPages;
    auto withheld = [&](uint32_t at, int v) { return kTest && a.skip_copy == static_cast<int32_t>(4 * at) + 2 * v + kWarp; };
    auto arm = [&](uint64_t* full, int32_t np, uint32_t* issued, uint32_t fills) {
        if (lane == 0) {
            *issued = fills;
            ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(np * kRegions * BI_PAGE * 128));
        }
        __syncwarp();
    };
    auto copy_k = [&](uint32_t at, const Copy& c) {
        const uint32_t st = at % kStagesK;
        if (at >= kStagesK && !wait(&sm.k_free[st], (at / kStagesK - 1) & 1u)) return false;
        if (withheld(at, 0)) return true;
        arm(&sm.k_full[st], c.np, &sm.k_issued[kWarp][st], at / kStagesK + 1);
        const int h = lane / kPages, x = lane & (kPages - 1);
        if (h < kRegions && x < c.np)
            ptx::tma_load_2d(&sm.k[st][h * kRegion + (kFrom + x) * (BI_PAGE * 128)], tmK, &sm.k_full[st], h * 64, c.y);
        __syncwarp();
        return true;
    };
    auto copy_v = [&](uint32_t at, const Copy& c) {
        const uint32_t st = at % kStagesV;
        if (at >= kStagesV && !wait(&sm.v_free[st], (at / kStagesV - 1) & 1u)) return false;
        if (withheld(at, 1)) return true;
        arm(&sm.v_full[st], c.np, &sm.v_issued[kWarp][st], at / kStagesV + 1);
        if (lane < c.np)
            ptx::tma_load_3d(&sm.v[st][(kFrom + lane) * (kRegions * BI_PAGE * 128)], tmV, &sm.v_full[st], 0, c.y, 0, policy);
        __syncwarp();
        return true;
    };
    uint32_t v_next = 0;  // first item whose V has not been copied
    auto copy_v_to = [&](uint32_t to) {
        for (; v_next < to; ++v_next)
            if (!copy_v(v_next, v_next & 1u ? late1 : late0)) return false;
        return true;
    };

    // one request per lane
    int32_t c0 = 0, n = 0, p0 = 0, steps = 1, tiles = 0, ss = 1;
    // Of one KV head of a request: segment by segment its pairs of tiles, then the odd tile's segments.
    auto pairs_work = [](int32_t steps, int32_t tiles, int32_t nseg) {
        return static_cast<int64_t>(tiles >> 1) * (steps + nseg * kRunCost);
    };
    auto head_work = [](int32_t steps, int32_t tiles, int32_t ss) {
        return static_cast<int64_t>((tiles + 1) >> 1) * (steps + (steps + ss - 1) / ss * kRunCost);
    };
    int64_t incl = 0;  // work of the batch up to and with this lane's request
    auto load_batch = [&](int32_t b0) {  // -> its work
        const int32_t r = b0 + lane;
        n = tiles = 0;
        steps = 1;
        if (r < a.B) {
            c0 = a.cu_q[r];
            const int32_t c1 = a.cu_q[r + 1];
            p0 = a.pos0[r];
            const bool rows_ok = c0 >= 0 && c1 >= c0 && c1 <= a.T;
            n = rows_ok ? c1 - c0 : 0;
            const bool valid = p0 >= 0 && n <= a.max_nodes && static_cast<int64_t>(p0) + n <= a.max_seq;
            if (kFirst && (!rows_ok || (!valid && n > 0))) report(a.status, BI_DEV_BAD_POSITION);
            steps = valid ? max((p0 + n + kStep - 1) / kStep, 1) : 1;
            tiles = valid ? (n + NT - 1) / NT : 0;  // (the merge writes the rows of others)
        }
        ss = segment_steps(steps, tiles * a.Hkv);
        incl = a.Hkv * head_work(steps, tiles, ss);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        return __shfl_sync(0xffffffffu, incl, 31);
    };
    int64_t W = 0, batch = 0, before = 0;  // work of the launch, of this batch of requests and of those before it
    for (int32_t b0 = 0; b0 < a.B; b0 += 32) {
        batch = load_batch(b0);
        W += batch;
    }
    const int64_t w0 = range_begin(W, cta, C), w1 = range_begin(W, cta + 1, C);
    int32_t b0 = 0;
    if (a.B > 32) batch = load_batch(0);

    for (int64_t pos = w0; pos < w1 && ok;) {
        while (pos >= before + batch) {  // pos < W: a later batch holds it
            before += batch;
            b0 += 32;
            batch = load_batch(b0);
        }
        const int L = __ffs(__ballot_sync(0xffffffffu, incl > pos - before)) - 1;
        auto pick = [&](int32_t v) { return __shfl_sync(0xffffffffu, v, L); };
        const int32_t rc0 = pick(c0), rn = pick(n), rp0 = pick(p0), rsteps = pick(steps), rtiles = pick(tiles);
        const int32_t rss = pick(ss), nseg = (rsteps + rss - 1) / rss, r = b0 + L, len = rp0 + rn;
        const int64_t head = head_work(rsteps, rtiles, rss), end = before + __shfl_sync(0xffffffffu, incl, L);
        const int32_t pairs = rtiles >> 1;
        const int64_t in_pairs = pairs_work(rsteps, rtiles, nseg), seg_work = static_cast<int64_t>(pairs) * (rss + kRunCost);
        const int32_t lone_work = rss + kRunCost;
        auto seg_steps = [&](int32_t s) { return s < nseg ? min(rss, rsteps - s * rss) : 0; };
        // the first run that begins at or after pos
        int64_t off = pos - (end - a.Hkv * head);
        int32_t g = static_cast<int32_t>(off / head), s, u = 0;
        off -= g * head;
        bool lone = off >= in_pairs;
        if (lone) {
            off -= in_pairs;
            s = static_cast<int32_t>((off + lone_work - 1) / lone_work);
        } else {
            s = min(static_cast<int32_t>(off / seg_work), nseg - 1);
            off -= s * seg_work;
            const int32_t one = seg_steps(s) + kRunCost;
            u = static_cast<int32_t>((off + one - 1) / one);
        }
        pos = end;
        const int32_t* table = a.page_table + static_cast<int64_t>(r) * a.max_pages;
        for (int32_t kind; ok; lone ? s += kind : ++u) {
            if (!lone && u >= pairs) {
                u = 0;
                ++s;
            }
            if (!lone && s >= nseg) {
                lone = true;
                s = 0;
            }
            if (lone && ((rtiles & 1) == 0 || s >= nseg)) {
                ++g;
                lone = pairs == 0;
                s = u = 0;
            }
            if (g >= a.Hkv) break;
            const int64_t begin = end - (a.Hkv - g) * head +
                                  (lone ? in_pairs + static_cast<int64_t>(s) * lone_work
                                        : s * seg_work + static_cast<int64_t>(u) * (seg_steps(s) + kRunCost));
            if (begin >= w1) {
                pos = w1;
                break;
            }
            // two segments of the odd tile side by side where this CTA has both
            kind = !lone ? 3 : s + 1 < nseg && begin + lone_work < w1 ? 2 : 1;
            const int32_t sb = lone ? s + 1 : s, steps_a = seg_steps(s), steps_b = kind == 1 ? 0 : seg_steps(sb);
            const int32_t tl_a = lone ? rtiles - 1 : 2 * u, tl_b = lone ? tl_a : tl_a + 1;
            const int32_t lanes = kind == 1 ? 1 : 2;
            // (a tile's first token and KV head tell it)
            const int64_t q_a = static_cast<int64_t>(rc0 + tl_a * NT) * a.Hkv + g, q_b = static_cast<int64_t>(rc0 + tl_b * NT) * a.Hkv + g;
            const bool new_q[2] = {q_a != last_q[0], q_b != last_q[1]};
            if constexpr (kFirst) {
                const int slot = runs & 1;
                // (the run before the last ends only with all its V)
                if (runs >= 2 && !(ok = copy_v_to(last_base) && wait(&sm.rd_free[slot], ((runs >> 1) - 1) & 1u))) break;
                if (lane < BI_TREE_MAX_NODES / 32) sm.bad[slot][lane] = 0u;
                if (lane < 2) {
                    const int32_t tl = lane ? tl_b : tl_a;
                    RunDesc& rd = sm.rd[slot];
                    rd.t0[lane] = rc0 + tl * NT;
                    rd.rows[lane] = min(NT, rn - tl * NT) * G;
                    rd.j0[lane] = (lane ? sb : s) * rss;
                    rd.steps[lane] = lane ? steps_b : steps_a;
                    rd.new_q[lane] = lane ? new_q[1] : new_q[0];
                    rd.part[lane] = (tile_id(r, rc0, tl, NT) * a.Hkv + g) * slots + (lane ? sb : s);
                    if (lane == 0) {
                        rd.kind = kind;
                        rd.g = g;
                        rd.r = r;
                        rd.p0 = rp0;
                        rd.n = rn;
                        rd.len = len;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.rd_full[slot]);
                ++runs;
            }
            // pages of the next 4 steps of a lane, read while the last 4 are copied
            auto load_pages = [&](int32_t window) {
                const int32_t lp = window * 32 + lane;
                return lp * BI_PAGE < len ? __ldg(table + lp) : 0;
            };
            int32_t now[2] = {0, 0}, next[2] = {load_pages(s * rss >> 2), steps_b > 0 && lone ? load_pages(sb * rss >> 2) : 0};
            const int32_t items = kind == 2 ? steps_a + steps_b : steps_a;
            // The lanes' queries: at once in the first run, else before K(1), when the scores of the run before are
            // done or need nothing that is still to be copied.  In any case before a lane's last K: with the queries
            // that it has, it may go through all its scores and let them go once more, unseen.
            const int32_t q_at = q_runs[0] == 0 || steps_a == 1 ? 0 : 1;
            for (int32_t m = 0; m < items; ++m) {
                if (kFirst && m == q_at) {
                    if (!(ok = base + m == 0 || copy_v_to(base + m - 1))) break;
                    for (int q = 0; q < lanes && ok; ++q) {
                        const uint32_t uses = q == 0 ? q_runs[0] : q_runs[1];
                        if (uses > 0 && !(ok = wait(&sm.q_free[q], (uses - 1) & 1u))) break;
                        if (q == 0) ++q_runs[0]; else ++q_runs[1];
                        if (q == 0 ? !new_q[0] : !new_q[1]) continue;
                        if (lane == 0) {
                            ++sm.q_issued[q];
                            ptx::mbar_arrive_expect_tx(&sm.q_full[q], static_cast<uint32_t>(kRegions * kRegion));
#pragma unroll
                            for (int h = 0; h < kRegions; ++h)
                                ptx::tma_load_3d(&sm.q[q][h * kRegion], tmQ, &sm.q_full[q], h * 64, g * G,
                                                 rc0 + (q == 0 ? tl_a : tl_b) * NT, policy);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    last_q[0] = q_a;
                    if (lanes == 2) last_q[1] = q_b;
                }
                const bool lane_b = kind == 2 && m < 2 * steps_b && (m & 1);
                const int32_t in_run = kind != 2 ? m : m < 2 * steps_b ? m >> 1 : m - steps_b;
                const int32_t j = (lane_b ? sb : s) * rss + in_run;
                if (in_run == 0 || (j & 3) == 0) {
                    int32_t page = lane_b ? next[1] : next[0];
                    if (page < 0 || page >= a.num_pages) {
                        report(a.status, BI_DEV_BAD_PAGE);
                        page = 0;
                    }
                    const int32_t after = load_pages((j >> 2) + 1);
                    if (lane_b) {
                        now[1] = page;
                        next[1] = after;
                    } else {
                        now[0] = page;
                        next[0] = after;
                    }
                }
                const int32_t np = min(max((min(kStep, len - j * kStep) + BI_PAGE - 1) / BI_PAGE - kFrom, 0), kPages);
                const int32_t page = __shfl_sync(0xffffffffu, lane_b ? now[1] : now[0], (j & 3) * kStepPages + kFrom + (lane & (kPages - 1)));
                const Copy copy{(page * a.Hkv + g) * BI_PAGE, np};
                if (!(ok = copy_k(base + m, copy))) break;
                const bool odd = (base + m) & 1u;
                if (base + m >= 2 && !(ok = copy_v_to(base + m - 1))) break;
                if (odd) late1 = copy; else late0 = copy;
            }
            last_base = base;
            base += items;
        }
    }
    ok = ok && copy_v_to(base);
    if constexpr (kFirst) {
        if (ok) {
            const int slot = runs & 1;
            if (runs >= 2) ok = wait(&sm.rd_free[slot], ((runs >> 1) - 1) & 1u);
            if (ok && lane == 0) {
                sm.rd[slot].kind = 0;
                mbar_arrive(&sm.rd_full[slot]);
            }
        }
    }
    if (lane == 0 && !ok) {
        report(a.status, BI_DEV_TIMEOUT_ATTENTION);
        *abort = 1;
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// The warp that issues the products.  Every lane runs the same code on the
// same values and one elected lane issues, so that descriptors and addresses
// stay in uniform registers (issued by a lane on its own branch, each product
// first moved its operands there: 129 cycles apart instead of the 64 a
// 128 x 128 x 16 product takes).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_ss_elected(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts_elected(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(at), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// The products of a lane, by half steps of 64 keys: S0, S1, then P V (h), S (h + 2):
// the scores take the buffer whose P was multiplied just before them, in order.
// Every stage of K and V is waited for and let go by both lanes, in turn, so
// that none can take one fill's phase for another's.
template <int DH, bool kTest>
__device__ __forceinline__ void issue_products(Smem<DH>& sm, uint32_t tmem, int lane_id, uint64_t wait_ns) {
    constexpr int kStagesK = Smem<DH>::kStagesK, kStagesV = Smem<DH>::kStagesV;
    constexpr uint32_t kUnit = 16;  // a descriptor's address field counts 16 bytes: steps of an operand are added to it
    const uint32_t idesc_s = ptx::idesc_bf16_f32(kRows, kHalf);
    const uint32_t idesc_pv = ptx::idesc_bf16_f32(kRows, DH) | (1u << 16);  // B (V) MN-major
    const uint64_t qd = desc(smem_u32(&sm.q[lane_id][0]), 16, 1024);
    const uint32_t col_s = tmem + kColS + lane_id * kStep, col_o = tmem + kColO + lane_id * DH;
    const int lane = threadIdx.x & 31;
    volatile int32_t* abort = &sm.abort;
    // runs, this lane's runs, its half steps and the fills of its Q, items of earlier runs
    uint32_t runs = 0, mine = 0, halves = 0, fills = 0, base = 0;
    uint32_t next_k = 0, next_v = 0;                    // items of K and V seen
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort, kTest ? wait_ns : kWaitLimitNs); };
    auto same = [](int32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
    // waits for item `to`; the ones before it are the other lane's
    auto see_k = [&](uint32_t to, bool own) {
        for (; next_k < to + own; ++next_k) {
            if (!wait(&sm.k_full[next_k % kStagesK], (next_k / kStagesK) & 1u)) return false;
            if (next_k < to && lane == 0) mbar_arrive(&sm.k_free[next_k % kStagesK]);
            __syncwarp();
        }
        return true;
    };
    auto see_v = [&](uint32_t to, bool own) {
        for (; next_v < to + own; ++next_v) {
            if (!wait(&sm.v_full[next_v % kStagesV], (next_v / kStagesV) & 1u)) return false;
            if (next_v < to && lane == 0) mbar_arrive(&sm.v_free[next_v % kStagesV]);
            __syncwarp();
        }
        return true;
    };
    while (ok) {
        const int slot = runs & 1;
        if (!(ok = wait(&sm.rd_full[slot], (runs >> 1) & 1u))) break;
        const RunDesc& rd = sm.rd[slot];
        const int32_t kind = same(rd.kind), j0 = same(rd.j0[lane_id]), p0 = same(rd.p0), steps_b = same(rd.steps[1]);
        const int32_t new_q = same(rd.new_q[lane_id]);
        const int32_t keys = min(same(rd.steps[lane_id]) * kStep, same(rd.len) - j0 * kStep), items = same(rd.items());
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.rd_free[slot]);
        ++runs;
        if (kind == 0) break;
        if (lane_id == 0 || kind > 1) {
            const int32_t H = (keys + kHalf - 1) / kHalf;
            auto scores = [&](int32_t h) {
                const uint32_t at = base + item_of(kind, lane_id, h >> 1, steps_b), st = at % kStagesK, buf = (halves + h) & 1u;
                if ((h & 1) == 0 && !see_k(at, true)) return false;
                ptx::tc_fence_after();
                const uint64_t kd = desc(smem_u32(&sm.k[st][(h & 1) * (kHalf * 128)]), 16, 1024);
                const uint32_t s = col_s + buf * kHalf;
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks) {
                    const uint32_t off = ((ks / 4) * kRegion + (ks % 4) * 32) / kUnit;
                    mma_ss_elected(s, qd + off, kd + off, idesc_s, ks > 0);
                }
                commit_elected(&sm.s_full[lane_id][buf]);
                if ((h & 1) || h + 1 == H) commit_elected(&sm.k_free[st]);
                if (h + 1 == H) commit_elected(&sm.q_free[lane_id]);
                return true;
            };
            if (new_q && !(ok = wait(&sm.q_full[lane_id], (fills++) & 1u))) break;
            if (!(ok = scores(0))) break;
            if (H > 1 && !(ok = scores(1))) break;
            for (int32_t h = 0; h < H; ++h) {
                const uint32_t hh = halves + h, buf = hh & 1u, at = base + item_of(kind, lane_id, h >> 1, steps_b), st = at % kStagesV;
                if ((h & 1) == 0 && (j0 + (h >> 1) + 1) * kStep > p0) {  // the step holds nodes: the softmax looks at its V
                    if (!(ok = see_v(at, true))) break;
                    if (lane == 0) mbar_arrive(&sm.v_seen[lane_id]);
                    __syncwarp();
                }
                if (!(ok = wait(&sm.p_full[lane_id][buf], (hh >> 1) & 1u))) break;
                if (next_v <= at && !(ok = see_v(at, true))) break;
                // a run's first product starts O afresh: the run before has been read
                if (h == 0 && mine > 0 && !(ok = wait(&sm.o_free[lane_id], (mine - 1) & 1u))) break;
                if (h + 1 == H) {  // (passes on what the softmax warps wrote before)
                    if (lane == 0) mbar_arrive(&sm.run_full[lane_id][mine & 1u]);
                    __syncwarp();
                }
                ptx::tc_fence_after();
                const uint64_t vd = desc(smem_u32(&sm.v[st][(h & 1) * (kHalf * DH * 2)]), BI_PAGE * 128, 1024);
                const uint32_t p = col_s + buf * kHalf;
                auto product = [&](int ks) {  // of 16 keys: the hi part, then the lo part
                    const uint64_t v = vd + ks * (DH / 64 * BI_PAGE * 128) / kUnit;
                    mma_ts_elected(col_o, p + 16 * ks, v, idesc_pv, ks > 0 || h > 0);
                    mma_ts_elected(col_o, p + 16 * ks + 8, v, idesc_pv, 1u);
                };
                const int ksteps = (min(kHalf, keys - h * kHalf) + 15) / 16;
                if (ksteps == kHalf / 16) {
#pragma unroll
                    for (int ks = 0; ks < kHalf / 16; ++ks) product(ks);
                } else {
                    for (int ks = 0; ks < ksteps; ++ks) product(ks);
                }
                // (the scores that follow in order tell that P V (h) is done, where there are any)
                if (h + 1 == H) commit_elected(&sm.o_done[lane_id]);
                else if (h + 2 == H) commit_elected(&sm.o_prev[lane_id]);
                if ((h & 1) || h + 1 == H) commit_elected(&sm.v_free[st]);
                if (h + 2 < H && !(ok = scores(h + 2))) break;
            }
            if (!ok) break;
            halves += H;
            ++mine;
        }
        base += items;
        // the other lane's rest, each K before its V, as they are copied; but the last, which the next run's wait will pass
        while (ok && next_v + 1 < base) ok = see_k(max(next_k, next_v + 1), false) && see_v(next_v + 1, false);
    }
    if (!ok) *abort = 1;
    // no product may be in flight when tensor memory is freed
    commit_elected(&sm.drain[lane_id]);
    volatile int32_t none = 0;
    ptx::mbar_wait_bounded(&sm.drain[lane_id], 0, &none);
}

__device__ __forceinline__ void tmem_ld_f32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld32(taddr, r);
    ptx::tmem_ld_wait();
    reg_fence<32>(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_f32(uint32_t taddr, const float (&v)[32]) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st32(taddr, r);
}

// ---------------------------------------------------------------------------
// The softmax warps: a warpgroup for each lane, one thread per row.  No barrier
// joins warps but mbarriers with bounded waits: a warp whose wait runs out sets
// abort and leaves, and the others follow.
// ---------------------------------------------------------------------------
template <int G, int DH>
__device__ __forceinline__ void consume(Smem<DH>& sm, uint32_t tmem, const TreeArgs& a, const Layout& lay) {
    constexpr int kStagesV = Smem<DH>::kStagesV;
    const int tid = threadIdx.x, lane = tid & 31, lane_id = tid / 128, lq = (tid / 32) & 3;
    const int row = tid & 127;  // = its tensor-memory lane
    const float c = __fmul_rn(a.scale, 1.44269504088896341f);
    volatile int32_t* abort = &sm.abort;
    const uint32_t col_o = lane_addr(tmem, kColO + lane_id * DH);
    // runs, the lane's own, its half steps, all items, phases of v_seen and o_prev
    uint32_t runs = 0, own = 0, halves = 0, base = 0, seen = 0, prevs = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort); };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    auto walk = [&] {  // every run; false: a wait ran out
        for (;; ++runs) {
            const int slot = runs & 1;
            if (!wait(&sm.rd_full[slot], (runs >> 1) & 1u)) return false;
            const RunDesc& rd = sm.rd[slot];
            const int32_t kind = rd.kind, items = rd.items();
            if (kind == 0) return true;
            if (lane_id == 1 && kind == 1) {
                arrive(&sm.rd_free[slot]);
                base += items;
                continue;
            }
            const int32_t p0 = rd.p0, first_key = rd.j0[lane_id] * kStep, rows = rd.rows[lane_id];
            const int32_t end = min(rd.len, first_key + rd.steps[lane_id] * kStep), H = (end - first_key + kHalf - 1) / kHalf;
            const bool mine = row < rows, active = 32 * lq < rows;  // (the latter uniform in the warp)
            const uint32_t* mask = mine ? a.mask + static_cast<int64_t>(rd.t0[lane_id] + row / G) * a.words : nullptr;
            int32_t looked = -1;            // step whose V has been waited for
            float L = 0.0f, M = -INFINITY;  // the sum so far and the reference that it is in
            for (int32_t h = 0; h < H; ++h) {
                const uint32_t hh = halves + h, buf = hh & 1u;
                const int32_t k0 = first_key + h * kHalf;
                const bool masked = k0 + kHalf > p0;  // there are nodes (or the end)
                uint32_t see[2];
                if (masked) {
                    see[0] = visible(mask, k0, p0, rd.n);
                    see[1] = visible(mask, k0 + 32, p0, rd.n);
                }
                if (!wait(&sm.s_full[lane_id][buf], (hh >> 1) & 1u)) return false;
                ptx::tc_fence_after();
                const uint32_t col_s = lane_addr(tmem, kColS + lane_id * kStep + buf * kHalf);
                if (active) {
                    uint32_t s[kHalf];
                    tmem_ld32(col_s, s);
                    tmem_ld32(col_s + 32, s + 32);
                    ptx::tmem_ld_wait();
                    reg_fence<kHalf>(s);
                    if (masked) {  // what the row does not attend: no score
#pragma unroll
                        for (int x = 0; x < kHalf; ++x) s[x] = see[x / 32] >> (x % 32) & 1u ? s[x] : 0xff800000u;
                    }
                    const float mx = __fmul_rn(max_of<kHalf>(s), c);
                    const bool up = h == 0 || mx > __fadd_rn(M, kSlack);
                    if (h > 0 && __any_sync(0xffffffffu, up)) {
                        // sum and O to the new references (by 1 in the warp's other rows)
                        const float al = up ? ex2(__fsub_rn(M, mx)) : 1.0f;
                        L = __fmul_rn(L, al);
                        // P V of the half step before is done: the next scores, issued after it, are, or its barrier says so
                        if (!(h + 1 < H ? wait(&sm.s_full[lane_id][buf ^ 1u], ((hh + 1) >> 1) & 1u)
                                        : wait(&sm.o_prev[lane_id], prevs & 1u)))
                            return false;
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int d0 = 0; d0 < DH; d0 += 32) {
                            float o[32];
                            tmem_ld_f32(col_o + d0, o);
#pragma unroll
                            for (int d = 0; d < 32; ++d) o[d] = __fmul_rn(o[d], al);
                            tmem_st_f32(col_o + d0, o);
                        }
                    }
                    M = up ? mx : M;
                    const float z = M == -INFINITY ? 0.0f : M;
                    const float2 c2 = make_float2(c, c), z2 = make_float2(-z, -z);
                    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int g = 0; g < kHalf; g += 16) {  // 16 keys: 8 packed pairs (of the hi, then of the lo parts)
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float2 e = fma2(make_float2(__uint_as_float(s[g + 2 * x]), __uint_as_float(s[g + 2 * x + 1])), c2, z2);
                            e.x = ex2(e.x);
                            e.y = ex2(e.y);
                            acc[x & 1] = add2(acc[x & 1], e);
                            pack_p(e.x, e.y, hi[x], lo[x]);
                        }
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            s[g + x] = hi[x];
                            s[g + 8 + x] = lo[x];
                        }
                    }
                    tmem_st32(col_s, s);
                    tmem_st32(col_s + 32, s + 32);
                    const float2 t = add2(acc[0], acc[1]);
                    L = __fadd_rn(L, __fadd_rn(t.x, t.y));
                }
                if (masked) {
                    // V of the request's nodes: values that are not finite are taken out (0 * NaN would reach every
                    // row), and rows past the last key up to the 16-key step are zeros.  Two lanes with the same V
                    // both do so: whichever finds a value notes it before the other can find it gone.
                    if (h >> 1 != looked) {
                        if (!wait(&sm.v_seen[lane_id], seen & 1u)) return false;
                        ++seen;
                        looked = h >> 1;
                    }
                    uint8_t* v = sm.v[(base + item_of(kind, lane_id, h >> 1, rd.steps[1])) % kStagesV] + (h & 1) * (kHalf * DH * 2);
                    auto place = [&](int32_t k, int32_t ch) {
                        return reinterpret_cast<uint4*>(v + ((k / BI_PAGE) * (DH / 64) + ch / 8) * (BI_PAGE * 128) +
                                                        sw128(k % BI_PAGE, ch % 8));
                    };
                    const int32_t keys = min(kHalf, end - k0), lo = max(p0 - k0, 0), chunks = (keys - lo) * (DH / 8);
                    for (int32_t x = keys * (DH / 8) + row; x < ((keys + 15) & ~15) * (DH / 8); x += kRows)
                        *place(x / (DH / 8), x % (DH / 8)) = make_uint4(0u, 0u, 0u, 0u);
                    // 0 * x is NaN where x is not finite
                    __nv_bfloat162 odd = __floats2bfloat162_rn(0.0f, 0.0f);
                    const __nv_bfloat162 zero = odd;
#pragma unroll 4
                    for (int32_t x = row; x < chunks; x += kRows) {
                        const uint4 d = *place(lo + x / (DH / 8), x % (DH / 8));
                        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[y]), zero, odd);
                    }
                    if (__hisnan(odd.x) || __hisnan(odd.y)) {
                        for (int32_t x = row; x < chunks; x += kRows) {
                            const int32_t k = lo + x / (DH / 8), node = k0 + k - p0;
                            uint4* at = place(k, x % (DH / 8));
                            const uint4 d = *at;
                            uint32_t w[4] = {d.x, d.y, d.z, d.w};
                            bool bad = false;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                if ((w[y] & 0x7f80u) == 0x7f80u) {
                                    w[y] &= 0xffff0000u;
                                    bad = true;
                                }
                                if ((w[y] & 0x7f800000u) == 0x7f800000u) {
                                    w[y] &= 0xffffu;
                                    bad = true;
                                }
                            }
                            if (bad) {
                                atomicOr(&sm.bad[slot][node >> 5], 1u << (node & 31));
                                __threadfence_block();
                                *at = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                tmem_st_wait();
                ptx::tc_fence_before();
                arrive(&sm.p_full[lane_id][buf]);
            }

            // ---- the run's reference, sum and O into the workspace ----
            if (H > 1 && !wait(&sm.o_prev[lane_id], (prevs++) & 1u)) return false;
            if (!wait(&sm.o_done[lane_id], own & 1u)) return false;
            if (!wait(&sm.run_full[lane_id][own & 1u], (own >> 1) & 1u)) return false;  // sm.bad
            ptx::tc_fence_after();
            if (mine) lay.ml[rd.part[lane_id] * lay.rows + row] = make_float2(M, L);
            if (!active) arrive(&sm.o_free[lane_id]);
#pragma unroll 1
            for (int d0 = 0; active && d0 < DH; d0 += 64) {
                uint32_t O[64];
                tmem_ld32(col_o + d0, O);
                tmem_ld32(col_o + d0 + 32, O + 32);
                ptx::tmem_ld_wait();
                reg_fence<64>(O);
                if (d0 + 64 == DH) {  // the next run's products may start O afresh
                    ptx::tc_fence_before();
                    arrive(&sm.o_free[lane_id]);
                }
                if (mine) {
                    // Nodes whose V is not finite were taken out of the product: the rows that attend them get it back.
                    for (int32_t w = 0; 32 * w < rd.n && p0 + 32 * w < end; ++w) {
                        uint32_t bad = *const_cast<volatile uint32_t*>(&sm.bad[slot][w]);
                        if (bad == 0u) continue;
                        for (bad &= mask[w]; bad != 0u; bad &= bad - 1u) {
                            const int32_t k = p0 + 32 * w + __ffs(bad) - 1;
                            if (k < first_key || k >= end) continue;
                            const int32_t pg = a.page_table[static_cast<int64_t>(rd.r) * a.max_pages + k / BI_PAGE];
                            if (pg < 0 || pg >= a.num_pages) continue;
                            const bi_bf16* v = a.vc + ((static_cast<int64_t>(pg) * a.Hkv + rd.g) * BI_PAGE + (k & (BI_PAGE - 1))) * DH + d0;
#pragma unroll
                            for (int d = 0; d < 64; ++d) {
                                const float x = bf16_to_f32(v[d]);
                                if (!(fabsf(x) <= 3.4e38f)) O[d] = __float_as_uint(__uint_as_float(O[d]) + x);
                            }
                        }
                    }
                    float4* dst = lay.o + (rd.part[lane_id] * (DH / 4) + d0 / 4) * lay.rows + row;
#pragma unroll
                    for (int d = 0; d < 64; d += 4)
                        dst[static_cast<int64_t>(d / 4) * lay.rows] = make_float4(__uint_as_float(O[d]), __uint_as_float(O[d + 1]),
                                                                                  __uint_as_float(O[d + 2]), __uint_as_float(O[d + 3]));
                }
                __syncwarp();
            }
            arrive(&sm.rd_free[slot]);
            base += items;
            halves += H;
            ++own;
        }
    };
    if (!walk()) {
        tmem_st_wait();  // (tensor memory is freed next)
        if (lane == 0) report(a.status, BI_DEV_TIMEOUT_ATTENTION);
        *abort = 1;  // the other roles' waits give up at once
    }
}

// kTest: bi_tree_attention_wait_test's form (the tests cost the other 1 to 2 %)
template <int G, int DH, bool kTest>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, TreeArgs a, Layout lay) {
    pdl_trigger();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem<DH>& sm = *reinterpret_cast<Smem<DH>*>(smem_raw);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid & 31;
    if (tid == 0) {
        sm.abort = 0;
        ptx::prefetch_tmap(&tmK);
        ptx::prefetch_tmap(&tmV);
        ptx::prefetch_tmap(&tmQ);
        for (int s = 0; s < Smem<DH>::kStagesK; ++s) {
            sm.k_issued[0][s] = sm.k_issued[1][s] = 0;
            ptx::mbar_init(&sm.k_full[s], 2);  // the copying warps
            ptx::mbar_init(&sm.k_free[s], 2);  // the lanes
        }
        for (int s = 0; s < Smem<DH>::kStagesV; ++s) {
            sm.v_issued[0][s] = sm.v_issued[1][s] = 0;
            ptx::mbar_init(&sm.v_full[s], 2);
            ptx::mbar_init(&sm.v_free[s], 2);
        }
        for (int i = 0; i < 2; ++i) {
            sm.q_issued[i] = 0;
            ptx::mbar_init(&sm.q_full[i], 1);
            ptx::mbar_init(&sm.q_free[i], 1);
            ptx::mbar_init(&sm.v_seen[i], 1);
            ptx::mbar_init(&sm.o_prev[i], 1);
            ptx::mbar_init(&sm.o_done[i], 1);
            ptx::mbar_init(&sm.o_free[i], 4);  // the warps of a warpgroup
            ptx::mbar_init(&sm.drain[i], 1);
            ptx::mbar_init(&sm.rd_full[i], 1);
            ptx::mbar_init(&sm.rd_free[i], kSoftWarps + 2);  // the softmax and the issuing warps
            for (int j = 0; j < 2; ++j) {
                ptx::mbar_init(&sm.s_full[i][j], 1);
                ptx::mbar_init(&sm.p_full[i][j], 4);
                ptx::mbar_init(&sm.run_full[i][j], 1);
            }
        }
        ptx::fence_barrier_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc<1>(&sm.tmem_base, kTmemCols);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_wait();
    const uint32_t tmem = sm.tmem_base;
    if (warp >= kSoftWarps) {
        if (warp == kSoftWarps) produce<G, DH, true, kTest>(sm, &tmK, &tmV, &tmQ, a, lay.slots);
        else if (warp == kSoftWarps + 2) produce<G, DH, false, kTest>(sm, &tmK, &tmV, nullptr, a, lay.slots);
        else issue_products<DH, kTest>(sm, tmem, warp == kSoftWarps + 1 ? 0 : 1, a.wait_ns);
    } else {
        consume<G, DH>(sm, tmem, a, lay);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) {
        ptx::tmem_dealloc<1>(tmem, kTmemCols);
        if (sm.abort && lane == 0) {
            // Every copy issued has landed before the shared memory is released (the issuing warps, had they not
            // stopped, would have waited for each).  A stage is filled anew only once both copying warps have
            // armed it and its fill was seen, so their counts differ by one at most: there the arrival of the warp
            // that stopped is made up for, so that the phase ends with the other's copies.
            volatile int32_t none = 0;
            auto landed = [&](uint64_t* full, uint32_t first, uint32_t second) {
                const uint32_t fills = max(first, second);
                if (first != second) mbar_arrive(full);
                if (fills > 0) ptx::mbar_wait_bounded(full, (fills - 1) & 1u, &none);
            };
            for (int st = 0; st < Smem<DH>::kStagesK; ++st) landed(&sm.k_full[st], sm.k_issued[0][st], sm.k_issued[1][st]);
            for (int st = 0; st < Smem<DH>::kStagesV; ++st) landed(&sm.v_full[st], sm.v_issued[0][st], sm.v_issued[1][st]);
            for (int st = 0; st < 2; ++st)
                if (sm.q_issued[st]) ptx::mbar_wait_bounded(&sm.q_full[st], (sm.q_issued[st] - 1) & 1u, &none);
        }
    }
}

// Folds the segments of each row in ascending order.  A block has 32 rows of a
// tile and all dims, or, kFew, 32 dims: a thread folds groups of four dims of a
// row (the warp's rows side by side), the partials of several segments in
// flight, then the block writes them out.  Also writes the zeros of requests
// without a valid context.
constexpr int kMergeRows = 32, kMergeWarps = 8, kMergeDims = 4 * kMergeWarps;

template <int G, int DH, bool kFew>
__global__ void __launch_bounds__(32 * kMergeWarps)
tree_merge_kernel(TreeArgs a, Layout lay) {
    pdl_trigger();
    pdl_wait();
    constexpr int NT = kRows / G, kGroups = kFew ? 1 : DH / kMergeDims, kBatch = kFew ? 8 : 2, kDims = kGroups * kMergeDims;
    __shared__ float out[kMergeRows][kDims + 4];
    const int32_t id = blockIdx.x, g = blockIdx.y;
    const int32_t r0 = blockIdx.z / (DH / kDims) * kMergeRows, d0 = blockIdx.z % (DH / kDims) * kDims;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    // last request whose first tile is <= id: 32 candidates at a time (one load's latency each, not one per halving)
    int lo = 0;
    for (int span = a.B; span > 1;) {
        const int step = (span + 31) / 32, r = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, r < lo + span && tile_id(r, a.cu_q[r], 0, NT) <= id);
        const int k = at == 0u ? 0 : 31 - __clz(at);  // ascending
        span = min(step, span - k * step);
        lo += k * step;
    }
    const int32_t c0 = a.cu_q[lo], c1 = a.cu_q[lo + 1], n = c1 - c0, p0 = a.pos0[lo];
    if (c0 < 0 || c1 < c0 || c1 > a.T) return;
    const int64_t tl = id - tile_id(lo, c0, 0, NT);
    if (tl < 0 || tl * NT >= n) return;
    const int32_t t0 = c0 + static_cast<int32_t>(tl) * NT, rows = min(NT, c1 - t0) * G;
    if (r0 >= rows) return;
    const bool valid = p0 >= 0 && n <= a.max_nodes && static_cast<int64_t>(p0) + n <= a.max_seq;
    const int row = r0 + lane;
    const bool mine = valid && row < rows;
    const int32_t steps = (p0 + n + kStep - 1) / kStep, ss = segment_steps(steps, (n + NT - 1) / NT * a.Hkv);
    const int32_t nseg = (steps + ss - 1) / ss;
    const int64_t part = (static_cast<int64_t>(id) * a.Hkv + g) * lay.slots;
    float m = 0.0f, l = 0.0f, o[kGroups][4] = {};
    for (int32_t s0 = 0; mine && s0 < nseg; s0 += kBatch) {
        float2 pm[kBatch];
        float4 po[kBatch][kGroups];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (s0 + u >= nseg) break;
            pm[u] = lay.ml[(part + s0 + u) * lay.rows + row];
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                po[u][q] = lay.o[((part + s0 + u) * (DH / 4) + d0 / 4 + q * kMergeWarps + warp) * lay.rows + row];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (s0 + u >= nseg) break;
            const bool first = s0 + u == 0;
            const Fold f = first ? Fold{pm[u].x, 0.0f, 1.0f} : fold_scales(m, pm[u].x);
            m = f.m;
            l = first ? pm[u].y : fold_value(f, l, pm[u].y);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const float p[4] = {po[u][q].x, po[u][q].y, po[u][q].z, po[u][q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) o[q][e] = first ? p[e] : fold_value(f, o[q][e], p[e]);
            }
        }
    }
    const float fac = out_factor(l);
#pragma unroll
    for (int q = 0; q < kGroups; ++q)
        *reinterpret_cast<float4*>(&out[lane][4 * (q * kMergeWarps + warp)]) =
            make_float4(__fmul_rn(o[q][0], fac), __fmul_rn(o[q][1], fac), __fmul_rn(o[q][2], fac), __fmul_rn(o[q][3], fac));
    __syncthreads();
    // (a request with too many nodes has tiles of more rows than the grid was sized for)
    const int last = valid || r0 + kMergeRows < lay.rows ? min(rows, r0 + kMergeRows) : rows;
    for (int i = threadIdx.x; i < (last - r0) * (kDims / 8); i += 32 * kMergeWarps) {
        const int rr = i / (kDims / 8), d = i % (kDims / 8) * 8, w = r0 + rr;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
        if (valid) {
            x = *reinterpret_cast<const float4*>(&out[rr][d]);
            y = *reinterpret_cast<const float4*>(&out[rr][d + 4]);
        }
        const int64_t at = ((static_cast<int64_t>(t0) + w / G) * a.H + static_cast<int64_t>(g) * G + w % G) * DH + d0 + d;
        if (a.out_f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
            dst[0] = x;
            dst[1] = y;
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        }
    }
}

// Tiles a launch may count (tile_id's bound), and a tile's rows (whole warps of the merge).
static int64_t launch_tiles(int32_t B, int32_t T, int32_t G) { return static_cast<int64_t>(T) / (kRows / G) + B; }
static int32_t launch_rows(int32_t max_nodes, int32_t G) {
    const int32_t n = max_nodes * G < kRows ? max_nodes * G : kRows;
    return (n + kMergeRows - 1) / kMergeRows * kMergeRows;
}
static size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
static int32_t launch_slots(int32_t max_seq, int32_t Hkv) { return most_segments((max_seq - 1) / kStep + 1, Hkv); }

template <int G, int DH, bool kTest>
cudaError_t launch_kernel(const TreeArgs& a, const Layout& lay, unsigned ctas, const CUtensorMap& tmK,
                          const CUtensorMap& tmV, const CUtensorMap& tmQ, cudaStream_t s) {
    const size_t smem = sizeof(Smem<DH>);
    static_assert(sizeof(Smem<DH>) <= 232448, "shared memory of a block");
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [smem] {
        attr_err = cudaFuncSetAttribute(tree_attention_kernel<G, DH, kTest>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(smem));
    });
    if (attr_err != cudaSuccess) return attr_err;
    return launch_pdl(tree_attention_kernel<G, DH, kTest>, dim3(ctas), dim3(kThreads), smem, s, tmK, tmV, tmQ, a, lay);
}

template <int G, int DH>
cudaError_t launch(const TreeArgs& a, void* ws, cudaStream_t s) {
    const int32_t slots = launch_slots(a.max_seq, a.Hkv);
    const int64_t tiles = launch_tiles(a.B, a.T, G) * a.Hkv;
    const unsigned ctas = static_cast<unsigned>(tiles * slots < num_sms() ? tiles * slots : num_sms());
    CUtensorMap tmK, tmV, tmQ;
    if (!encode_kv_map(&tmK, a.kc, a.num_pages, a.Hkv, DH) || !encode_v_map(&tmV, a.vc, a.num_pages, a.Hkv, DH) ||
        !encode_q_map(&tmQ, a.q, a.T, a.H, DH, G))
        return cudaErrorInvalidValue;
    Layout lay{nullptr, nullptr, slots, launch_rows(a.max_nodes, G)};
    char* w = reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(ws)));
    lay.ml = reinterpret_cast<float2*>(w);
    lay.o = reinterpret_cast<float4*>(w + align_up(static_cast<size_t>(tiles) * slots * lay.rows * sizeof(float2)));
    const cudaError_t e = a.wait_ns == kWaitLimitNs && a.skip_copy < 0 ? launch_kernel<G, DH, false>(a, lay, ctas, tmK, tmV, tmQ, s)
                                                                       : launch_kernel<G, DH, true>(a, lay, ctas, tmK, tmV, tmQ, s);
    if (e != cudaSuccess) return e;
    // one block for all dims of its rows, or, while that leaves SMs without one, a block for each 32
    const bool few = tiles * (lay.rows / kMergeRows) < 4 * num_sms();
    const dim3 grid(static_cast<unsigned>(launch_tiles(a.B, a.T, G)), a.Hkv, lay.rows / kMergeRows * (few ? DH / kMergeDims : 1));
    return launch_pdl(few ? tree_merge_kernel<G, DH, true> : tree_merge_kernel<G, DH, false>, grid, dim3(32 * kMergeWarps), 0, s, a, lay);
}

}  // namespace tree

int32_t tree_segment(int32_t positions, int32_t nodes, int32_t H, int32_t Hkv) {
    const int32_t NT = tree::kRows / (H / Hkv), steps = (positions + tree::kStep - 1) / tree::kStep;
    return tree::segment_steps(steps, (nodes + NT - 1) / NT * Hkv) * tree::kStep;
}

size_t tree_ws_bytes(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t Dh, int32_t max_nodes, int32_t max_seq) {
    using namespace tree;
    const size_t parts = static_cast<size_t>(launch_tiles(B, T, H / Hkv)) * Hkv * launch_slots(max_seq, Hkv) *
                         launch_rows(max_nodes, H / Hkv);
    return 256 + align_up(parts * sizeof(float2)) + parts * Dh * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeArgs& a, void* ws, cudaStream_t s) {
    if (a.B <= 0 || a.T <= 0) return cudaSuccess;
    const int32_t G = a.H / a.Hkv;
    if (a.Dh == 128) {
        if (G == 1) return tree::launch<1, 128>(a, ws, s);
        if (G == 2) return tree::launch<2, 128>(a, ws, s);
        if (G == 4) return tree::launch<4, 128>(a, ws, s);
        if (G == 8) return tree::launch<8, 128>(a, ws, s);
    } else if (a.Dh == 64) {
        if (G == 1) return tree::launch<1, 64>(a, ws, s);
        if (G == 2) return tree::launch<2, 64>(a, ws, s);
        if (G == 4) return tree::launch<4, 64>(a, ws, s);
        if (G == 8) return tree::launch<8, 64>(a, ws, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace bi
