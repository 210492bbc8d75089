// Beam search: log-probabilities of logits rows and the best continuations of
// a group of beams (arithmetic specification, section 17), and the block
// tables of the beams that were chosen.
//
// A row's continuation i scores score + l_i - lse(l), lse = M + ln sum exp(l_i
// - M) in Q16 with M the row's maximum. The exponentials are rounded against M,
// so the maximum is settled over the whole row first; within a row the order
// is that of the logits, so a row's best n need no lse.
//
// One thread-block cluster per row, its values in registers between the
// passes: one read of the logits. Pass 1 takes maxima; the cluster's warps are
// put into at least n groups, and the smallest of the groups' maxima is a
// bound that n values or more reach and few more do (about g ln g of g
// groups, whatever the row's distribution, as every group samples the whole
// row). Pass 2 sums the exponentials and hands what reaches the bound to the
// cluster's first CTA, which ranks it by counting. Values carry their index
// as the low half of a 64-bit key, so that equal logits do not all pass.
#pragma once
#include "kernels.h"
#include "ptx.cuh"
#include "cluster.cuh"
#include "int_device.cuh"

namespace detint {

constexpr int BM_THREADS = 512, BM_WARPS = BM_THREADS / 32;
constexpr int BM_MAX_CL = 16;            // CTAs of a row
constexpr int BM_CAP = 1024;             // values over the bound that are ranked by counting
constexpr int BM_MAX_OUT = 64;           // continuations of a group; beams
constexpr int BM_MASKED = -2147483647 - 1;

struct BeamArgs {
    const int32_t* logits;
    size_t stride;                       // elements between rows
    const long long* scores;             // [rows]
    const int32_t* done;                 // [rows] or null
    int rows, n, n_out, end_id, beams;
    int lg_cl;                           // log2 of the CTAs of a row
    int lg_groups, per_warp;             // log2 of the groups of warps; values of a warp that count for the bound
    long long* ws_score;                       // [rows][n_out], best first
    int32_t* ws_tok;                     // [rows][n_out], -1 behind the last
    int32_t *parent, *token, *done_out;  // [groups][n_out]
    long long* score_out;
};

// a value and its index as one key: larger values, then smaller indexes, are
// larger (0 is no value's key, and neither are all ones)
__device__ __forceinline__ u64 bm_key(int v, int idx) { return ((u64)((unsigned)v ^ 0x80000000u) << 32) | (unsigned)(0x7fffffff - idx); }
__device__ __forceinline__ int bm_value(u64 key) { return (int)((unsigned)(key >> 32) ^ 0x80000000u); }
__device__ __forceinline__ int bm_index(u64 key) { return 0x7fffffff - (int)(unsigned)key; }
__device__ __forceinline__ u64 umax64(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 umin64(u64 a, u64 b) { return a < b ? a : b; }

// exp(l - M) in Q30 of Q16 logits l <= M: delta in Q10 octaves, exp2q's cubic on
// its fraction; zero from 31 octaves down, where the difference is clamped
__device__ __forceinline__ unsigned bm_exp(int l, int M) {
    const int d = -(int)min((unsigned)M - (unsigned)l, 1u << 22);
    const int delta = (int)(((i64)d * 47274 + (1 << 20)) >> 21);
    const int f = delta & 1023;
    const int v1 = (2562 * f + (512 + (7419 << 10))) >> 10;
    const int v2 = (f * v1 + (512 + (22787 << 10))) >> 10;
    const unsigned p = (unsigned)((f * v2 + (512 + (32768 << 10))) >> 10) << 15;
    const int sh = -(delta >> 10);
    return sh >= 31 ? 0u : (p + ((1u << sh) >> 1)) >> sh;
}
// ln(S / 2^30) in Q16, S >= 2^30: log2 to 20 bits below the point, a bit per
// squaring of the 32-bit mantissa, times ln 2
__device__ __forceinline__ i64 bm_ln(u64 S) {
    const int b = bitlen_u64(S);
    u64 y = b <= 32 ? S << (32 - b) : S >> (b - 32);
    i64 lg = b - 31;
    for (int i = 0; i < 20; ++i) {
        const u64 z = y * y;
        const int bit = (int)(z >> 63);
        y = z >> (31 + bit);
        lg = 2 * lg + bit;
    }
    return rshr(lg * 726817, 24);
}

// four consecutive logits of a row (VEC: one aligned load), masked ones past the end
template <bool VEC>
__device__ __forceinline__ int4 bm_load(const int32_t* row, int at, int n) {
    int4 v = make_int4(BM_MASKED, BM_MASKED, BM_MASKED, BM_MASKED);
    if (VEC && at + 4 <= n) return __ldg((const int4*)(row + at));
    if (at < n) v.x = __ldg(row + at);
    if (at + 1 < n) v.y = __ldg(row + at + 1);
    if (at + 2 < n) v.z = __ldg(row + at + 2);
    if (at + 3 < n) v.w = __ldg(row + at + 3);
    return v;
}

// Q quads of a row per thread and round. HELD: one round, kept in registers
// for the second pass; otherwise rounds over the row, read again by it.
template <int Q, bool HELD, bool VEC>
__global__ void __launch_bounds__(BM_THREADS) k_beam_rows(BeamArgs a) {
    constexpr int NL = BM_MAX_CL * BM_WARPS / 32;        // warps of a cluster per lane
    __shared__ u64 wkey[BM_WARPS], wsum[BM_WARPS], cand[BM_CAP], sums[BM_MAX_CL], best, tau_s;
    __shared__ int wtop[BM_WARPS], max_s;
    __shared__ i64 base_s;
    __shared__ unsigned count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CL = (int)cl_size(), rank = (int)cl_rank(), r = (int)(blockIdx.x >> a.lg_cl);
    pdl_launch();
    long long* const ws_score = a.ws_score + (size_t)r * a.n_out;
    int32_t* const ws_tok = a.ws_tok + (size_t)r * a.n_out;
    const i64 score = min((i64)a.scores[r], 1ll << 62);
    const bool dead = score < -(1ll << 62);
    if (dead || (a.done && a.done[r])) {                 // (the whole cluster takes this way out)
        if (rank == 0)
            for (int i = tid; i < a.n_out; i += BM_THREADS) {
                ws_tok[i] = i == 0 && !dead ? a.end_id : -1;
                ws_score[i] = score;
            }
        return;
    }
    const int32_t* row = a.logits + (size_t)r * a.stride;
    const int step = CL * BM_THREADS * 4, first = (rank * BM_THREADS + tid) * 4;
    int4 x[Q];
    auto load = [&](int base) {
#pragma unroll
        for (int q = 0; q < Q; ++q) x[q] = bm_load<VEC>(row, base + q * step, a.n);
    };
    auto each = [&](int base, auto f) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            f(x[q].x, base + q * step);
            f(x[q].y, base + q * step + 1);
            f(x[q].z, base + q * step + 2);
            f(x[q].w, base + q * step + 3);
        }
    };
    // ---- pass 1: this thread's largest value, the first of equal ones
    int top = BM_MASKED, at = 0;
    for (int base = first; base < a.n; base += Q * step) {
        load(base);
        each(base, [&](int v, int i) {
            if (v > top) { top = v; at = i; }
        });
        if (HELD) break;
    }
    {
        u64 k = top == BM_MASKED ? 0 : bm_key(top, at), wk = redux_max_u64(k);
        if (lane == 0) wtop[warp] = wk ? bm_value(wk) : BM_MASKED;
        for (int i = 1; i < a.per_warp; ++i) {           // the per_warp-th largest of the warp's
            if (k == wk) k = 0;
            wk = redux_max_u64(k);
        }
        if (lane == 0) wkey[warp] = wk;
        if (tid == 0) count = 0;
    }
    cl_sync();
    // ---- the row's maximum, and the bound: entry e (a warp) is in group e mod 2^lg_groups
    if (warp == 0) {
        const int NE = CL * BM_WARPS, NG = 1 << a.lg_groups;
        u64 g[NL], tau = ~0ull;
        int m = BM_MASKED;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int e = lane + 32 * j;
            g[j] = 0;
            if (e < NE) {
                g[j] = (u64)cl_ld64((const i64*)&wkey[e & (BM_WARPS - 1)], e / BM_WARPS);
                m = max(m, cl_ld32(&wtop[e & (BM_WARPS - 1)], e / BM_WARPS));
            }
        }
#pragma unroll
        for (int h = NL / 2; h; h >>= 1)
            if (32 * h >= NG)
#pragma unroll
                for (int j = 0; j < h; ++j) g[j] = umax64(g[j], g[j + h]);
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (j == 0 || 32 * j < NG) tau = umin64(tau, g[j]);
        for (int o = 16; o >= NG; o >>= 1) tau = umax64(tau, __shfl_xor_sync(0xffffffffu, tau, o));
        for (int o = 16; o; o >>= 1) tau = umin64(tau, __shfl_xor_sync(0xffffffffu, tau, o));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) {
            tau_s = umax64(tau, 1);                      // (a masked value has no key)
            max_s = m;
        }
    }
    __syncthreads();
    const int M = max_s;
    const u64 tau = tau_s;
    const int tau_v = tau > 1 ? bm_value(tau) : BM_MASKED + 1;
    // ---- pass 2: the sum, and what reaches the bound (nothing of a row without candidates)
    u64 sum = 0;
    for (int base = first; base < a.n; base += Q * step) {
        if (!HELD) load(base);
        each(base, [&](int v, int i) {
            if (v != BM_MASKED) sum += bm_exp(v, M);
            if (v >= tau_v) {
                const u64 k = bm_key(v, i);
                if (k >= tau) {
                    const unsigned to = cl_add32(&count, 0, 1);
                    if (to < BM_CAP) cl_st64(&cand[to], 0, k);
                }
            }
        });
        if (HELD) break;
    }
    sum = redux_sum_u64(sum);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        u64 t = 0;
        for (int w = 0; w < BM_WARPS; ++w) t += wsum[w];
        cl_st64(&sums[rank], 0, t);
    }
    cl_sync();
    const unsigned c = cl_ld32u(&count, 0);
    if (c > BM_CAP) {                                    // too many: n_out times the best one below the last
        u64 last = ~0ull;
        for (int i = 0; i < a.n_out; ++i) {
            u64 k = 0;
            for (int base = first; base < a.n; base += Q * step) {
                if (!HELD) load(base);
                each(base, [&](int v, int j) {
                    const u64 y = v == BM_MASKED ? 0 : bm_key(v, j);
                    if (y < last) k = umax64(k, y);
                });
                if (HELD) break;
            }
            k = redux_max_u64(k);
            if (lane == 0) wkey[warp] = k;
            __syncthreads();
            if (tid == 0) {
                u64 t = 0;
                for (int w = 0; w < BM_WARPS; ++w) t = umax64(t, wkey[w]);
                best = t;
            }
            cl_sync();
            k = 0;
            for (int q = 0; q < CL; ++q) k = umax64(k, (u64)cl_ld64((const i64*)&best, q));
            cl_sync();
            last = k;
            if (rank == 0 && tid == 0) cand[i] = k;
        }
    }
    if (rank == 0) {
        if (tid == BM_THREADS - 1) {
            u64 t = 0;
            for (int q = 0; q < CL; ++q) t += sums[q];
            base_s = t ? score - M - bm_ln(t) : 0;
        }
        __syncthreads();
        const int m = c > BM_CAP ? a.n_out : (int)c;
        for (int i = tid; i < m; i += BM_THREADS) {
            const u64 k = cand[i];
            int better = 0;
            for (int j = 0; j < m; ++j) better += cand[j] > k;
            if (better < a.n_out) {
                ws_tok[better] = bm_index(k);
                ws_score[better] = base_s + bm_value(k);
            }
        }
        for (int i = m + tid; i < a.n_out; i += BM_THREADS) {
            ws_tok[i] = -1;
            ws_score[i] = 0;
        }
    }
    cl_sync();                                           // no CTA leaves while another reads its shared memory
}

// The best n_out of a group: a candidate's place is the number of better ones,
// found in every other beam's sorted list by halving.
constexpr int BM_MERGE_THREADS = 256;
__global__ void __launch_bounds__(BM_MERGE_THREADS) k_beam_merge(BeamArgs a) {
    extern __shared__ __align__(16) unsigned char bm_raw[];
    __shared__ int len[BM_MAX_OUT], ended[BM_MAX_OUT];
    const int W = a.beams, n = a.n_out, tid = threadIdx.x, r0 = (int)blockIdx.x * W;
    i64* sc = (i64*)bm_raw;                              // [W][n]
    if (tid < W) ended[tid] = a.done && a.done[r0 + tid];
    pdl_wait();
    const long long* ws = a.ws_score + (size_t)r0 * n;
    const int32_t* wt = a.ws_tok + (size_t)r0 * n;
    for (int i = tid; i < W * n; i += BM_MERGE_THREADS) sc[i] = __ldcg(ws + i);
    if (tid < W) {
        int lo = 0, hi = n;                              // entries of the beam: the tokens before the first -1
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldcg(wt + tid * n + mid) >= 0) lo = mid + 1;
            else hi = mid;
        }
        len[tid] = lo;
    }
    __syncthreads();
    const size_t out = (size_t)blockIdx.x * n;
    int total = 0;
    for (int q = 0; q < W; ++q) total += len[q];
    for (int i = tid; i < n; i += BM_MERGE_THREADS)
        if (i >= total) {
            a.parent[out + i] = a.token[out + i] = -1;
            a.score_out[out + i] = (long long)(1ull << 63);
            a.done_out[out + i] = 0;
        }
    // (a thread per beam and place, the places side by side)
    for (int b = 0; b < W; ++b)
        for (int i = tid; i < len[b]; i += BM_MERGE_THREADS) {
            const i64 s = sc[b * n + i];
            int place = i;
            for (int q = 0; q < W && place < n; ++q) {
                if (q == b) continue;
                // a lower beam goes before at an equal score
                int lo = 0, hi = len[q];
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    const i64 o = sc[q * n + mid];
                    if (o > s || (o == s && q < b)) lo = mid + 1;
                    else hi = mid;
                }
                place += lo;
            }
            if (place < n) {
                const int tok = __ldcg(wt + b * n + i);
                a.parent[out + place] = b;
                a.token[out + place] = tok;
                a.score_out[out + place] = s;
                a.done_out[out + place] = ended[b] || tok == a.end_id;
            }
        }
}

// ---- the chosen beams' block tables. Whole pages are shared. Of the page that
// is still being filled (column len / 64) a beam's first child becomes the
// owner; every other child takes the page of a beam without children, into
// which its parent's is to be copied (src, dst: -1 where nothing is). So a
// group's beams keep as many growing pages as they had, nothing is allocated,
// and no page that is copied to is copied from. A column's entries are read by
// one CTA before it writes them: out may be the table itself.
constexpr int BR_COLS = 64, BR_THREADS = 256;
__global__ void __launch_bounds__(BR_THREADS) k_beam_reorder(const int32_t* table, int32_t* out, const int32_t* parent,
                                                            const int32_t* lens, int W, int max_blocks, int32_t* src,
                                                            int32_t* dst) {
    __shared__ int32_t old[BM_MAX_OUT][BR_COLS];
    __shared__ int par[BM_MAX_OUT], first[BM_MAX_OUT], used[BM_MAX_OUT], spare[BM_MAX_OUT];
    const int tid = threadIdx.x, c0 = (int)blockIdx.x * BR_COLS, r0 = (int)blockIdx.y * W;
    const int len = max(lens[blockIdx.y], 0), full = len >> 6;
    const bool grows = (len & 63) && full < max_blocks, here = grows && full >= c0 && full < c0 + BR_COLS;
    if (blockIdx.x == 0 && !grows)
        for (int b = tid; b < W; b += BR_THREADS) src[r0 + b] = dst[r0 + b] = -1;
    if (c0 > full && table == out) return;               // columns of pages to come stay
    for (int b = tid; b < W; b += BR_THREADS) {
        const int p = parent[r0 + b];
        par[b] = p >= 0 && p < W ? p : -1;
    }
    for (int i = tid; i < W * BR_COLS; i += BR_THREADS) {
        const int b = i / BR_COLS, c = c0 + (i & (BR_COLS - 1));
        old[b][c - c0] = c < max_blocks ? table[(size_t)(r0 + b) * max_blocks + c] : -1;
    }
    __syncthreads();
    if (here) {
        for (int b = tid; b < W; b += BR_THREADS) {
            bool f = par[b] >= 0, any = false;
            for (int q = 0; q < W; ++q) {
                f = f && (q >= b || par[q] != par[b]);
                any = any || par[q] == b;
            }
            first[b] = f;
            used[b] = any;
        }
        __syncthreads();
        for (int b = tid; b < W; b += BR_THREADS) {
            int n = 0;                                   // beams before b that have no child
            for (int u = 0; u < b; ++u) n += !used[u];
            if (!used[b]) spare[n] = b;
        }
    }
    __syncthreads();
    for (int i = tid; i < W * BR_COLS; i += BR_THREADS) {
        const int b = i / BR_COLS, c = c0 + (i & (BR_COLS - 1));
        if (c >= max_blocks) continue;
        int32_t v = old[c < full && par[b] >= 0 ? par[b] : b][c - c0];
        if (here && c == full) {
            int32_t s = -1, d = -1;
            if (first[b]) {
                v = old[par[b]][c - c0];
            } else {
                int n = 0;                               // beams before b that take a spare page
                for (int q = 0; q < b; ++q) n += !first[q];
                v = old[spare[n]][c - c0];
                if (par[b] >= 0) { s = old[par[b]][c - c0]; d = v; }
            }
            src[r0 + b] = s;
            dst[r0 + b] = d;
        }
        out[(size_t)(r0 + b) * max_blocks + c] = v;
    }
}

}  // namespace detint
