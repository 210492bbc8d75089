// Beam search: log-probabilities of logits rows and the best continuations of
// a group of beams (arithmetic specification, section 17), and the block
// tables of the beams that were chosen.
//
// A row's continuation i scores score + l_i - lse(l), lse = M + ln sum exp(l_i
// - M) in Q16 with M the row's maximum. The exponentials are rounded against M,
// so the maximum is settled over the whole row first; within a row the order
// is that of the logits, so a row's best n need no lse.
//
// Three launches, each starting while the one before drains. k_beam_top: the
// largest values of the row's parts, a part per CTA, and of their warps. Where n
// of these entries or more reach a bound, so do n values; the n-th largest entry
// is such a bound, and few more values reach it, as most lie in warps of their
// own. (The least of n groups' maxima, which is cheaper to find, lets n ln n
// through, and whatever there is where a group is short.) k_beam_sum: the same
// parts again, from L2, now that the maximum is known: the exponentials' sum,
// and what reaches the bound goes to the row's list. k_beam_merge: a warp per
// row ranks the list by counting, then the beams' lists are merged. Values
// carry their index (in the bound, their quad's) as the low half of a 64-bit
// key, so that equal logits do not all pass.
// Bound: over 24 x 5 rows of 128256 logits (28.7 us) the first launch by memory
// (10.7 us, 5.7 TB/s of the 62 MB), the second by integer instructions (13.6 us, 21
// a logit and the CTAs' starts), the third by one warp's latency (4.4 us); over 1 x
// 4 of 151936 (9.9 us) by the three launches' latencies. (A cluster of 8 or 16
// CTAs per row, the row in registers between the passes, took 41 and 11.5 us.)
#pragma once
#include "kernels.h"
#include "ptx.cuh"
#include "int_device.cuh"

namespace detint {

constexpr int BM_NT = 256, BM_NW = BM_NT / 32;   // threads, warps of a part
constexpr int BM_Q = 4;                  // quads of a thread and round
constexpr int BM_ROUND = BM_NT * BM_Q * 4;
constexpr int BM_PARTS = 64;             // parts of a row, at most
constexpr int BM_CAP = 512;              // values of a row over the bound that are listed
constexpr int BM_MAX_OUT = 64;           // continuations of a group; beams
constexpr int BM_MASKED = -2147483647 - 1;

struct BeamArgs {
    const int32_t* logits;
    size_t stride;                       // elements between rows
    const long long* scores;             // [rows]
    const int32_t* done;                 // [rows] or null
    int n, n_out, end_id, beams;
    int parts, rounds;                   // of a row; of a part
    int per_part, per_warp;              // place of the bound among the parts' entries (0: not taken), and the warps'
    int lanes;                           // a warp's entry is the lanes-th largest of its lanes' maxima
    unsigned long long *part_key, *key;  // [rows][parts], [rows][parts BM_NW]: the entries
    unsigned long long *sum, *list;      // [rows][parts], [rows][BM_CAP]
    int32_t *top, *most;                 // [rows][parts] maxima, [rows]: the row's
    unsigned* count;                     // [rows]
    int32_t *parent, *token, *done_out;  // [groups][n_out]
    long long* score_out;
};
// whether a row has continuations of its own (k_beam_merge gives a finished beam its one)
__device__ __forceinline__ bool bm_open(const BeamArgs& a, int r) {
    return a.scores[r] >= -(1ll << 62) && !(a.done && a.done[r]);
}

// a value and its index as one key: larger values, then smaller indexes, are
// larger (0 is no value's key, and neither are all ones)
__device__ __forceinline__ u64 bm_key(int v, int idx) { return ((u64)((unsigned)v ^ 0x80000000u) << 32) | (unsigned)(0x7fffffff - idx); }
__device__ __forceinline__ int bm_value(u64 key) { return (int)((unsigned)(key >> 32) ^ 0x80000000u); }
__device__ __forceinline__ int bm_index(u64 key) { return 0x7fffffff - (int)(unsigned)key; }
__device__ __forceinline__ u64 umax64(u64 a, u64 b) { return a > b ? a : b; }

// exp(l - M) in Q30 of Q16 logits l <= M: with d = M - l, -delta = (d L2E + 2^20 -
// 1) >> 21 octaves in Q10, which is the high word of d (L2E 2^11) + (2^20 - 1)
// 2^11; here m = -delta - 1, so that the fraction is ~m and the octaves down
// are (m >> 10) + 1. exp2q's cubic p of the fraction comes from a table of the
// CTA's (2^16 p; computing it took 25 instructions a logit in place of 21); then
// rshr(2^15 p, sh) = (((2^16 p) >> sh) + 1) >> 1. Zero from 31 octaves down:
// below `least` (what it is there is not used, but computed: a branch for each
// value cost more).
constexpr int BM_TABLE = 1024;
__device__ __forceinline__ unsigned bm_octave(int f) {
    const int v1 = (2562 * f + (512 + (7419 << 10))) >> 10;
    const int v2 = (f * v1 + (512 + (22787 << 10))) >> 10;
    return (unsigned)((f * v2 + (512 + (32768 << 10))) >> 10) << 16;
}
__device__ __forceinline__ unsigned bm_exp(const unsigned* table, int l, int M, int least) {
    const u64 w = (u64)((unsigned)M - (unsigned)l) * (47274u << 11) + (((1ull << 20) - 1) << 11) - (1ull << 32);
    const int m = (int)(w >> 32);
    unsigned e;
    asm("shr.u32 %0, %1, %2;" : "=r"(e) : "r"(table[~m & (BM_TABLE - 1)]), "r"((m + 1024) >> 10));
    e = (e + 1) >> 1;
    return l >= least ? e : 0u;
}
// -delta <= 30 2^10, that is d L2E + 2^20 - 1 < 30721 2^21
constexpr int BM_FAR = (int)(((30721ull << 21) - (1ull << 20)) / 47274);
__device__ __forceinline__ int bm_least(int M) { return (int)max((i64)M - BM_FAR, (i64)BM_MASKED + 1); }
// ln(S / 2^30) in Q16, S >= 2^30: log2 to 20 bits below the point, a bit per
// squaring of the 32-bit mantissa, times ln 2
__device__ __forceinline__ i64 bm_ln(u64 S) {
    const int b = bitlen_u64(S);
    unsigned y = (unsigned)(b <= 32 ? S << (32 - b) : S >> (b - 32));
    int lg = b - 31;                                     // (at most 24 2^20)
#pragma unroll 4
    for (int i = 0; i < 20; ++i) {
        const u64 z = (u64)y * y;
        const unsigned hi = (unsigned)(z >> 32);
        lg = 2 * lg + (int)(hi >> 31);
        y = (int)hi < 0 ? hi : (unsigned)(z >> 31);
    }
    return rshr((i64)lg * 726817, 24);
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

// a round of a part: BM_Q quads per thread, from `base` on
template <bool VEC>
struct BmRound {
    int4 x[BM_Q];
    __device__ __forceinline__ void load(const int32_t* row, int base, int n) {
#pragma unroll
        for (int q = 0; q < BM_Q; ++q) x[q] = bm_load<VEC>(row, base + (q * BM_NT + (int)threadIdx.x) * 4, n);
    }
    template <class F>
    __device__ __forceinline__ void each(int base, F f) const {
#pragma unroll
        for (int q = 0; q < BM_Q; ++q) {
            const int i = base + (q * BM_NT + (int)threadIdx.x) * 4;
            f(x[q].x, i);
            f(x[q].y, i + 1);
            f(x[q].z, i + 2);
            f(x[q].w, i + 3);
        }
    }
    __device__ __forceinline__ int most() const {        // the largest value
        int m = BM_MASKED;
#pragma unroll
        for (int q = 0; q < BM_Q; ++q) m = max(m, max(max(x[q].x, x[q].y), max(x[q].z, x[q].w)));
        return m;
    }
};

template <bool VEC>
__global__ void __launch_bounds__(BM_NT) k_beam_top(BeamArgs a) {
    __shared__ u64 best[BM_NW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x, r = blockIdx.y;
    pdl_launch();
    const int32_t* row = a.logits + (size_t)r * a.stride;
    const int first = part * a.rounds * BM_ROUND;
    BmRound<VEC> x, y;
    y.load(row, first, a.n);                             // (on its way while the beam is looked at)
    if (!bm_open(a, r)) return;
    int top = BM_MASKED, at = 0;                         // this thread's largest value, the first quad that holds it
    for (int i = 0; i < a.rounds; ++i) {
        const int base = first + i * BM_ROUND;
        x = y;
        if (i + 1 < a.rounds) y.load(row, base + BM_ROUND, a.n);
#pragma unroll
        for (int q = 0; q < BM_Q; ++q) {
            const int m = max(max(x.x[q].x, x.x[q].y), max(x.x[q].z, x.x[q].w));
            if (m > top) { top = m; at = base + (q * BM_NT + (int)threadIdx.x) * 4; }
        }
    }
    u64 k = top == BM_MASKED ? 0 : bm_key(top, at), wk = redux_max_u64(k);
    if (lane == 0) best[warp] = wk;
    for (int i = 1; i < a.lanes; ++i) {                  // the lanes-th largest of the warp's lanes
        if (k == wk) k = 0;
        wk = redux_max_u64(k);
    }
    const size_t e = (size_t)r * a.parts + part;
    if (lane == 0) a.key[e * BM_NW + warp] = wk;
    __syncthreads();
    if (threadIdx.x == 0) {
        u64 m = 0;
#pragma unroll
        for (int w = 0; w < BM_NW; ++w) m = umax64(m, best[w]);
        a.part_key[e] = m;
        a.top[e] = m ? bm_value(m) : BM_MASKED;
        if (part == 0) a.count[r] = 0;
    }
}

// the want-th largest of n entries (0 where fewer have a value): the rank of each
// by counting; entries that have a value differ
__device__ __forceinline__ void bm_nth(const u64* key, int n, int want, u64* out) {
    for (int e = threadIdx.x; e < n; e += BM_NT) {
        const u64 k = key[e];
        int better = 0;
#pragma unroll 8
        for (int j = 0; j < n; j += 2) {                 // (an entry of 0 behind an odd end)
            const ulonglong2 o = *(const ulonglong2*)(key + j);
            better += (o.x > k) + (o.y > k);
        }
        if (better == want - 1) *out = k;
    }
}

template <bool VEC>
__global__ void __launch_bounds__(BM_NT, 4) k_beam_sum(BeamArgs a) {
    __shared__ __align__(16) u64 key[BM_PARTS * BM_NW + 2];
    __shared__ u64 wsum[BM_NW], tau_s;
    __shared__ unsigned table[BM_TABLE];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = blockIdx.x, r = blockIdx.y;
    pdl_launch();
    const int32_t* row = a.logits + (size_t)r * a.stride;
    const int first = part * a.rounds * BM_ROUND;
    BmRound<VEC> x, y;
    y.load(row, first, a.n);
    const bool open = bm_open(a, r);
    if (tid == 0) tau_s = 0;
#pragma unroll
    for (int i = 0; i < BM_TABLE; i += BM_NT) table[i + tid] = bm_octave(i + tid);
    pdl_wait();                                          // (every CTA, so that this launch ends after the one before)
    if (!open) return;
    int m = max(lane < a.parts ? __ldcg(a.top + (size_t)r * a.parts + lane) : BM_MASKED,
                lane + 32 < a.parts ? __ldcg(a.top + (size_t)r * a.parts + lane + 32) : BM_MASKED);
    for (int fine = a.per_part ? 0 : 1; fine < 2; ++fine) {
        // the parts' entries, and the warps' where too few of those have a value
        const int n = fine ? a.parts * BM_NW : a.parts, per = fine ? a.per_warp : a.per_part;
        const unsigned long long* src = (fine ? a.key : a.part_key) + (size_t)r * n;
        for (int e = tid; e < n + (n & 1); e += BM_NT) key[e] = e < n ? __ldcg(src + e) : 0;
        __syncthreads();
        bm_nth(key, n, per, &tau_s);
        __syncthreads();
        if (tau_s) break;
    }
    const int M = __reduce_max_sync(0xffffffffu, m);
    if (part == 0 && tid == 0) a.most[r] = M;
    // the bound names a quad: equal values up to its last element reach it; a masked value has no key
    const u64 tau = tau_s ? tau_s - 3 : 1;
    const int tau_v = tau_s ? bm_value(tau_s) : BM_MASKED + 1, least = bm_least(M);
    u64 sum = 0;
    for (int i = 0; i < a.rounds; ++i) {
        const int base = first + i * BM_ROUND;
        x = y;
        if (i + 1 < a.rounds) y.load(row, base + BM_ROUND, a.n);
#pragma unroll
        for (int q = 0; q < BM_Q; ++q) {
            // (two exponentials stay below 2^32)
            sum += bm_exp(table, x.x[q].x, M, least) + bm_exp(table, x.x[q].y, M, least);
            sum += bm_exp(table, x.x[q].z, M, least) + bm_exp(table, x.x[q].w, M, least);
        }
        if (x.most() >= tau_v)
            x.each(base, [&](int v, int j) {
                if (v >= tau_v && bm_key(v, j) >= tau) {
                    const unsigned to = atomicAdd(a.count + r, 1u);
                    if (to < BM_CAP) a.list[(size_t)r * BM_CAP + to] = bm_key(v, j);
                }
            });
    }
    sum = redux_sum_u64(sum);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        u64 t = 0;
#pragma unroll
        for (int w = 0; w < BM_NW; ++w) t += wsum[w];
        a.sum[(size_t)r * a.parts + part] = t;
    }
}

// A group's rows, a warp each: the sum's logarithm, and the list ranked by
// counting. A list that ran over is found again by n_out sweeps of the row.
// Then the best n_out of the group: a candidate's place is the number of
// better ones, found in every other beam's sorted list by halving.
constexpr int BM_MERGE = 512, BM_MERGE_NW = BM_MERGE / 32;
__global__ void __launch_bounds__(BM_MERGE) k_beam_merge(BeamArgs a) {
    extern __shared__ __align__(16) unsigned char bm_raw[];
    __shared__ int len[BM_MAX_OUT], ended[BM_MAX_OUT], over[BM_MAX_OUT];
    __shared__ u64 best[BM_MERGE_NW];
    const int W = a.beams, n = a.n_out, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r0 = (int)blockIdx.x * W;
    constexpr int NT = BM_MERGE, NW = BM_MERGE_NW;
    i64* sc = (i64*)bm_raw;                              // [W][n] scores, best first
    int* tk = (int*)(sc + W * n);                        // [W][n] tokens
    u64* buf = (u64*)(bm_raw + ((W * n * 12 + 15) & ~15)) + min(warp, W - 1) * BM_CAP;
    pdl_wait();
    for (int b = warp; b < W; b += NW) {
        const int r = r0 + b;
        // (one trip to memory: what follows the list's end is not looked at)
        const size_t e0 = (size_t)r * a.parts;
        const u64 l0 = __ldcg(a.list + (size_t)r * BM_CAP + lane), l1 = __ldcg(a.list + (size_t)r * BM_CAP + 32 + lane);
        u64 t = lane < a.parts ? __ldcg(a.sum + e0 + lane) : 0;
        const u64 t1 = lane + 32 < a.parts ? __ldcg(a.sum + e0 + 32 + lane) : 0;
        int c = (int)__ldcg(a.count + r);
        const int m = __ldcg(a.most + r);
        const i64 score = min((i64)a.scores[r], 1ll << 62);
        const bool dead = score < -(1ll << 62), end = !dead && a.done && a.done[r];
        if (dead || end) {
            if (lane == 0 && end) { sc[b * n] = score; tk[b * n] = a.end_id; }
            c = end;
        } else {
            buf[lane] = l0;
            buf[lane + 32] = l1;
            for (int i = 64 + lane; i < min(c, BM_CAP); i += 32) buf[i] = __ldcg(a.list + (size_t)r * BM_CAP + i);
            t = redux_sum_u64(t + t1);
            const i64 base = t ? score - m - bm_ln(t) : 0;
            __syncwarp();
            if (c <= BM_CAP) {
                for (int i = lane; i < c; i += 32) {
                    const u64 k = buf[i];
                    int better = 0;
#pragma unroll 8
                    for (int j = 0; j < c; ++j) better += buf[j] > k;
                    if (better < n) {
                        sc[b * n + better] = base + bm_value(k);
                        tk[b * n + better] = bm_index(k);
                    }
                }
            } else if (lane == 0) {
                sc[b * n] = base;
            }
            __syncwarp();
        }
        if (lane == 0) {
            len[b] = min(c, n);
            ended[b] = end;
            over[b] = c > BM_CAP;
        }
    }
    __syncthreads();
    for (int b = 0; b < W; ++b) {
        if (!over[b]) continue;
        const int32_t* row = a.logits + (size_t)(r0 + b) * a.stride;
        const i64 base = sc[b * n];
        u64 last = ~0ull;
        for (int i = 0; i < n; ++i) {                    // the best one below the last
            u64 k = 0;
            for (int j = tid; j < a.n; j += NT) {
                const int v = __ldg(row + j);
                const u64 y = v == BM_MASKED ? 0 : bm_key(v, j);
                if (y < last) k = umax64(k, y);
            }
            k = redux_max_u64(k);
            __syncthreads();
            if (lane == 0) best[warp] = k;
            __syncthreads();
            k = 0;
            for (int w = 0; w < NW; ++w) k = umax64(k, best[w]);
            last = k;
            if (tid == 0) {
                sc[b * n + i] = base + bm_value(k);
                tk[b * n + i] = bm_index(k);
            }
        }
        __syncthreads();
    }
    const size_t out = (size_t)blockIdx.x * n;
    int total = 0;
    for (int q = 0; q < W; ++q) total += len[q];
    for (int i = total + tid; i < n; i += NT) {
        a.parent[out + i] = a.token[out + i] = -1;
        a.score_out[out + i] = (long long)(1ull << 63);
        a.done_out[out + i] = 0;
    }
    for (int b = warp; b < W; b += NW)
        for (int i = lane; i < len[b]; i += 32) {
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
                const int tok = tk[b * n + i];
                a.parent[out + place] = b;
                a.token[out + place] = tok;
                a.score_out[out + place] = s;
                a.done_out[out + place] = ended[b] || tok == a.end_id;
            }
        }
}

// cache blocks of a model, one launch for every layer (a copy call for each part of
// a layer would be 56 calls a pair at 28 layers): pair blockIdx.x, part and layer
// blockIdx.y; bound by memory once there are a few pairs
constexpr int CB_PAIRS = 64;
struct BlockPairs {
    int src[CB_PAIRS], dst[CB_PAIRS];
};
__global__ void __launch_bounds__(256) k_copy_blocks(BlockParts b, BlockPairs p) {
    int part = 0, layer = blockIdx.y;
    while (layer >= b.layers) { layer -= b.layers; ++part; }
    const size_t bytes = b.bytes[part];
    uint8_t* base = b.base[part] + (size_t)layer * b.nblocks * bytes;
    const int4* s = (const int4*)(base + (size_t)p.src[blockIdx.x] * bytes);
    int4* d = (int4*)(base + (size_t)p.dst[blockIdx.x] * bytes);
#pragma unroll 4
    for (int i = threadIdx.x; i < (int)(bytes >> 4); i += 256) d[i] = s[i];
}

// ---- the chosen beams' block tables. Whole pages are shared. Of the page that
// is still being filled (column len / 64) a beam's first child becomes the
// owner; every other child takes the page of a beam without children, into
// which its parent's is to be copied (src, dst: -1 where nothing is), and so does a
// row without a parent, which holds no beam any more and gets no copy. So a
// group's beams keep as many growing pages as they had, nothing is allocated,
// and no page that is copied to is copied from. A column's entries are read by
// one CTA before it writes them: out may be the table itself.
// Bound: latency (lengths, parents and table, then a pass over W parents for the
// growing column); with the copies 4.7 us for 1 x 4 beams of 575 tokens, 7.3 us
// for 32 x 8 of 4000 with their weights (8 kv heads of 128).
constexpr int BR_COLS = 64, BR_THREADS = 256;
__global__ void __launch_bounds__(BR_THREADS) k_beam_reorder(const int32_t* table, int32_t* out, const int32_t* parent,
                                                            const int32_t* lens, int W, int max_blocks, int32_t* src,
                                                            int32_t* dst) {
    __shared__ int32_t old[BM_MAX_OUT][BR_COLS];
    __shared__ int par[BM_MAX_OUT], first[BM_MAX_OUT], used[BM_MAX_OUT], spare[BM_MAX_OUT];
    const int tid = threadIdx.x, c0 = (int)blockIdx.x * BR_COLS, r0 = (int)blockIdx.y * W;
    pdl_launch();                                        // (k_kv4_copy waits for the lists)
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
