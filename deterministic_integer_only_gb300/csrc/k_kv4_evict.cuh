// What a context costs and what is kept of it: the attention probabilities of
// query tokens added up for each cached key (weigh), the keys of the largest
// sums moved to new pages (evict), and copies of whole pages. Arithmetic
// specification, sections 18 and 19.
#pragma once
#include "k_kv4.cuh"

namespace detint {

struct Kv4Weigh {
    long long* weight;                   // [n_blocks][n_kv][64], Q24, added to
};

// p = rshr(E RS, bl - 1) with RS = floor(2^(bl + 23) / sum E), bl = bitlen(sum E)
// >= 15: the probability in Q24. E RS < 2^39; p <= 2^24 and a rounding.
__device__ __forceinline__ unsigned kv4_p24(int E, unsigned RS, int bl) {
    return (unsigned)(((u64)((i64)E * RS) + (1ull << (bl - 2))) >> (bl - 1));
}

// ------------------------------------------------- weights, single tokens
// A unit is a token, a kv head and up to GT of its q heads; its pages are
// split over a cluster of CTAs that keep their scores in shared memory, as in
// k_kv4_decode: scores (dp4a, a page per warp), the maximum over the cluster,
// exponentials in the scores' places and their sum over the cluster, then the
// heads' probabilities of a key are added and sent to the key's weight by one
// 64-bit integer atomic (exact, so the order does not matter; tokens of
// sequences that share pages meet there).
template <int GT>
struct Kv4WeighSm {
    int red[8][GT];
    int cmax[GT], tmax[GT];
    unsigned se[8][GT], csum[GT];
    unsigned RS[GT];
    int bl[GT];
    Kv4Row row[GT];
};

template <int D, int GT>
__global__ void __launch_bounds__(KV4_DT, 2) k_kv4_weigh(Kv4Args a, Kv4Attn p, Kv4Weigh wg) {
    using C = Kv4Ring<D>;
    using Q = Kv4Q<D, GT>;
    constexpr int LPK = Q::LPK, HPL = Q::HPL, NPASS = (GT + 1) / 2;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ Kv4WeighSm<GT> sm;
    __shared__ unsigned long long full[8][C::NST];
    int* pg = (int*)(kv4_raw + C::BYTES);                // [cap / 64]
    const int pitch = p.cap + 8;                         // 8 banks between heads
    int* ts = pg + (((p.cap >> 6) + 3) & ~3);            // [GT][pitch]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.z + p.t0;
    const unsigned rank = blockIdx.x, S = gridDim.x;
    int g = blockIdx.y, hg = 0;
    while (g >= a.n_kv) { g -= a.n_kv; ++hg; }
    const int nh = min(GT, p.G - hg * GT), h0 = g * p.G + hg * GT;
    const int pos = p.tok_pos[t], seq = p.tok_seq[t];
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (pos < 0 || pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks) {
        // no key (the whole unit takes this way out)
        if (rank == 0 && pos >= 0 && tid == 0 && a.status) a.status[ST_CTX] = 1;
        return;
    }
    const int j1 = pos + 1, j0 = p.window > 0 ? max(0, j1 - p.window) : 0;
    const int b0 = j0 >> 6, nb = ((j1 + 63) >> 6) - b0;
    const int per = (int)(((u64)(nb + (int)S - 1) * p.smul) >> 32);     // ceil(nb / S)
    const int pg0 = b0 + (int)rank * per, np = max(0, min(per, b0 + nb - pg0));
    // this CTA's pages, -1 for an entry outside the pool (its keys are masked)
    for (int i = tid; i < np; i += KV4_DT) {
        int blk = a.block_table[(size_t)seq * a.max_blocks + pg0 + i];
        if (blk < 0 || blk >= a.n_blocks) {
            blk = -1;
            if (a.status) a.status[ST_CTX] = 1;
        }
        pg[i] = blk;
    }
    if (tid < GT) {
        const size_t qi = (size_t)t * a.nq + h0 + min(tid, nh - 1);
        sm.row[tid] = kv4_row(p.mq[qi], p.kq[qi], kvp[6], kvp[7]);
    }
    if (lane == 0)
        for (int i = 0; i < C::NST; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    Q qr;
    qr.load(p.q8 + ((size_t)t * a.nq + h0) * D, nh);
    __syncthreads();

    // ---- scores: this warp's pages warp, warp + 8, ... through its ring
    const int nk = np > warp ? (np - warp + 7) >> 3 : 0;
    unsigned char* ring = kv4_raw + warp * (C::NST * C::SLOT);
    auto issue = [&](int q) {
        if (q >= nk || lane) return;
        const int st = q & (C::NST - 1), blk = pg[warp + 8 * q];
        const uint32_t bar = smem_u32(&full[warp][st]), dst = smem_u32(ring + st * C::SLOT);
        if (blk < 0) {
            mbar_arrive(bar);
        } else {
            const size_t u = (size_t)blk * a.n_kv + g;
            mbar_arrive_expect_tx(bar, C::PG + KV_BLK);
            bulk_g2s(dst, a.k + u * C::PG, C::PG, bar);
            bulk_g2s(dst + C::PG, a.ks + u * KV_BLK, KV_BLK, bar);
        }
    };
#pragma unroll
    for (int q = 0; q < C::NST; ++q) issue(q);
    int tm[HPL];
#pragma unroll
    for (int x = 0; x < HPL; ++x) tm[x] = p.none;
    const int sub = lane & (LPK - 1), hb = sub / Q::LPG * HPL;
    for (int q = 0; q < nk; ++q) {
        const int pi = warp + 8 * q, jb = (pg0 + pi) << 6;
        const bool ok = pg[pi] >= 0;
        kv4_wait(&full[warp][q & (C::NST - 1)], (q / C::NST) & 1, p.polls, a.status);
        qr.page(ring + (q & (C::NST - 1)) * C::SLOT, ts + hb * pitch + pi * KV_BLK + lane / LPK, pitch,
                ok && jb >= j0 && jb + 64 <= j1, j0 - jb, ok ? j1 - jb : -1, tm);
        __syncwarp();
        issue(q + C::NST);
    }
#pragma unroll
    for (int x = 0; x < HPL; ++x) {
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) tm[x] = max(tm[x], __shfl_xor_sync(0xffffffffu, tm[x], o));
        if (lane < LPK && (sub & (Q::LPG - 1)) == 0) sm.red[warp][hb + x] = tm[x];
    }
    __syncthreads();
    // ---- the maximum over every CTA of the unit
    if (tid < GT) {
        int m = sm.red[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, sm.red[w][tid]);
        sm.cmax[tid] = m;
    }
    if (S > 1) cl_sync();
    else __syncthreads();
    for (int h = warp; h < GT; h += 8) {
        int m = KV4_NEG;
        for (unsigned r = lane; r < S; r += 32) m = max(m, S > 1 ? cl_ld32(&sm.cmax[h], r) : sm.cmax[h]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) sm.tmax[h] = m;
    }
    __syncthreads();

    // ---- exponentials in the scores' places, four keys of a head per thread
    unsigned sumE[NPASS];
#pragma unroll
    for (int x = 0; x < NPASS; ++x) {
        sumE[x] = 0;
        const int h = 2 * x + (tid >> 7);
        if (h < GT) {
            const Kv4Row rw = sm.row[h];
            const int T = sm.tmax[h];
            for (int k = 4 * (tid & 127); k < np * KV_BLK; k += 512) {
                int4* at = (int4*)(ts + h * pitch + k);
                const int jb = (pg0 << 6) + k;
                const bool ok = pg[k >> 6] >= 0;
                int4 v = make_int4(0, 0, 0, 0);
                if (ok) {
                    v = *at;
                    v.x = jb >= j0 && jb < j1 ? kv4_E(rw, v.x, T) : 0;
                    v.y = jb + 1 >= j0 && jb + 1 < j1 ? kv4_E(rw, v.y, T) : 0;
                    v.z = jb + 2 >= j0 && jb + 2 < j1 ? kv4_E(rw, v.z, T) : 0;
                    v.w = jb + 3 >= j0 && jb + 3 < j1 ? kv4_E(rw, v.w, T) : 0;
                }
                *at = v;
                sumE[x] += (unsigned)(v.x + v.y + v.z + v.w);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < NPASS; ++x) {
        const int h = 2 * x + (tid >> 7);
        const unsigned e = __reduce_add_sync(0xffffffffu, sumE[x]);
        if (lane == 0 && h < GT) sm.se[warp][h] = e;
    }
    __syncthreads();
    if (tid < GT) {
        unsigned e = 0;
        const int wbase = (tid & 1) * 4;                 // head h = 2 x + (warp >= 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) e += sm.se[wbase + k][tid];
        sm.csum[tid] = e;                                // below 2^15 keys of a CTA: below 2^30
    }
    if (S > 1) cl_sync();
    else __syncthreads();
    for (int h = warp; h < GT; h += 8) {
        u64 e = 0;
        for (unsigned r = lane; r < S; r += 32) e += (unsigned)(S > 1 ? cl_ld32((const int*)&sm.csum[h], r) : (int)sm.csum[h]);
        e = redux_sum_u64(e);
        if (lane == 0) {
            const int bl = bitlen_u64(e);
            sm.RS[h] = e && h < nh ? (unsigned)pow2_recip(e, bl, 1, 23) : 0;
            sm.bl[h] = max(bl, 2);
        }
    }
    if (S > 1) cl_sync();      // (no CTA leaves while another reads its shared memory)
    else __syncthreads();
    // ---- the heads' probabilities of a key
    unsigned RS[GT];
    int bl[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) { RS[h] = sm.RS[h]; bl[h] = sm.bl[h]; }
    for (int k = tid; k < np * KV_BLK; k += KV4_DT) {
        unsigned s = 0;
#pragma unroll
        for (int h = 0; h < GT; ++h) s += kv4_p24(ts[h * pitch + k], RS[h], bl[h]);
        if (s) atomicAdd((unsigned long long*)wg.weight + ((size_t)pg[k >> 6] * a.n_kv + g) * KV_BLK + (k & 63), (unsigned long long)s);
    }
}

// ------------------------------------------------------------------ eviction
// The kept places of one sequence and kv head, ascending: the first `sinks`
// and last `recent` ones and, between them, those of the largest weights, the
// lower place first among equal ones. A cluster per sequence and kv head, a
// run of whole pages per CTA, the weights in shared memory as order-preserving
// keys. The least kept key is found from its leading bits: a histogram of the
// next 11 bits of the keys that agree so far, until its bin is taken whole or
// the bits run out. Then a prefix sum over the places deals the kept ones out.
constexpr int EV_THREADS = 512, EV_WARPS = EV_THREADS / 32;
constexpr int EV_BITS = 11, EV_BINS = 1 << EV_BITS;

struct Kv4Evict {
    const long long* weight_in;          // = weight
    long long* weight;
    const int32_t *seq, *lens;           // [n]
    const int32_t* new_table;            // [n][pages of keep]
    int32_t* kept;                       // [n][n_kv][keep]
    int max_len, keep, sinks, recent;
    int new_blocks;                      // pages of keep
    int lg_s, cap;                       // log2 of the CTAs of a cluster; keys of a CTA (whole pages)
    int held;                            // the keys fit shared memory
};

__device__ __forceinline__ u64 ev_key(long long w) { return (u64)w ^ (1ull << 63); }

__global__ void __launch_bounds__(EV_THREADS) k_kv4_evict_select(Kv4Args a, Kv4Evict p) {
    extern __shared__ __align__(16) unsigned char ev_raw[];
    u64* keys = (u64*)ev_raw;                            // [cap] where they are held
    __shared__ unsigned hist[EV_BINS];
    __shared__ u64 red[2][EV_WARPS], range[2];           // largest key, smallest key (complemented)
    __shared__ unsigned scan[2][EV_WARPS], mine[2], pick[3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = 1 << p.lg_s, rank = (int)blockIdx.x & (S - 1), i = (int)blockIdx.x >> p.lg_s, g = blockIdx.y;
    const int seq = p.seq[i], max_len = min(p.max_len, a.max_blocks * KV_BLK);
    int len = p.lens[i];
    int32_t* out = p.kept + ((size_t)i * a.n_kv + g) * p.keep;
    if (seq < 0 || seq >= a.n_seq || len < 0 || len > max_len) {
        if (tid == 0 && a.status) a.status[ST_CTX] = 1;
        len = 0;
    }
    if (len <= p.keep) {                                 // everything stays (the whole cluster takes this way out)
        for (int j = rank * EV_THREADS + tid; j < p.keep; j += S * EV_THREADS) out[j] = j < len ? j : -1;
        return;
    }
    const int lo = p.sinks, hi = len - p.recent;         // the places that are weighed
    unsigned want = (unsigned)(p.keep - p.sinks - p.recent);
    const int j0 = rank * p.cap, j1 = min(len, j0 + p.cap);
    const int32_t* row = a.block_table + (size_t)seq * a.max_blocks;
    auto fetch = [&](int j) -> u64 {
        const int blk = row[j >> 6];
        if (blk < 0 || blk >= a.n_blocks) {
            if (a.status) a.status[ST_CTX] = 1;
            return ev_key(0);
        }
        return ev_key(p.weight_in[((size_t)blk * a.n_kv + g) * KV_BLK + (j & 63)]);
    };
    auto key = [&](int j) -> u64 { return p.held ? keys[j - j0] : fetch(j); };
    u64 top = 0, bot = 0;                                // of the keys, and of their complements
    for (int j = j0 + tid; j < j1; j += EV_THREADS) {
        const u64 k = fetch(j);
        if (p.held) keys[j - j0] = k;
        if (j >= lo && j < hi) {
            top = k > top ? k : top;
            bot = ~k > bot ? ~k : bot;
        }
    }
    top = redux_max_u64(top);
    bot = redux_max_u64(bot);
    if (lane == 0) { red[0][warp] = top; red[1][warp] = bot; }
    __syncthreads();
    if (tid < 2) {
        u64 m = 0;
        for (int w = 0; w < EV_WARPS; ++w) m = red[tid][w] > m ? red[tid][w] : m;
        range[tid] = m;
    }
    for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
    cl_sync();
    top = bot = 0;
    for (int r = 0; r < S; ++r) {
        const u64 x = (u64)cl_ld64((const i64*)&range[0], r), y = (u64)cl_ld64((const i64*)&range[1], r);
        top = x > top ? x : top;
        bot = y > bot ? y : bot;
    }
    bot = ~bot;
    // ---- the want-th largest key: `left` low bits are open, the others agree with `top`
    int left = want ? bitlen_u64(top ^ bot) : 0;
    u64 cut = want ? top : ~0ull;                        // its open bits are yet to be found
    bool whole = false;                                  // every key that agrees with cut's closed bits is kept
    while (left > 0 && !whole) {
        const int sh = max(left - EV_BITS, 0);
        const u64 agree = left >= 64 ? 0 : cut >> left, bins = (1ull << (left - sh)) - 1;
        for (int j = max(j0, lo) + tid; j < min(j1, hi); j += EV_THREADS) {
            const u64 k = key(j);
            if (left >= 64 || k >> left == agree) atomicAdd(&hist[(k >> sh) & bins], 1u);
        }
        __syncthreads();
        if (rank)                                        // the first CTA's bins become the cluster's
            for (int b = tid; b < EV_BINS; b += EV_THREADS)
                if (hist[b]) {
                    cl_add32(&hist[b], 0, hist[b]);
                    hist[b] = 0;
                }
        cl_sync();
        if (rank == 0) {
            // from the highest bin down: the bin in which `want` is reached
            unsigned c[EV_BINS / EV_THREADS], sum = 0;
#pragma unroll
            for (int x = 0; x < EV_BINS / EV_THREADS; ++x) {
                c[x] = hist[EV_BINS - 1 - (tid * (EV_BINS / EV_THREADS) + x)];
                sum += c[x];
            }
            unsigned inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) scan[0][warp] = inc;
            __syncthreads();
            unsigned before = inc - sum;
            for (int w = 0; w < warp; ++w) before += scan[0][w];
            if (before < want && want <= before + sum) {
                int x = 0;
#pragma unroll
                for (; x < EV_BINS / EV_THREADS - 1; ++x) {
                    if (want <= before + c[x]) break;
                    before += c[x];
                }
                unsigned n = 0;
#pragma unroll
                for (int y = 0; y < EV_BINS / EV_THREADS; ++y)
                    if (y == x) n = c[y];
                pick[0] = (unsigned)(EV_BINS - 1 - (tid * (EV_BINS / EV_THREADS) + x));
                pick[1] = want - before;                 // of the bin's n keys
                pick[2] = n;
            }
            __syncthreads();
            for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
        }
        cl_sync();
        const unsigned bin = cl_ld32u(&pick[0], 0), n = cl_ld32u(&pick[2], 0);
        want = cl_ld32u(&pick[1], 0);
        cut = (agree << (left - sh) | bin) << sh;
        left = sh;
        whole = want == n;
        cl_sync();                                       // pick is read before it is written again
    }
    // kept: places outside [lo, hi), keys past the bits of cut (all that agree with
    // them too when whole), and the first `want` of those equal to it
    const u64 edge = cut >> left;
    unsigned take = 0, ties = 0;
    // a thread's run of places, so that the places ascend with the threads
    const int span = (p.cap + EV_THREADS - 1) / EV_THREADS, a0 = j0 + tid * span, a1 = min(j1, a0 + span);
    auto kind = [&](int j) -> int {                      // 2 kept, 1 equal to the cut, 0 not kept
        if (j < lo || j >= hi) return 2;
        if (!want) return 0;
        const u64 k = key(j) >> left;
        return k > edge || (whole && k == edge) ? 2 : (k == edge ? 1 : 0);
    };
    for (int j = a0; j < a1; ++j) {
        const int t = kind(j);
        take += t == 2;
        ties += t == 1;
    }
    unsigned it = take, ie = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, it, o), z = __shfl_up_sync(0xffffffffu, ie, o);
        if (lane >= o) { it += y; ie += z; }
    }
    if (lane == 31) { scan[0][warp] = it; scan[1][warp] = ie; }
    __syncthreads();
    unsigned bt = it - take, be = ie - ties, nt = 0, ne = 0;
    for (int w = 0; w < EV_WARPS; ++w) {
        if (w == warp) { bt += nt; be += ne; }
        nt += scan[0][w];
        ne += scan[1][w];
    }
    if (tid == 0) { mine[0] = nt; mine[1] = ne; }
    cl_sync();
    for (int r = 0; r < rank; ++r) {
        bt += cl_ld32u(&mine[0], r);
        be += cl_ld32u(&mine[1], r);
    }
    for (int j = a0; j < a1; ++j) {
        const int t = kind(j);
        if (t == 2 || (t == 1 && be < want)) out[bt + min(be, want)] = j;
        bt += t == 2;
        be += t == 1;
    }
    cl_sync();                                           // no CTA leaves while another reads its shared memory
}

// The kept tokens of 64 new places (a page of one kv head), a CTA each: rows
// of keys, scale codes and weights by gathers; the values' codes, packed by
// channel, by one thread per channel that walks the kept places in order,
// takes a source word's kept codes out of it and fills the new words. Places
// behind the last kept token are left as they were. The new pages may not be
// among the sequences' own.
constexpr int KV4_ZEROS = -0x77777778;   // eight codes of zero (8 each)
template <int D>
__global__ void __launch_bounds__(128) k_kv4_evict_move(Kv4Args a, Kv4Evict p) {
    __shared__ int from[KV_BLK], page[KV_BLK];           // places in their pages, and those pages (-1: outside the pool)
    const int tid = threadIdx.x, b = blockIdx.x, g = blockIdx.y, i = blockIdx.z;
    const int seq = p.seq[i];
    const int32_t* kept = p.kept + ((size_t)i * a.n_kv + g) * p.keep;
    int n = 0;
    if (tid < KV_BLK) {
        const int s = b * KV_BLK + tid, j = s < p.keep ? __ldcg(kept + s) : -1;
        int blk = -1;
        if (j >= 0) blk = a.block_table[(size_t)seq * a.max_blocks + (j >> 6)];
        from[tid] = j < 0 ? -1 : j & 63;
        page[tid] = blk >= 0 && blk < a.n_blocks ? blk : -1;
    }
    n = __syncthreads_count(tid < KV_BLK && from[tid & 63] >= 0);        // the kept ones come first
    if (!n) return;
    const int to = p.new_table[(size_t)i * p.new_blocks + b];
    if (to < 0 || to >= a.n_blocks) {
        if (tid == 0 && a.status) a.status[ST_CTX] = 1;
        return;
    }
    const size_t u = (size_t)to * a.n_kv + g;
    // keys: rows of D / 2 bytes
    constexpr int V = D / 32;                            // 16-byte pieces of a row
    for (int x = tid; x < n * V; x += 128) {
        const int s = x / V, c = x & (V - 1), blk = page[s];
        int4 v = make_int4(KV4_ZEROS, KV4_ZEROS, KV4_ZEROS, KV4_ZEROS);
        if (blk >= 0) v = *((const int4*)(a.k + (((size_t)blk * a.n_kv + g) * KV_BLK + from[s]) * (D / 2)) + c);
        *((int4*)(a.k + (u * KV_BLK + s) * (D / 2)) + c) = v;
    }
    if (tid < n) {
        const int blk = page[tid];
        const size_t o = ((size_t)max(blk, 0) * a.n_kv + g) * KV_BLK + from[tid];
        a.ks[u * KV_BLK + tid] = blk >= 0 ? a.ks[o] : 1;
        a.vs[u * KV_BLK + tid] = blk >= 0 ? a.vs[o] : 1;
        p.weight[u * KV_BLK + tid] = blk >= 0 ? p.weight[o] : 0;
    }
    if (tid >= D) return;
    // values: word [key / 16][channel / 8 mod 2][key / 8 mod 2] of a channel's row of 16
    const size_t ch = (size_t)(tid >> 4) * 128 + (tid & 7) * 16 + ((tid >> 3) & 1) * 2;
    const uint32_t* vin = (const uint32_t*)a.v;
    uint32_t* vout = (uint32_t*)a.v + u * (D * KV_BLK / 8) + ch;
    unsigned w = 0;
    for (int s = 0; s < n; ++s) {
        const int blk = page[s], j = from[s];
        unsigned code = 8;
        if (blk >= 0)
            code = vin[((size_t)blk * a.n_kv + g) * (D * KV_BLK / 8) + ch + (j >> 4) * 4 + ((j >> 3) & 1)] >> (8 * (j & 3) + (j & 4)) & 15;
        w |= code << (8 * (s & 3) + (s & 4));
        if ((s & 7) == 7 || s == n - 1) {
            uint32_t* d = vout + (s >> 4) * 4 + ((s >> 3) & 1);
            unsigned keep = 0;                           // codes behind the last kept token
            for (int k = (s & 7) + 1; k < 8; ++k) keep |= 15u << (8 * (k & 3) + (k & 4));
            *d = w | (keep ? *d & keep : 0u);
            w = 0;
        }
    }
}

// whole pages of every kv head, src[i] to dst[i]; -1 on either side: none
__global__ void __launch_bounds__(256) k_kv4_copy(Kv4Args a, const int32_t* src, const int32_t* dst, int page_bytes, long long* weight) {
    const int s = src[blockIdx.x], d = dst[blockIdx.x], g = blockIdx.y;
    if (s < 0 || d < 0) return;
    if (s >= a.n_blocks || d >= a.n_blocks) {
        if (threadIdx.x == 0 && a.status) a.status[ST_CTX] = 1;
        return;
    }
    const size_t us = (size_t)s * a.n_kv + g, ud = (size_t)d * a.n_kv + g;
    const int n = page_bytes >> 4;                       // 16-byte pieces of K, and of V
    for (int x = threadIdx.x; x < 2 * n + 8 + (weight ? 32 : 0); x += 256) {
        const int4* f;
        int4* t;
        if (x < n) { f = (const int4*)(a.k + us * page_bytes) + x; t = (int4*)(a.k + ud * page_bytes) + x; }
        else if (x < 2 * n) { f = (const int4*)(a.v + us * page_bytes) + (x - n); t = (int4*)(a.v + ud * page_bytes) + (x - n); }
        else if (x < 2 * n + 4) { f = (const int4*)(a.ks + us * KV_BLK) + (x - 2 * n); t = (int4*)(a.ks + ud * KV_BLK) + (x - 2 * n); }
        else if (x < 2 * n + 8) { f = (const int4*)(a.vs + us * KV_BLK) + (x - 2 * n - 4); t = (int4*)(a.vs + ud * KV_BLK) + (x - 2 * n - 4); }
        else { f = (const int4*)(weight + us * KV_BLK) + (x - 2 * n - 8); t = (int4*)(weight + ud * KV_BLK) + (x - 2 * n - 8); }
        *t = *f;
    }
}

}  // namespace detint
