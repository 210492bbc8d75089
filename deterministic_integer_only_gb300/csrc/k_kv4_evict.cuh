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
    return (unsigned)(((u64)(unsigned)E * RS + (1ull << (bl - 2))) >> (bl - 1));
}

// the same for sums below 2^32, whose shift one funnel shift does
__device__ __forceinline__ unsigned kv4_p24s(int E, unsigned RS, int bl) {
    const u64 x = (u64)(unsigned)E * RS + (1u << (bl - 2));
    return __funnelshift_r((unsigned)x, (unsigned)(x >> 32), bl - 1);
}

// ------------------------------------------------- weights, single tokens
// A unit is a token, a kv head and up to GT of its q heads; its pages are
// split over a cluster of CTAs that keep their scores in shared memory, as in
// k_kv4_decode: scores (dp4a, a page per warp, whose codes go straight to
// registers: without a ring there is room for twice the scores, and half as many
// CTAs exchange), the maximum over the cluster,
// exponentials in the scores' places and their sum over the cluster, then the
// heads' probabilities of a key are added and sent to the key's weight by one
// 64-bit integer atomic (exact, so the order does not matter; tokens of
// sequences that share pages meet there).
// Bound: phases that wait for memory and for each other: 64 tokens of 4001..16384
// keys, 32 + 8 heads of 128, take 135 us, 2.9 TB/s, for 117 instructions per 32
// scores (32 of them dp4a, the rest unpacking, exponentials and probabilities) that
// would issue in about 65; the ALU is 33 % busy with 24 warps on an SM. 1 token of
// 4000 by latency, 5 us.
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
__global__ void __launch_bounds__(KV4_DT, 3) k_kv4_weigh(Kv4Args a, Kv4Attn p, Kv4Weigh wg) {
    using Q = Kv4Q<D, GT>;
    constexpr int LPK = Q::LPK, HPL = Q::HPL, NPASS = (GT + 1) / 2;
    constexpr int PG = KV_BLK * D / 2, N = KV_BLK / Q::KPL;             // loads of a lane for a page
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ Kv4WeighSm<GT> sm;
    int* pg = (int*)kv4_raw;                             // [cap / 64]
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
    Q qr;
    qr.load(p.q8 + ((size_t)t * a.nq + h0) * D, nh);
    __syncthreads();

    // ---- scores: this warp's pages warp, warp + 8, ...
    const int nk = np > warp ? (np - warp + 7) >> 3 : 0;
    int tm[HPL];
#pragma unroll
    for (int x = 0; x < HPL; ++x) tm[x] = p.none;
    const int sub = lane & (LPK - 1), kl = lane / LPK, hb = sub / Q::LPG * HPL;
    for (int q = 0; q < nk; ++q) {
        const int pi = warp + 8 * q, jb = (pg0 + pi) << 6, blk = pg[pi];
        if (blk < 0) continue;                           // (its scores are not looked at)
        const size_t u = (size_t)blk * a.n_kv + g;
        const unsigned char *kr = a.k + u * PG + kl * (D / 2) + sub * 16, *cr = a.ks + u * KV_BLK + kl;
        const bool clear = jb >= j0 && jb + 64 <= j1;
        int* out = ts + hb * pitch + pi * KV_BLK + kl;
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += 4) {
            int4 kv[4];
            int cv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kv[i] = __ldg((const int4*)(kr + (i0 + i) * (Q::KPL * D / 2)));
                cv[i] = __ldg(cr + (i0 + i) * Q::KPL);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) qr.keys(kv[i], cv[i], i0 + i, out, pitch, clear, j0 - jb, j1 - jb, tm);
        }
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
                int4 v = make_int4(0, 0, 0, 0);
                if (pg[k >> 6] >= 0) {
                    v = *at;
                    v = make_int4(kv4_E(rw, v.x, T), kv4_E(rw, v.y, T), kv4_E(rw, v.z, T), kv4_E(rw, v.w, T));
                    if (jb < j0 || jb + 4 > j1) {
                        if (jb < j0 || jb >= j1) v.x = 0;
                        if (jb + 1 < j0 || jb + 1 >= j1) v.y = 0;
                        if (jb + 2 < j0 || jb + 2 >= j1) v.z = 0;
                        if (jb + 3 < j0 || jb + 3 >= j1) v.w = 0;
                    }
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

// ------------------------------------------------- weights, blocks of tokens
// A cluster of CTAs takes 16 query rows (16 / Gp consecutive tokens times up to
// 16 q heads of one kv head, Gp a power of two) and all their keys at once: a
// warp scores up to 4 pages of 64 keys on the int8 tensor pipe and keeps the
// scores, of one page in its registers, of the others in shared memory, so that
// each is computed once (three sweeps, for the maxima, the sums and the weights,
// would take the tensor pipe three times).
// Two exchanges settle the rows' maxima and sums over the warps and CTAs; then
// the 16 rows' probabilities of a key are added over the lanes and go to the
// key's weight by one 64-bit atomic. Bound: the tensor pipe (45 % busy), the ALU
// (32 %) and the exchanges take turns, as 16 warps fill an SM: 1 x 4096 tokens of 16
// + 8 heads of 128 463 us (217 us would be the pipe's measured rate), 3 x 61 tokens
// after 8000, 32 + 8 of 64, 118 us. Column n of score tile j is key 16 (n / 2)
// + 2 j + (n & 1), so that a lane's scores are 16 neighbouring keys. K fragments
// come straight from the pages: a warp's load is eight whole rows. A block's
// tokens may belong to several sequences: each run of one sequence whose pages
// fit the cluster is a round of its own with the other rows masked.
constexpr int WB_ROWS = 16;
constexpr int WB_PG = 4;                 // pages of a warp
constexpr int WB_SMEM = (WB_PG - 1) * 4096;      // shared memory of a warp, and per warp of the cluster
constexpr int WB_EXCH = 2 * WB_ROWS * 4;

template <int D, int LGW>
__global__ void __launch_bounds__(32 << LGW, 16 >> LGW) k_kv4_weigh_block(Kv4Args a, Kv4Attn p, Kv4Weigh wg) {
    constexpr int KS = D / 32, PG = KV_BLK * D / 2, NW = 1 << LGW;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ int r_pos[WB_ROWS];
    __shared__ Kv4Row r_row[WB_ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
    const int S = 1 << p.lgC, rank = (int)blockIdx.x;
    // the warps' maxima and sums, [warp of the cluster][row]: every warp writes its
    // own to every CTA, so that one cluster barrier is an exchange
    int* const x_top = (int*)(kv4_raw + NW * WB_SMEM);
    int* const x_sum = x_top + S * NW * WB_ROWS;
    int g = blockIdx.y, hg = 0;
    while (g >= a.n_kv) { g -= a.n_kv; ++hg; }
    const int BQ = WB_ROWS >> p.lgGp, Gp = 1 << p.lgGp, h0 = g * p.G + hg * Gp, nh = min(Gp, p.G - hg * Gp);
    const int t0 = p.t0 + (int)(gridDim.z - 1 - blockIdx.z) * BQ;    // later tokens tend to have more keys
    const int nt = min(BQ, p.T - t0);
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (S > 1) cl_arrive();
    if (tid < WB_ROWS) {
        const int i = tid >> p.lgGp, hh = tid & (Gp - 1);
        int pos = -1;
        if (i < nt && hh < nh) {
            pos = p.tok_pos[t0 + i];
            const int seq = p.tok_seq[t0 + i];
            if (pos >= 0 && (pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks)) {
                pos = -1;
                if (a.status) a.status[ST_CTX] = 1;
            }
        }
        r_pos[tid] = pos;
        const bool in = i < nt && hh < nh;
        const size_t qi = (size_t)(t0 + i) * a.nq + h0 + hh;
        r_row[tid] = kv4_row(in ? p.mq[qi] : 0, in ? p.kq[qi] : 0, kvp[6], kvp[7]);
    }
    const int rA = gid, rB = gid + 8;
    int qf[KS][4], qo[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = x ? rB : rA, i = r >> p.lgGp, hh = r & (Gp - 1);
        int w[2 * KS];
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j) w[j] = 0;
        if (i < nt && hh < nh) {
            const int* qp = (const int*)(p.q8 + ((size_t)(t0 + i) * a.nq + h0 + hh) * D + tig * (D / 4));
#pragma unroll
            for (int j = 0; j < 2 * KS; ++j) w[j] = __ldg(qp + j);
        }
        int sq = 0;
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j) sq = __dp4a(w[j], 0x01010101, sq);
        sq += __shfl_xor_sync(0xffffffffu, sq, 1);
        sq += __shfl_xor_sync(0xffffffffu, sq, 2);
        qo[x] = -8 * sq;                                 // the codes are values + 8
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s][x] = w[2 * s];
            qf[s][2 + x] = w[2 * s + 1];
        }
    }
    __syncthreads();
    const Kv4Row rw[2] = {r_row[rA], r_row[rB]};
    if (S > 1) cl_wait();                                // every CTA runs: its shared memory may be written
    // gives row lane mod 16's value of this warp to every CTA / waits for all of them
    auto give = [&](int* x, int va, int vb) {
        const int u = __shfl_sync(0xffffffffu, va, 4 * (lane & 7)), v = __shfl_sync(0xffffffffu, vb, 4 * (lane & 7));
        int* at = x + (rank * NW + warp) * WB_ROWS + (lane & 15);
        for (int c = lane >> 4; c < S; c += 2) cl_st32(at, c, lane & 8 ? v : u);
        if (S > 1) cl_sync();
        else __syncthreads();
    };
    for (int s0 = 0; s0 < nt;) {
        // tokens [s0, s1) of one sequence whose pages fit the cluster (one token's always do)
        const int seq = p.tok_seq[t0 + s0];
        int s1 = s0, kmax = -1, kmin = 0x7fffffff;
        for (; s1 < nt && p.tok_seq[t0 + s1] == seq; ++s1) {
            const int pos = r_pos[s1 << p.lgGp];
            if (pos < 0) continue;
            const int hi = max(kmax, pos), lo = min(kmin, p.window > 0 ? max(0, pos + 1 - p.window) : 0);
            if (kmax >= 0 && (hi >> 6) - (lo >> 6) >= S * NW * WB_PG) break;
            kmax = hi;
            kmin = lo;
        }
        const int iA = rA >> p.lgGp, iB = rB >> p.lgGp;
        const int hiA = iA >= s0 && iA < s1 ? r_pos[rA] : -1, hiB = iB >= s0 && iB < s1 ? r_pos[rB] : -1;
        const int loA = p.window > 0 ? max(0, hiA + 1 - p.window) : 0, loB = p.window > 0 ? max(0, hiB + 1 - p.window) : 0;
        // the keys that every row takes
        const int cmax = __reduce_min_sync(0xffffffffu, min(hiA, hiB)), cmin = __reduce_max_sync(0xffffffffu, max(loA, loB));
        s0 = s1;
        if (kmax < 0) continue;
        const int p0 = kmin >> 6, np = (kmax >> 6) - p0 + 1;
        // ---- scores of this warp's pages rank NW + warp, + S NW, ...; the first one's stay in registers
        const int first = rank * NW + warp, mine = np > first ? ((np - first - 1) >> (p.lgC + LGW)) + 1 : 0;
        int4* const store = (int4*)kv4_raw + warp * ((WB_PG - 1) * 256) + lane - 256;      // page q from [256 q]
        int t[8][4], T[2] = {p.none, p.none}, blk_l = -1;
        if (lane < mine) {
            blk_l = a.block_table[(size_t)seq * a.max_blocks + p0 + first + (lane << (p.lgC + LGW))];
            if (blk_l < 0 || blk_l >= a.n_blocks) {
                blk_l = -1;
                if (a.status) a.status[ST_CTX] = 1;
            }
        }
        auto page_of = [&](int q) { return __shfl_sync(0xffffffffu, blk_l, q); };          // -1: its scores are not looked at
        auto key_of = [&](int q) { return (p0 + first + (q << (p.lgC + LGW))) << 6; };
#pragma unroll 1
        for (int q = mine - 1; q >= 0; --q) {
            const int blk = page_of(q);
            if (blk < 0) continue;
            const size_t u = (size_t)blk * a.n_kv + g;
            const unsigned char* kr = a.k + u * PG + (16 * (gid >> 1) + (gid & 1)) * (D / 2) + tig * (D / 8);
            const int4 cv = __ldg((const int4*)(a.ks + u * KV_BLK) + tig);
            const int cw[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                int w[4][KS];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned char* at = kr + 2 * (4 * hf + j) * (D / 2);
                    if (D == 128) {
                        const int4 v = __ldg((const int4*)at);
                        w[j][0] = v.x; w[j][1] = v.y; w[j][KS - 2] = v.z; w[j][KS - 1] = v.w;
                    } else {
                        const int2 v = __ldg((const int2*)at);
                        w[j][0] = v.x; w[j][1] = v.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    int (&c)[4] = t[4 * hf + j];
                    c[0] = c[1] = qo[0];
                    c[2] = c[3] = qo[1];
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        mma_s8u8(c, qf[s][0], qf[s][1], qf[s][2], qf[s][3], kv4_lo(w[j][s]), kv4_hi(w[j][s]));
                }
            }
            const int kb = key_of(q), k0 = kb + 16 * tig;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int sc = cw[j >> 1] >> (8 * (2 * (j & 1) + e)) & 255;
                    t[j][e] *= sc;
                    t[j][2 + e] *= sc;
                }
            if (kb >= cmin && kb + 63 <= cmax) {         // no key of the page is masked
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    T[0] = max(T[0], max(t[j][0], t[j][1]));
                    T[1] = max(T[1], max(t[j][2], t[j][3]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = k0 + 2 * j + e;
                        if (key <= hiA && key >= loA) T[0] = max(T[0], t[j][e]);
                        if (key <= hiB && key >= loB) T[1] = max(T[1], t[j][2 + e]);
                    }
            }
            if (q)
#pragma unroll
                for (int j = 0; j < 8; ++j) store[256 * q + 32 * j] = make_int4(t[j][0], t[j][1], t[j][2], t[j][3]);
        }
        // ---- the rows' maxima over the warps and CTAs
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 1));
            T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 2));
        }
        give(x_top, T[0], T[1]);
        {
            int m = p.none;
            for (int e = lane >> 4; e < S * NW; e += 2) m = max(m, x_top[e * WB_ROWS + (lane & 15)]);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
            T[0] = __shfl_sync(0xffffffffu, m, rA);
            T[1] = __shfl_sync(0xffffffffu, m, rB);
        }
        // ---- exponentials in the scores' places, and their sums
        unsigned sum[2] = {0, 0};
        auto exps = [&](int (&v)[4]) {
            v[0] = kv4_E(rw[0], v[0], T[0]);
            v[1] = kv4_E(rw[0], v[1], T[0]);
            v[2] = kv4_E(rw[1], v[2], T[1]);
            v[3] = kv4_E(rw[1], v[3], T[1]);
        };
        auto mask = [&](int (&v)[4], int k) {            // keys k, k + 1
            if (k > hiA || k < loA) v[0] = 0;
            if (k + 1 > hiA || k + 1 < loA) v[1] = 0;
            if (k > hiB || k < loB) v[2] = 0;
            if (k + 1 > hiB || k + 1 < loB) v[3] = 0;
        };
#pragma unroll 1
        for (int q = 0; q < mine; ++q) {
            if (page_of(q) < 0) continue;
            const int kb = key_of(q), k0 = kb + 16 * tig;
            const bool clear = kb >= cmin && kb + 63 <= cmax;
            if (q == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    exps(t[j]);
                    if (!clear) mask(t[j], k0 + 2 * j);
                    sum[0] += (unsigned)(t[j][0] + t[j][1]);
                    sum[1] += (unsigned)(t[j][2] + t[j][3]);
                }
            } else {
#pragma unroll 4
                for (int j = 0; j < 8; ++j) {
                    const int4 s = store[256 * q + 32 * j];
                    int v[4] = {s.x, s.y, s.z, s.w};
                    exps(v);
                    if (!clear) mask(v, k0 + 2 * j);
                    sum[0] += (unsigned)(v[0] + v[1]);
                    sum[1] += (unsigned)(v[2] + v[3]);
                    store[256 * q + 32 * j] = make_int4(v[0], v[1], v[2], v[3]);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        }
        give(x_sum, (int)sum[0], (int)sum[1]);           // (the maxima are read before any warp gets past this)
        // ---- the rows' probabilities of each key, added over the lanes: lane gid ends with keys 2 gid, 2 gid + 1 of its 16
        unsigned RSa, RSb;
        int bla, blb;
        {
            unsigned m = 0;                              // at most 2^15 keys: below 2^30
            for (int e = lane >> 4; e < S * NW; e += 2) m += (unsigned)x_sum[e * WB_ROWS + (lane & 15)];
            m += __shfl_xor_sync(0xffffffffu, m, 16);
            const int bl = 32 - __clz(m);
            const unsigned RS = m ? (unsigned)pow2_recip(m, bl, 1, 23) : 0;
            RSa = __shfl_sync(0xffffffffu, RS, rA);
            RSb = __shfl_sync(0xffffffffu, RS, rB);
            bla = max(__shfl_sync(0xffffffffu, bl, rA), 2);
            blb = max(__shfl_sync(0xffffffffu, bl, rB), 2);
        }
#pragma unroll 1
        for (int q = 0; q < mine; ++q) {
            const int blk = page_of(q);
            if (blk < 0) continue;
            unsigned v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                int4 s = make_int4(t[j][0], t[j][1], t[j][2], t[j][3]);
                if (q) s = store[256 * q + 32 * j];
                v[2 * j] = kv4_p24s(s.x, RSa, bla) + kv4_p24s(s.z, RSb, blb);
                v[2 * j + 1] = kv4_p24s(s.y, RSa, bla) + kv4_p24s(s.w, RSb, blb);
            }
#pragma unroll
            for (int n = 8, o = 16; o >= 4; n >>= 1, o >>= 1) {
                const bool up = (lane & o) != 0;
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (h < n) {
                        const unsigned keep = up ? v[h + n] : v[h], give = up ? v[h] : v[h + n];
                        v[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
            }
            unsigned long long* w = (unsigned long long*)wg.weight + ((size_t)blk * a.n_kv + g) * KV_BLK + 16 * tig + 2 * gid;
            if (v[0]) atomicAdd(w, (unsigned long long)v[0]);
            if (v[1]) atomicAdd(w + 1, (unsigned long long)v[1]);
        }
    }
}

// ------------------------------------------------------------------ eviction
// The kept places of one sequence and kv head, ascending: the first `sinks`
// and last `recent` ones and, between them, those of the largest weights, the
// lower place first among equal ones. A cluster per sequence and kv head, a run
// of whole pages per CTA, the weights in shared memory as order-preserving
// keys. The least kept key is found in a histogram with 16 bins to an octave on
// either side of zero (attention weights are heavy-tailed: in even bins most
// would share one), whose few keys in the bin in question are then ranked by
// counting; where that bin is too full, its keys are split by 11 bits at a time
// first. Then every warp deals the kept places of its run out. Keys that are not
// held are read again in each pass: weights that another stream changes meanwhile
// give some choice, of fewer places perhaps, but every entry of the lists is written
// (-1 behind the last place) and nothing past them.
// Bound: latency of the phases, eight barriers of the cluster among them, so that
// three CTAs per SM (five of 256 threads) take turns: 16 sequences of 9000..32768
// keys, 8 kv heads, 36 us for 21 MB of weights (two CTAs per SM 38); 1 of 4097 11 us.
constexpr int EV_BITS = 11, EV_BINS = 1 << EV_BITS;
constexpr int EV_LIST = 512;             // keys that are ranked by counting
constexpr int EV_PAGES = EV_BINS / 4;    // pages of a CTA

struct Kv4Evict {
    long long* weight;
    const int32_t *seq, *lens;           // [n]
    const int32_t* new_table;            // [n][pages of keep]
    int32_t* kept;                       // [n][n_kv][keep]
    int max_len, keep, sinks, recent;
    int new_blocks;                      // pages of keep
    int lg_s;                            // log2 of the CTAs of a cluster
    int held;                            // the keys fit shared memory
};

__device__ __forceinline__ u64 ev_key(long long w) { return (u64)w ^ (1ull << 63); }
// octave bin of a key, the bits of a key that its bin leaves open, and the least key in it
__device__ __forceinline__ int ev_bin(u64 key) {
    const bool neg = !(key >> 63);
    const u64 v = neg ? ~key & ~(1ull << 63) : key & ~(1ull << 63);     // w, or -1 - w below zero
    const int e = bitlen_u64(v), b = e <= 4 ? (int)v : ((e - 4) << 4) + (int)(v >> (e - 5) & 15);
    return neg ? EV_BINS / 2 - 1 - b : EV_BINS / 2 + b;
}
__device__ __forceinline__ int ev_open(int bin) {
    const int b = bin < EV_BINS / 2 ? EV_BINS / 2 - 1 - bin : bin - EV_BINS / 2;
    return b < 16 ? 0 : (b >> 4) - 1;
}
__device__ __forceinline__ u64 ev_least(int bin) {
    const bool neg = bin < EV_BINS / 2;
    const int b = neg ? EV_BINS / 2 - 1 - bin : bin - EV_BINS / 2, open = ev_open(bin);
    const u64 v = b < 16 ? (u64)b : (u64)(16 + (b & 15)) << open;
    return neg ? (~v & ~(1ull << 63)) >> open << open : v | 1ull << 63;
}

template <int EV_THREADS>
__global__ void __launch_bounds__(EV_THREADS, EV_THREADS == 512 ? 3 : 5) k_kv4_evict_select(Kv4Args a, Kv4Evict p) {
    constexpr int EV_WARPS = EV_THREADS / 32;
    extern __shared__ __align__(16) unsigned char ev_raw[];
    u64* keys = (u64*)ev_raw;                            // the CTA's, where they are held
    __shared__ __align__(16) unsigned hist[EV_BINS];
    __shared__ u64 found;
    u64* const list = (u64*)hist;                        // (the bins are clear and done with when it is filled)
    __shared__ unsigned scan[2][EV_WARPS], mine[2], pick[3], count;
    __shared__ int page[EV_PAGES];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = 1 << p.lg_s, rank = (int)blockIdx.x & (S - 1), i = (int)blockIdx.x >> p.lg_s, g = blockIdx.y;
    const int seq = p.seq[i], max_len = min(p.max_len, min(a.max_blocks, 1 << 13) * KV_BLK);
    int len = p.lens[i];
    pdl_launch();
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
    // this CTA's pages
    const int all = (len + KV_BLK - 1) >> 6, per = (all + S - 1) >> p.lg_s;
    const int b0 = rank * per, nb = max(0, min(per, all - b0)), j0 = b0 << 6;
    for (int b = tid; b < nb; b += EV_THREADS) {
        int blk = a.block_table[(size_t)seq * a.max_blocks + b0 + b];
        if (blk < 0 || blk >= a.n_blocks) {
            blk = -1;
            if (a.status) a.status[ST_CTX] = 1;
        }
        page[b] = blk;
    }
    for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
    if (tid == 0) count = 0;
    __syncthreads();
    // a warp takes pages; a lane two neighbouring places of a page
    auto fetch = [&](int b) -> ulonglong2 {
        const int blk = page[b];
        if (blk < 0) return make_ulonglong2(ev_key(0), ev_key(0));
        const longlong2 w = *((const longlong2*)(p.weight + ((size_t)blk * a.n_kv + g) * KV_BLK) + lane);
        return make_ulonglong2(ev_key(w.x), ev_key(w.y));
    };
    auto each = [&](auto f) {                            // f(key) of every key that is weighed
        for (int b = warp; b < nb; b += EV_WARPS) {
            const ulonglong2 k = p.held ? *((const ulonglong2*)(keys + (b << 6)) + lane) : fetch(b);
            const int j = j0 + (b << 6) + 2 * lane;
            if (j >= lo && j < hi) f(k.x);
            if (j + 1 >= lo && j + 1 < hi) f(k.y);
        }
    };
    if (p.held) {
#pragma unroll 4
        for (int b = warp; b < nb; b += EV_WARPS) *((ulonglong2*)(keys + (b << 6)) + lane) = fetch(b);
        __syncwarp();                                    // (`each` gives a lane its own keys back)
    }
    cl_sync();                                           // the first CTA's bins are clear and may be added to
    // the want-th largest key: cut, whose `open` low bits are yet to be found
    int open = 64;
    u64 cut = 0;
    const bool any = want > 0;
    bool whole = !any;                                   // every key that agrees with cut's closed bits is kept
    if (!any) open = 0;
    while (open > 0 && !whole) {
        const int sh = max(open - EV_BITS, 0);
        const u64 agree = open >= 64 ? 0 : cut >> open, bins = (1ull << (open - sh)) - 1;
        each([&](u64 k) {
            if (open >= 64) atomicAdd(&hist[ev_bin(k)], 1u);
            else if (k >> open == agree) atomicAdd(&hist[(k >> sh) & bins], 1u);
        });
        __syncthreads();
        if (rank)                                        // the first CTA's bins become the cluster's
            for (int b = tid; b < EV_BINS; b += EV_THREADS)
                if (hist[b]) {
                    cl_red32(&hist[b], 0, hist[b]);
                    hist[b] = 0;
                }
        cl_sync();
        if (rank == 0) {
            // from the highest bin down: the bin in which `want` is reached
            constexpr int BPT = EV_BINS / EV_THREADS;
            unsigned c[BPT], sum = 0;
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                c[x] = hist[EV_BINS - 1 - (tid * BPT + x)];
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
#pragma unroll
                for (int x = 0; x < BPT; ++x) {
                    if (before < want && want <= before + c[x]) {
                        pick[0] = (unsigned)(EV_BINS - 1 - (tid * BPT + x));
                        pick[1] = want - before;         // of the bin's keys
                        pick[2] = c[x];
                    }
                    before += c[x];
                }
            }
            for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
        }
        cl_sync();
        const unsigned bin = cl_ld32u(&pick[0], 0), n = cl_ld32u(&pick[2], 0);
        want = cl_ld32u(&pick[1], 0);
        if (open >= 64) {
            open = ev_open((int)bin);
            cut = ev_least((int)bin);
        } else {
            cut = (agree << (open - sh) | bin) << sh;
            open = sh;
        }
        whole = want == n;
        if (!whole && open > 0 && n <= EV_LIST) {        // few: ranked by the first CTA
            const u64 near = cut >> open;
            each([&](u64 k) {
                if (k >> open == near) {
                    const unsigned to = cl_add32(&count, 0, 1);
                    if (to < EV_LIST) cl_st64(&list[to], 0, k);
                }
            });
            cl_sync();
            if (rank == 0) {
                for (int x = tid; x < (int)n; x += EV_THREADS) {
                    const u64 d = list[x];
                    unsigned above = 0, same = 0;
#pragma unroll 4
                    for (int y = 0; y < (int)n; ++y) {
                        above += list[y] > d;
                        same += list[y] == d;
                    }
                    if (above < want && want <= above + same) {      // (equal keys write the same)
                        found = d;
                        pick[1] = want - above;
                    }
                }
            }
            cl_sync();
            cut = (u64)cl_ld64((const i64*)&found, 0);
            want = cl_ld32u(&pick[1], 0);
            open = 0;
        }
        if (open > 0 && !whole) cl_sync();               // what was read is not written again before all have read it
    }
    // ---- kept: places outside [lo, hi), keys past the closed bits of cut (all that
    // agree with them too when whole), and the first `want` of those equal to it
    const u64 edge = cut >> open;
    const int bpw = (nb + EV_WARPS - 1) / EV_WARPS, w0 = min(nb, warp * bpw), w1 = min(nb, w0 + bpw);   // this warp's pages
    unsigned* mask = hist;                               // [page][half][kept, equal to the cut] of 32 places (the bins are done)
    unsigned take = 0, ties = 0;
    for (int b = w0; b < w1; ++b)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int x = 32 * hf + lane, j = j0 + (b << 6) + x;
            u64 k = ev_key(0);
            if (p.held) k = keys[(b << 6) + x];
            else if (page[b] >= 0) k = ev_key(p.weight[((size_t)page[b] * a.n_kv + g) * KV_BLK + x]);
            const u64 d = k >> open;
            const bool in = j >= lo && j < hi;
            const unsigned mk = __ballot_sync(0xffffffffu, j < len && (!in || (any && (d > edge || (whole && d == edge)))));
            const unsigned mt = __ballot_sync(0xffffffffu, in && !whole && d == edge);
            if (lane < 2) mask[4 * b + 2 * hf + lane] = lane ? mt : mk;
            take += __popc(mk);
            ties += __popc(mt);
        }
    if (lane == 0) { scan[0][warp] = take; scan[1][warp] = ties; }
    __syncthreads();
    unsigned bt = 0, be = 0, nt = 0, ne = 0;
    for (int w = 0; w < EV_WARPS; ++w) {
        if (w == warp) { bt = nt; be = ne; }
        nt += scan[0][w];
        ne += scan[1][w];
    }
    if (tid == 0) { mine[0] = nt; mine[1] = ne; }
    cl_sync();
    for (int r = 0; r < rank; ++r) {
        bt += cl_ld32u(&mine[0], r);
        be += cl_ld32u(&mine[1], r);
    }
    for (int b = w0; b < w1; ++b)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const unsigned mk = mask[4 * b + 2 * hf], mt = mask[4 * b + 2 * hf + 1], lt = (1u << lane) - 1;
            const unsigned e = be + __popc(mt & lt);
            const unsigned to = bt + __popc(mk & lt) + min(e, want);
            if (((mk >> lane & 1) || ((mt >> lane & 1) && e < want)) && to < (unsigned)p.keep) out[to] = j0 + (b << 6) + 32 * hf + lane;
            bt += __popc(mk);
            be += __popc(mt);
        }
    if (rank == S - 1 && warp == EV_WARPS - 1)           // behind the last place (nothing is left over unless weights changed meanwhile)
        for (unsigned j = bt + min(be, want) + lane; j < (unsigned)p.keep; j += 32) out[j] = -1;
    cl_sync();                                           // no CTA leaves while another reads its shared memory
}

// The kept tokens of 64 new places (a page of one kv head), a CTA each. Rows
// of keys, scale codes and weights are gathered. A thread of the values takes
// two channels that share 16 bytes of every 16 places of a page, and walks the
// kept places in order: one load for those that lie in the same 16, a nibble
// out of it for each, one store for 16 new places. Places behind the last kept
// token are left as they were. The new pages may not be among the sequences'
// own. Bound: memory, 62 us for those 16 sequences to 4099 keys each: 304 MB, most
// of them values of which a sector holds 32 places, at 5.1 TB/s.
constexpr int KV4_ZEROS = -0x77777778;   // eight codes of zero (8 each)
template <int D>
__global__ void __launch_bounds__(128) k_kv4_evict_move(Kv4Args a, Kv4Evict p) {
    constexpr int PW = D * KV_BLK / 8;                   // words of a page of values
    __shared__ int from[KV_BLK], page[KV_BLK];           // places in their pages, and those pages (-1: outside the pool)
    __shared__ int run[KV_BLK + 1], runs;                // first kept places of the same 16 places of a page
    __shared__ int2 move[KV_BLK];                        // shift of a place's code in its word (negative: the second of two); what brings it to its new one
    const int tid = threadIdx.x, b = blockIdx.x, g = blockIdx.y, i = blockIdx.z;
    const int seq = p.seq[i], to = p.new_table[(size_t)i * p.new_blocks + b];
    const int32_t* kept = p.kept + ((size_t)i * a.n_kv + g) * p.keep;
    pdl_wait();
    if (tid < KV_BLK) {
        const int s = b * KV_BLK + tid, j = s < p.keep ? __ldcg(kept + s) : -1;
        int blk = -1;
        const bool in = (unsigned)(j >> 6) < (unsigned)a.max_blocks;      // (none of a sequence out of range is kept)
        if (in) blk = a.block_table[(size_t)seq * a.max_blocks + (j >> 6)];
        from[tid] = in ? j & 63 : -1;
        page[tid] = blk >= 0 && blk < a.n_blocks ? blk : -1;
        move[tid] = make_int2((8 * (j & 3) + (j & 4)) | (j & 8 ? (int)0x80000000 : 0), 1 << (8 * (tid & 3) + (tid & 4)));
    }
    const int n = __syncthreads_count(tid < KV_BLK && from[tid & 63] >= 0);      // the kept ones come first
    if (!n) return;
    if (to < 0 || to >= a.n_blocks) {
        if (tid == 0 && a.status) a.status[ST_CTX] = 1;
        return;
    }
    const size_t u = (size_t)to * a.n_kv + g;
    if (tid < 32) {
        int at = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = 32 * h + tid;
            const bool lead = s < n && (s == 0 || page[s] != page[s - 1] || from[s] >> 4 != from[s - 1] >> 4);
            const unsigned m = __ballot_sync(0xffffffffu, lead);
            if (lead) run[at + __popc(m & ((1u << tid) - 1))] = s;
            at += __popc(m);
        }
        if (tid == 0) { runs = at; run[at] = n; }
    }
    __syncthreads();
    if (tid < D / 2) {
        // values: row tid of 16 words holds channels 16 (tid / 8) + tid % 8 and 8 more
        const int4* vin = (const int4*)(a.v + (size_t)g * PW * 4) + tid * 4;
        int4* vout = (int4*)(a.v + u * PW * 4) + tid * 4;
        auto load = [&](int r) -> int4 {
            const int s = run[r], blk = page[s];
            return blk >= 0 ? vin[(size_t)blk * a.n_kv * (PW / 4) + (from[s] >> 4)] : make_int4(KV4_ZEROS, KV4_ZEROS, KV4_ZEROS, KV4_ZEROS);
        };
        constexpr int AHEAD = 2;                         // (4 and 6 leave room for fewer CTAs: those 16 sequences 103 and 111 us in place of 98; 8 of 16384 40 and 39 in place of 42)
        int4 next[AHEAD];
#pragma unroll
        for (int r = 0; r < AHEAD; ++r)
            if (r < runs) next[r] = load(r);
        unsigned w0 = 0, w1 = 0, lo0 = 0, lo1 = 0;       // eight places of both channels; the eight before them
        for (int r0 = 0; r0 < runs; r0 += AHEAD) {
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                if (r0 + x >= runs) break;
                const int4 v = next[x];
                if (r0 + x + AHEAD < runs) next[x] = load(r0 + x + AHEAD);
                const int s1 = run[r0 + x + 1];
                for (int s = run[r0 + x]; s < s1; ++s) {
                    const int2 f = move[s];
                    const unsigned c0 = f.x < 0 ? v.y : v.x, c1 = f.x < 0 ? v.w : v.z;
                    w0 += (__funnelshift_r(c0, 0, f.x) & 15) * f.y;      // (the shift is taken mod 32)
                    w1 += (__funnelshift_r(c1, 0, f.x) & 15) * f.y;
                    if ((s & 7) == 7) {
                        if (s & 8) vout[s >> 4] = make_int4((int)lo0, (int)w0, (int)lo1, (int)w1);
                        lo0 = w0;
                        lo1 = w1;
                        w0 = w1 = 0;
                    }
                }
            }
        }
        if (n & 15) {                                    // the last 16 places are not all taken
            auto rest = [](int k) -> unsigned {          // nibbles of places k and up of a word of eight
                unsigned m = 0;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (x >= k) m |= 15u << (8 * (x & 3) + (x & 4));
                return m;
            };
            const int4 old = vout[n >> 4];
            const unsigned m0 = rest(n & 15), m1 = rest((n & 15) - 8);
            if (!(n & 8)) { lo0 = w0; lo1 = w1; w0 = w1 = 0; }
            vout[n >> 4] = make_int4((int)(lo0 | ((unsigned)old.x & m0)), (int)(w0 | ((unsigned)old.y & m1)),
                                     (int)(lo1 | ((unsigned)old.z & m0)), (int)(w1 | ((unsigned)old.w & m1)));
        }
        return;
    }
    // keys: rows of D / 2 bytes
    constexpr int V = D / 32, NK = 128 - D / 2;          // 16-byte pieces of a row; threads
    const int kt = tid - D / 2;
#pragma unroll 4
    for (int x = kt; x < n * V; x += NK) {
        const int s = x / V, c = x & (V - 1), blk = page[s];
        int4 v = make_int4(KV4_ZEROS, KV4_ZEROS, KV4_ZEROS, KV4_ZEROS);
        if (blk >= 0) v = *((const int4*)(a.k + (((size_t)blk * a.n_kv + g) * KV_BLK + from[s]) * (D / 2)) + c);
        *((int4*)(a.k + (u * KV_BLK + s) * (D / 2)) + c) = v;
    }
    if (kt < n) {
        const int blk = page[kt];
        const size_t o = ((size_t)max(blk, 0) * a.n_kv + g) * KV_BLK + max(from[kt], 0);
        const uint8_t ck = a.ks[o], cv = a.vs[o];
        const long long w = p.weight[o];
        a.ks[u * KV_BLK + kt] = blk >= 0 ? ck : 1;
        a.vs[u * KV_BLK + kt] = blk >= 0 ? cv : 1;
        p.weight[u * KV_BLK + kt] = blk >= 0 ? w : 0;
    }
}

// whole pages of every kv head, src[i] to dst[i]; -1 on either side: none. A CTA
// per page and head, 16 bytes per thread and step; latency of one page (128 pages
// of 8 heads of 128 with their weights 5 us).
__global__ void __launch_bounds__(256) k_kv4_copy(Kv4Args a, const int32_t* src, const int32_t* dst, int page_bytes, long long* weight) {
    pdl_wait();
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
