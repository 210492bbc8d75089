// The 4-bit paged key/value cache: append (QK-norm, rotation, quantisation,
// paged write), attention of single tokens and attention of token blocks.
//
// Cache format. A page holds 64 tokens of one kv head. A value is a 4-bit
// code q in -7..7, stored as q + 8, times the token's scale code c in 1..255
// (one byte per token and kv head): the cached integer is q c, |q c| <= 1785.
//   K page [64][D/2]: 32-bit word w of a token's row holds channels 8w..8w+7,
//     byte b with channel 8w+b in the low nibble and 8w+4+b in the high one,
//     so (word & 0x0f0f0f0f) and (word >> 4 & 0x0f0f0f0f) are four
//     consecutive channels each: dp4a and mma.sync operands.
//   V page [D/16][8][4][2][2] words: group of 16 channels, channel % 8,
//     key / 16, channel / 8 % 2, key / 8 % 2; a word holds 8 keys of one
//     channel in the same nibble order. A lane's 16-byte load is the
//     mma.sync fragment of two channels and two 32-key steps, and a warp's
//     load is 512 contiguous bytes.
//
// Attention of a query row over its keys (docs: section 16):
//   t_j = c_j sum q8 k4_j, T = max t, delta_j = rshr((t_j - T) m_q CSTM, sh),
//   E_j = min(32767, exp2q(delta_j)), W_j = rshr(E_j cv_j, 7) (16 bits),
//   num = sum W_j v4_j, o = one deferred division by sum E_j.
// The exponential is rounded against the row's maximum, so partial sums of
// other maxima cannot be rescaled exactly: the maximum is settled over all
// keys before the first probability is formed.
#pragma once
#include "kernels.h"
#include "ptx.cuh"
#include "int_device.cuh"

namespace detint {

constexpr int KV4_XMAX = 1785;             // 7 * 255
constexpr int KV4_NEG = -2147483647 - 1;   // score of a masked key

__device__ __forceinline__ int kv4_lo(int w) { return w & 0x0f0f0f0f; }
__device__ __forceinline__ int kv4_hi(int w) { return (int)((unsigned)w >> 4) & 0x0f0f0f0f; }

// ---------------------------------------------------------------- append
// LPH lanes hold one head, four consecutive channels each: 32 lanes for 128
// channels, 16 for 64 (two heads per warp).
// The two heads of a warp may be a query and a key, so every exchange names
// its own lanes only.
template <int LPH>
__device__ __forceinline__ unsigned seg_mask() {
    return LPH == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
}
template <int LPH>
__device__ __forceinline__ unsigned seg_max(unsigned v) {
    return __reduce_max_sync(seg_mask<LPH>(), v);
}
template <int LPH>
__device__ __forceinline__ u64 seg_sum64(u64 v) {
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) v += __shfl_xor_sync(seg_mask<LPH>(), v, o);
    return v;
}
__device__ __forceinline__ unsigned uabs32(int v) { return v < 0 ? 0u - (unsigned)v : (unsigned)v; }

// (page row or -1, offset in the page) of a token, -1 for a position or a
// table entry outside its range (recorded unless the position is negative)
__device__ __forceinline__ int kv4_slot(const Kv4Args& a, int seq, int pos, int* off) {
    *off = pos & (KV_BLK - 1);
    if (pos < 0) return -1;
    int blk = -1;
    if (seq >= 0 && seq < a.n_seq && (pos >> 6) < a.max_blocks) blk = a.block_table[(size_t)seq * a.max_blocks + (pos >> 6)];
    if (blk < 0 || blk >= a.n_blocks) {
        if (a.status) a.status[ST_CTX] = 1;
        return -1;
    }
    return blk;
}

// the scale code of a row of cached integers x and the four codes (+ 8) of
// this lane: c = max(1, ceil(max|x| / 7)), q = rshr(x R, b + 16) with
// R = floor(2^(b + 16) / c), b = bitlen(c); |x| / c <= 7, so no clamp
template <int LPH>
__device__ __forceinline__ int kv4_codes(const int (&x)[4], int (&q)[4]) {
    unsigned m = max(max(uabs32(x[0]), uabs32(x[1])), max(uabs32(x[2]), uabs32(x[3])));
    m = seg_max<LPH>(m);
    const int c = max(1, (int)((m + 6) / 7));
    const int b = 32 - __clz(c);
    const int R = (int)pow2_recip((u64)c, b, 1, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = rshr32(x[j] * R, b + 16) + 8;   // |x R| < 2^11 2^17
    return c;
}

// a warp's q or k heads of one token: norm, rotation, quantisation
template <int LPH>
__device__ void kv4_qk_head(const Kv4Args& a, const Kv4Append& p, int t, int slot, bool live) {
    constexpr int D = 4 * LPH;
    const int lane = threadIdx.x & (LPH - 1);
    const bool isq = slot < a.nq;
    const int kvh = isq ? (slot * a.gmul) >> 16 : slot - a.nq;
    const int pos = live ? p.tok_pos[t] : -1;
    const bool ok = pos >= 0 && pos < p.max_pos;
    if (live && pos >= p.max_pos && lane == 0 && a.status) a.status[ST_CTX] = 1;
    int y[4] = {0, 0, 0, 0};
    if (ok) {
        const int4 v = *(const int4*)(p.qkv + (size_t)t * p.qkv_stride + (size_t)slot * D + 4 * lane);
        y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
    }
    const int16_t* gamma = isq ? p.q_gamma : p.k_gamma;
    if (gamma) {
        const unsigned ax = seg_max<LPH>(max(max(uabs32(y[0]), uabs32(y[1])), max(uabs32(y[2]), uabs32(y[3]))));
        const int sig = (32 - __clz(ax)) - 24;
        int xp[4];
        u64 ss = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned u = uabs32(y[j]);
            const int m = (int)(sig >= 0 ? u >> sig : u << min(-sig, 31));
            xp[j] = y[j] < 0 ? -m : m;
            ss += (u64)((i64)xp[j] * xp[j]);
        }
        ss = seg_sum64<LPH>(ss);
        const i64 eps_s = !ax ? 0 : (sig >= 0 ? p.eps >> (2 * sig) : p.eps << (-2 * sig));   // eps < 2^15: < 2^61
        const u64 r = isqrt_fast((ss >> (LPH == 32 ? 7 : 6)) + (u64)eps_s);
        const int bl = bitlen_u64(r);
        const i64 Rr = ax ? (i64)pow2_recip(r, bl, 1, 23) : 0;
        const short4 gm = *(const short4*)(gamma + 4 * lane);
        const int g4[4] = {gm.x, gm.y, gm.z, gm.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = sat32(rshr((i64)xp[j] * g4[j] * Rr, bl + 21));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = sat32((i64)y[j] * 4);
    }
    // rotation of the first rot channels
    const int R2 = p.rot >> 1;
    if (p.inter) {
        if (4 * lane < p.rot) {
            short2 c = make_short2(0, 0), s = c;
            if (ok) {
                c = *(const short2*)(p.cos + (size_t)pos * R2 + 2 * lane);
                s = *(const short2*)(p.sin + (size_t)pos * R2 + 2 * lane);
            }
            const int a0 = y[0], a1 = y[1], a2 = y[2], a3 = y[3];
            y[0] = sat32(rshr((i64)a0 * c.x - (i64)a1 * s.x, 14));
            y[1] = sat32(rshr((i64)a1 * c.x + (i64)a0 * s.x, 14));
            y[2] = sat32(rshr((i64)a2 * c.y - (i64)a3 * s.y, 14));
            y[3] = sat32(rshr((i64)a3 * c.y + (i64)a2 * s.y, 14));
        }
    } else if (R2) {
        const int sh = R2 >> 2;                     // lanes between a pair's halves
        const bool first = lane < sh, in = lane < 2 * sh;
        const int src = (threadIdx.x & 31) + (first ? sh : (in ? -sh : 0));
        int z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = __shfl_sync(seg_mask<LPH>(), y[j], src);
        if (in) {
            short4 c = make_short4(0, 0, 0, 0), s = c;
            if (ok) {
                const int i0 = 4 * (first ? lane : lane - sh);
                c = *(const short4*)(p.cos + (size_t)pos * R2 + i0);
                s = *(const short4*)(p.sin + (size_t)pos * R2 + i0);
            }
            const int c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const i64 m = (i64)y[j] * c4[j], n = (i64)z[j] * s4[j];
                y[j] = sat32(rshr(first ? m - n : m + n, 14));
            }
        }
    }
    const int32_t* kvp = a.params + (size_t)kvh * (8 + D);
    const int4 ev = *(const int4*)(kvp + 8 + 4 * lane);
    const int e4[4] = {ev.x & 3, ev.y & 3, ev.z & 3, ev.w & 3};
    if (isq) {
        const int E = (int)seg_max<LPH>((unsigned)max(max(e4[0], e4[1]), max(e4[2], e4[3])));
        unsigned am = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = sat32((i64)y[j] << (E - e4[j]));
            am = max(am, uabs32(y[j]));
        }
        am = seg_max<LPH>(am);
        const int e = 32 - __clz(am);
        const i64 R = am ? (i64)pow2_recip(am, e, 127, 16) : 0;
        int q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = (int)rshr((i64)y[j] * R, e + 16);
        if (live) {
            const size_t qi = (size_t)t * a.nq + slot;
            *(char4*)(p.q8 + qi * D + 4 * lane) = make_char4((signed char)q[0], (signed char)q[1], (signed char)q[2], (signed char)q[3]);
            if (lane == 0) {
                int m = 0, k = 0;
                if (am) { dyadic_fast(am, 127ull, &m, &k); k += 14; }
                p.mq[qi] = m;
                p.kq[qi] = k;
            }
        }
    } else {
        int x[4], q[4];
        const i64 KQM = kvp[0];
        const int KQS = min(max(kvp[1], 0), 62);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = (int)sat_b(rshr((i64)y[j] * (KQM << e4[j]), KQS), KV4_XMAX);
        const int c = kv4_codes<LPH>(x, q);
        const int w4 = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        const int up = __shfl_down_sync(seg_mask<LPH>(), w4, 1);
        int off = 0, blk = -1;
        if (ok) blk = kv4_slot(a, p.tok_seq[t], pos, &off);
        if (blk >= 0) {
            const size_t row = ((size_t)blk * a.n_kv + kvh) * KV_BLK + off;
            if (!(lane & 1)) *(int*)(a.k + row * (D / 2) + 2 * lane) = w4 | (up << 4);
            if (lane == 0) a.ks[row] = (uint8_t)c;
        }
        if (live && p.k_val) {
            const size_t o = ((size_t)t * a.n_kv + kvh) * D + 4 * lane;
            *(short4*)(p.k_val + o) = blk < 0 ? make_short4(0, 0, 0, 0)
                : make_short4((short)((q[0] - 8) * c), (short)((q[1] - 8) * c), (short)((q[2] - 8) * c), (short)((q[3] - 8) * c));
        }
    }
}

// blockIdx.x is a tile of consecutive tokens. blockIdx.y below qk_blocks: one
// warp (half a warp for 64 channels) per q or k head, a token at a time;
// above: the values of one kv head, quantised a token at a time into shared
// memory and then written by words of 8 keys. A run of tokens that fills a
// word is one store; a shorter run changes its own nibbles with two atomics,
// so that another CTA's tokens in the same word are kept (the nibbles are
// distinct, so the order of the atomics does not matter).
constexpr int KV4_APT = 128;     // append threads
constexpr int KV4_VTILE = 64;    // most tokens in a tile

template <int LPH>
__global__ void __launch_bounds__(KV4_APT) k_kv4_append(Kv4Args a, Kv4Append p) {
    constexpr int D = 4 * LPH, HPW = 32 / LPH, HPB = (KV4_APT / 32) * HPW;
    const int warp = threadIdx.x >> 5;
    const int t0 = (int)blockIdx.x * p.tile, nt = min(p.tile, p.T - t0);
    if ((int)blockIdx.y < p.qk_blocks) {
        const int slot = (int)blockIdx.y * HPB + (int)(threadIdx.x / LPH);
        const bool live = slot < a.nq + a.n_kv;
        for (int i = 0; i < nt; ++i) kv4_qk_head<LPH>(a, p, t0 + i, live ? slot : 0, live);
        return;
    }
    __shared__ uint8_t codes[KV4_VTILE][D];
    __shared__ int page[KV4_VTILE], offs[KV4_VTILE];
    const int g = (int)blockIdx.y - p.qk_blocks;
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    const i64 VQM = kvp[2];
    const int VQS = min(max(kvp[3], 0), 62);
    for (int i0 = warp * HPW; i0 < nt; i0 += HPB) {
        const int i = i0 + (int)((threadIdx.x & 31) / LPH), lane = threadIdx.x & (LPH - 1);
        const bool live = i < nt;
        const int t = t0 + (live ? i : 0);
        const int pos = live ? p.tok_pos[t] : -1;
        int off = 0, blk = -1;
        if (pos >= 0 && pos < p.max_pos) blk = kv4_slot(a, p.tok_seq[t], pos, &off);
        int x[4] = {0, 0, 0, 0}, q[4];
        if (blk >= 0) {
            const int4 v = *(const int4*)(p.qkv + (size_t)t * p.qkv_stride + (size_t)(a.nq + a.n_kv + g) * D + 4 * lane);
            const int v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = (int)sat_b(rshr((i64)v4[j] * VQM, VQS), KV4_XMAX);
        }
        const int c = kv4_codes<LPH>(x, q);
        if (live) {
            *(int*)&codes[i][4 * lane] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
            if (lane == 0) {
                page[i] = blk;
                offs[i] = off;
                if (blk >= 0) a.vs[((size_t)blk * a.n_kv + g) * KV_BLK + off] = (uint8_t)c;
            }
            if (p.v_val)
                *(short4*)(p.v_val + ((size_t)t * a.n_kv + g) * D + 4 * lane) = blk < 0 ? make_short4(0, 0, 0, 0)
                    : make_short4((short)((q[0] - 8) * c), (short)((q[1] - 8) * c), (short)((q[2] - 8) * c), (short)((q[3] - 8) * c));
        }
    }
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
        const int blk = page[i], off = offs[i];
        if (blk < 0) continue;
        // a run starts where the word changes or the positions stop ascending
        if (i > 0 && page[i - 1] == blk && (offs[i - 1] >> 3) == (off >> 3) && offs[i - 1] < off) continue;
        uint32_t* vp = (uint32_t*)(a.v + ((size_t)blk * a.n_kv + g) * (D * KV_BLK / 2));
        for (int ch = threadIdx.x; ch < D; ch += KV4_APT) {
            unsigned w = 0, mask = 0;
            int last = -1;
            for (int j = i; j < nt && page[j] == blk && (offs[j] >> 3) == (off >> 3) && offs[j] > last; ++j) {
                last = offs[j];
                const int sh = 8 * (last & 3) + (last & 4);
                w |= (unsigned)codes[j][ch] << sh;
                mask |= 15u << sh;
            }
            uint32_t* d = vp + (ch >> 4) * 128 + (ch & 7) * 16 + (off >> 4) * 4 + ((ch >> 3) & 1) * 2 + ((off >> 3) & 1);
            if (mask == 0xffffffffu) {
                *d = w;
            } else {
                atomicAnd(d, ~mask);
                atomicOr(d, w);
            }
        }
    }
}

// ------------------------------------------------------------ attention
// What a query row's scores become: E = exp2q(rshr((t - T) M, sh)). Below
// t - T = dmin the result is zero, and clamping there keeps the shifted
// product in 32 bits: |dmin M| < (24577 << sh) + M.
struct Kv4Row {
    int M, sh, dmin;
    unsigned rlo;      // 2^(sh - 1), the rounding constant
    unsigned rhi;
};
__device__ __forceinline__ Kv4Row kv4_row(int mq, int kq, int cstm, int cstk) {
    Kv4Row r;
    const i64 M = (i64)mq * cstm;                       // <= 2^30 for dyadic mantissas
    r.M = (int)min(max(M, 0ll), 2147483647ll);
    r.sh = min(max(kq + cstk - 10, 0), 62);
    r.dmin = -(1 << 28);                                // |t - T| < 2^27
    if (r.M > 0 && r.sh < 44) {
        const u64 n = 24577ull << r.sh;
        if (n < ((u64)r.M << 28)) r.dmin = -(int)udiv_small(n, (u64)r.M) - 1;
    }
    const u64 h = r.sh ? 1ull << (r.sh - 1) : 0;
    r.rlo = (unsigned)h;
    r.rhi = (unsigned)(h >> 32);
    return r;
}
// 15-bit probability of score t against the row maximum T
__device__ __forceinline__ int kv4_E(const Kv4Row& r, int t, int T) {
    const int d = max(t - T, r.dmin);
    const i64 p = (i64)d * r.M + (i64)(((u64)r.rhi << 32) | r.rlo);
    const unsigned lo = (unsigned)p, hi = (unsigned)((u64)p >> 32);
    const bool far = r.sh >= 32;
    const int delta = (int)__funnelshift_r(far ? hi : lo, far ? (unsigned)((int)hi >> 31) : hi, r.sh & 31);
    const int n = -(delta >> 10);
    const int f = delta & 1023;
    const int inner = 7419 + ((2562 * f + 512) >> 10);
    const int mid = 22787 + ((f * inner + 512) >> 10);
    const int p2 = 32768 + ((f * mid + 512) >> 10);
    const int ns = min(n, 24);
    const int e = (p2 + ((1 << ns) >> 1)) >> ns;
    return n >= 24 ? 0 : min(e, 32767);
}
__device__ __forceinline__ int kv4_W(int E, int cv) { return (E * cv + 64) >> 7; }   // < 2^16

__device__ __forceinline__ void mma_u8u8(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8u8(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the output of one channel from the row's sums
__device__ __forceinline__ int kv4_out(i64 num, i64 RS, int bl, i64 MV, int KVS) {
    return sat32(rshr(rshr(num * RS, bl + 7) * MV, min(max(KVS + 4, 0), 62)));
}

// ------------------------------------------- attention of single tokens
// One unit is a token, a kv head and up to GT of its q heads; its keys are
// split by pages over S CTAs, which keep their scores in shared memory and
// settle the maximum, and later the sums, among themselves: as one
// thread-block cluster (S <= 16, distributed shared memory), or as CTAs of a
// cooperative launch through a workspace.
//   scores: a lane holds 32 channels of a key (one 16-byte load) and the
//     matching 8 words of every q head in registers; dp4a, then a
//     reduce-scatter over the key's lanes leaves each lane its own heads;
//   probabilities: four keys of a head per thread, split into the two bytes
//     of W, tiles of 8 pages in shared memory;
//   P V: mma.sync, V^T codes as the 16-row operand and the bytes of W as its
//     columns 2 h + limb; a warp owns 16 channels, so nothing is reduced
//     between warps at 128 channels.
// dp4a and mma.sync run on different pipes (a loop of one does not slow the
// other), so the two products overlap between the CTAs of an SM.
constexpr int KV4_DT = 256;      // decode threads
constexpr int KV4_TP = 8;        // pages per probability tile

template <int GT>
struct Kv4DecSm {
    uint32_t wp[2][KV4_TP][2 * GT][16];
    int red[8][GT];
    int cmax[GT];
    int tmax[GT];
    unsigned se[8][GT], sw[8][GT];
    unsigned csum[2][GT];
    i64 tot[3][GT];              // RS, bl, -8 sum W
    Kv4Row row[GT];
};

__device__ __forceinline__ unsigned cl_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cl_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cl_addr(const void* p, unsigned rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ int cl_ld32(const int* p, unsigned rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cl_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ i64 cl_ld64(const i64* p, unsigned rank) {
    i64 v;
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(cl_addr(p, rank)) : "memory");
    return v;
}

// all S CTAs of a unit of a cooperative launch; false when the bounded wait
// ran out (recorded; the results are then invalid)
__device__ __forceinline__ bool kv4_unit_barrier(unsigned* cnt, unsigned target, bool alive, int32_t* status) {
    __shared__ int s_ok;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(cnt, 1u);
        bool ok = false;
        if (alive)
            for (int i = 0; i < (1 << 20) && !ok; ++i) ok = *(volatile unsigned*)cnt >= target;
        if (!ok && status) status[ST_TIMEOUT] = 1;
        __threadfence();
        s_ok = ok;
    }
    __syncthreads();
    return s_ok != 0;
}

template <int D, int GT, bool GRID>
__global__ void __launch_bounds__(KV4_DT, 2) k_kv4_decode(Kv4Args a, Kv4Attn p) {
    constexpr int LPK = D / 32, KPL = 32 / LPK, UK = 4 * KPL, UPP = KV_BLK / UK;
    constexpr int HPL = GT >= LPK ? GT / LPK : 1;
    constexpr int NG = D / 16, WPG = 8 / NG, NV = KV4_TP / WPG;
    constexpr int NT = (2 * GT + 7) / 8, NPASS = (GT + 1) / 2;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ Kv4DecSm<GT> sm;
    i64* num_s = (i64*)kv4_raw;                       // [GT][D]
    int* pg = (int*)(num_s + GT * D);                 // [cap / 64]
    const int pitch = p.cap + 8;                      // 8 banks between heads
    int* ts = pg + (((p.cap >> 6) + 3) & ~3);         // [GT][pitch]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.z + p.t0;
    const unsigned rank = blockIdx.x, S = gridDim.x;
    int g = blockIdx.y, hg = 0;
    while (g >= a.n_kv) { g -= a.n_kv; ++hg; }
    const int nh = min(GT, p.G - hg * GT), h0 = g * p.G + hg * GT;
    const int pos = p.tok_pos[t], seq = p.tok_seq[t];
    int32_t* orow = p.o + (size_t)t * p.o_stride + (size_t)h0 * D;
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (pos < 0 || pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks) {
        // no key: a zero row (the whole unit takes this way out)
        if (rank == 0) {
            for (int i = tid; i < nh * D; i += KV4_DT) orow[i] = 0;
            if (pos >= 0 && tid == 0 && a.status) a.status[ST_CTX] = 1;
        }
        return;
    }
    const int j1 = pos + 1, j0 = p.window > 0 ? max(0, j1 - p.window) : 0;
    const int b0 = j0 >> 6, nb = ((j1 + 63) >> 6) - b0;
    const int per = (int)(((u64)(nb + (int)S - 1) * p.smul) >> 32);     // ceil(nb / S)
    const int pg0 = b0 + (int)rank * per, np = max(0, min(per, b0 + nb - pg0));
    // this CTA's pages
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
    const int sub = lane & (LPK - 1), kl = lane / LPK;
    int qw[GT][8], qoff[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) {
        int4 u = make_int4(0, 0, 0, 0), v = u;
        if (h < nh) {
            const int4* qp = (const int4*)(p.q8 + ((size_t)t * a.nq + h0 + h) * D + sub * 32);
            u = qp[0];
            v = qp[1];
        }
        qw[h][0] = u.x; qw[h][1] = u.y; qw[h][2] = u.z; qw[h][3] = u.w;
        qw[h][4] = v.x; qw[h][5] = v.y; qw[h][6] = v.z; qw[h][7] = v.w;
        int sq = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __dp4a(qw[h][j], 0x01010101, sq);
        qoff[h] = -8 * sq;                             // the codes are values + 8
    }
    __syncthreads();

    // ---- scores
    int tm[HPL];
#pragma unroll
    for (int x = 0; x < HPL; ++x) tm[x] = KV4_NEG;
    const int hb = GT >= LPK ? sub * HPL : (sub * GT) / LPK;
    const bool writer = GT >= LPK || (sub & (LPK / GT - 1)) == 0;
    const int nu = np * UPP;
    auto load = [&](int u, int4 (&w)[4], int& blk) {
        blk = -1;
        if (u < nu) blk = pg[u / UPP];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_int4(0, 0, 0, 0);
        if (blk < 0) return;
        const uint8_t* base = a.k + (((size_t)blk * a.n_kv + g) * KV_BLK + (u & (UPP - 1)) * UK + kl) * (D / 2) + sub * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg((const int4*)(base + (size_t)i * KPL * (D / 2)));
    };
    int4 cur[4];
    int cblk;
    load(warp, cur, cblk);
    for (int u = warp; u < nu; u += 8) {
        int4 nxt[4];
        int nblk;
        load(u + 8, nxt, nblk);
        const uint8_t* ckp = a.ks + ((size_t)max(cblk, 0) * a.n_kv + g) * KV_BLK + (u & (UPP - 1)) * UK + kl;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ck = __ldg(ckp + i * KPL);
            int acc[GT];
#pragma unroll
            for (int h = 0; h < GT; ++h) acc[h] = qoff[h];
            const int w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int lo = kv4_lo(w[x]), hi = kv4_hi(w[x]);
#pragma unroll
                for (int h = 0; h < GT; ++h) acc[h] = __dp4a(lo, qw[h][2 * x], acc[h]);
#pragma unroll
                for (int h = 0; h < GT; ++h) acc[h] = __dp4a(hi, qw[h][2 * x + 1], acc[h]);
            }
            // reduce over the key's lanes; each keeps HPL heads where it can
            int n = GT;
#pragma unroll
            for (int o = LPK / 2; o; o >>= 1) {
                if (n > 1) {
                    n >>= 1;
#pragma unroll
                    for (int h = 0; h < GT / 2; ++h)
                        if (h < n) {
                            const bool upper = (sub & o) != 0;
                            const int keep = upper ? acc[h + n] : acc[h];
                            const int give = upper ? acc[h] : acc[h + n];
                            acc[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                } else {
                    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
                }
            }
            const int key = u * UK + i * KPL + kl;
            const int j = (pg0 << 6) + key;
            const bool in = cblk >= 0 && j >= j0 && j < j1;
#pragma unroll
            for (int x = 0; x < HPL; ++x) {
                const int tv = in ? acc[x] * ck : KV4_NEG;
                tm[x] = max(tm[x], tv);
                if (writer) ts[(hb + x) * pitch + key] = tv;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
        cblk = nblk;
    }
#pragma unroll
    for (int x = 0; x < HPL; ++x) {
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) tm[x] = max(tm[x], __shfl_xor_sync(0xffffffffu, tm[x], o));
        if (lane < LPK && writer) sm.red[warp][hb + x] = tm[x];
    }
    __syncthreads();
    // ---- the maximum over every CTA of the unit
    const int unit = (blockIdx.z * gridDim.y + blockIdx.y);
    unsigned* cnt = GRID ? p.ws_cnt + unit : nullptr;
    bool alive = true;
    if (tid < GT) {
        int m = sm.red[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, sm.red[w][tid]);
        sm.cmax[tid] = m;
        if (GRID) p.ws_max[((size_t)unit * S + rank) * GT + tid] = m;
    }
    if (GRID) alive = kv4_unit_barrier(cnt, S, alive, a.status);
    else if (S > 1) cl_sync();
    else __syncthreads();
    if (warp == 0) {
        for (int h = 0; h < GT; ++h) {
            int m = KV4_NEG;
            for (unsigned r = lane; r < S; r += 32)
                m = max(m, GRID ? __ldcg(p.ws_max + ((size_t)unit * S + r) * GT + h)
                                : (S > 1 ? cl_ld32(&sm.cmax[h], r) : sm.cmax[h]));
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) sm.tmax[h] = m;
        }
    }
    __syncthreads();

    // ---- probabilities and P V, tiles of KV4_TP pages
    const int cg = warp & (NG - 1), ph = warp / NG;
    const int gid = lane >> 2, tig = lane & 3;
    int acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
    unsigned sumE[NPASS], sumW[NPASS];
#pragma unroll
    for (int x = 0; x < NPASS; ++x) sumE[x] = sumW[x] = 0;
    int buf = 0;
    for (int p0 = 0; p0 < np; p0 += KV4_TP, buf ^= 1) {
        int4 vv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int pi = p0 + i * WPG + ph;
            const int blk = pi < np ? pg[pi] : -1;
            vv[i] = make_int4(0, 0, 0, 0);
            if (blk >= 0)
                vv[i] = __ldg((const int4*)(a.v + ((size_t)blk * a.n_kv + g) * (D * KV_BLK / 2) + cg * 512) + lane);
        }
        {
            const int qd = tid & 127, pi = p0 + (qd >> 4);
            const int blk = pi < np ? pg[pi] : -1;
            const uint32_t cvw = blk >= 0 ? __ldg((const uint32_t*)(a.vs + ((size_t)blk * a.n_kv + g) * KV_BLK) + (qd & 15)) : 0;
#pragma unroll
            for (int x = 0; x < NPASS; ++x) {
                const int h = 2 * x + (tid >> 7);
                if (h < GT) {
                    int w[4] = {0, 0, 0, 0};
                    if (blk >= 0) {
                        const Kv4Row rw = sm.row[h];
                        const int T = sm.tmax[h];
                        const int4 tv = *(const int4*)(ts + h * pitch + p0 * KV_BLK + qd * 4);
                        const int t4[4] = {tv.x, tv.y, tv.z, tv.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int E = t4[k] == KV4_NEG ? 0 : kv4_E(rw, t4[k], T);
                            w[k] = kv4_W(E, (int)(cvw >> (8 * k)) & 255);
                            sumE[x] += E;
                            sumW[x] += w[k];
                        }
                    }
                    const unsigned wa = (unsigned)w[0] | ((unsigned)w[1] << 16), wb = (unsigned)w[2] | ((unsigned)w[3] << 16);
                    sm.wp[buf][qd >> 4][2 * h][qd & 15] = __byte_perm(wa, wb, 0x6420);
                    sm.wp[buf][qd >> 4][2 * h + 1][qd & 15] = __byte_perm(wa, wb, 0x7531);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int pt = i * WPG + ph;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                int4 b = make_int4(0, 0, 0, 0);
                if (8 * n + gid < 2 * GT) b = *(const int4*)&sm.wp[buf][pt][8 * n + gid][4 * tig];
                mma_u8u8(acc[n], kv4_lo(vv[i].x), kv4_lo(vv[i].z), kv4_hi(vv[i].x), kv4_hi(vv[i].z), b.x, b.y);
                mma_u8u8(acc[n], kv4_lo(vv[i].y), kv4_lo(vv[i].w), kv4_hi(vv[i].y), kv4_hi(vv[i].w), b.z, b.w);
            }
        }
    }
    // ---- this CTA's sums: numerators [GT][D], sum E and sum W per head
#pragma unroll
    for (int x = 0; x < NPASS; ++x) {
        const int h = 2 * x + (tid >> 7);
        const unsigned e = __reduce_add_sync(0xffffffffu, sumE[x]), w = __reduce_add_sync(0xffffffffu, sumW[x]);
        if (lane == 0 && h < GT) { sm.se[warp][h] = e; sm.sw[warp][h] = w; }
    }
#pragma unroll
    for (int part = 0; part < WPG; ++part) {
        if (ph == part) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int h = 4 * n + tig;
                if (h < GT) {
                    i64* d0 = num_s + h * D + cg * 16 + gid;
                    const i64 v0 = (i64)acc[n][0] + (i64)acc[n][1] * 256, v1 = (i64)acc[n][2] + (i64)acc[n][3] * 256;
                    d0[0] = part ? d0[0] + v0 : v0;
                    d0[8] = part ? d0[8] + v1 : v1;
                }
            }
        }
        __syncthreads();
    }
    if (tid < GT) {
        unsigned e = 0, w = 0;
        const int wbase = (tid & 1) * 4;               // head h = 2 x + (warp >= 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) { e += sm.se[wbase + k][tid]; w += sm.sw[wbase + k][tid]; }
        sm.csum[0][tid] = e;
        sm.csum[1][tid] = w;
        if (GRID) {
            p.ws_sum[(((size_t)unit * S + rank) * GT + tid) * 2] = e;
            p.ws_sum[(((size_t)unit * S + rank) * GT + tid) * 2 + 1] = w;
        }
    }
    if (GRID)
        for (int i = tid; i < GT * D; i += KV4_DT) p.ws_num[((size_t)unit * S + rank) * (GT * D) + i] = num_s[i];
    if (GRID) kv4_unit_barrier(cnt, 2 * S, alive, a.status);
    else if (S > 1) cl_sync();
    else __syncthreads();
    // ---- the row sums, then this CTA's share of the outputs
    if (warp < GT) {
        for (int h = warp; h < GT; h += 8) {
            u64 e = 0, w = 0;
            for (unsigned r = lane; r < S; r += 32) {
                if (GRID) {
                    e += __ldcg(p.ws_sum + (((size_t)unit * S + r) * GT + h) * 2);
                    w += __ldcg(p.ws_sum + (((size_t)unit * S + r) * GT + h) * 2 + 1);
                } else {
                    e += (unsigned)(S > 1 ? cl_ld32((const int*)&sm.csum[0][h], r) : (int)sm.csum[0][h]);
                    w += (unsigned)(S > 1 ? cl_ld32((const int*)&sm.csum[1][h], r) : (int)sm.csum[1][h]);
                }
            }
            e = redux_sum_u64(e);
            w = redux_sum_u64(w);
            if (lane == 0) {
                const int bl = bitlen_u64(e);
                sm.tot[0][h] = e ? (i64)pow2_recip(e, bl, 1, 23) : 0;
                sm.tot[1][h] = bl;
                sm.tot[2][h] = -8 * (i64)w;
            }
        }
    }
    __syncthreads();
    const i64 MV = kvp[4];
    const int KVS = kvp[5];
    const int n_out = nh * D;
    for (int i = (int)rank * KV4_DT + tid; i < n_out; i += (int)S * KV4_DT) {
        const int h = i / D;
        i64 num = sm.tot[2][h];
        for (unsigned r = 0; r < S; ++r)
            num += GRID ? __ldcg(p.ws_num + ((size_t)unit * S + r) * (GT * D) + i) : (S > 1 ? cl_ld64(num_s + i, r) : num_s[i]);
        orow[i] = kv4_out(num, sm.tot[0][h], (int)sm.tot[1][h], MV, KVS);
    }
    if (!GRID && S > 1) cl_sync();      // no CTA leaves while another reads its shared memory
}

// -------------------------------------------- attention of token blocks
// A CTA takes 64 query rows (64 / Gp consecutive tokens times the G q heads of
// one kv head, Gp the power of two >= G) and sweeps its keys twice, as the
// maximum has to be known first: sweep 1 scores and maxima, sweep 2 scores,
// probabilities and P V. A warp owns 16 rows, all 64 keys of a page and all
// channels. Column n of score tile j is key 16 (n / 2) + 2 j + (n & 1), so
// that the scores a lane holds are the keys of its own P V operand: the
// probabilities never leave the registers. The tokens of a block may belong
// to several sequences: each run of one sequence is swept by itself with the
// other rows masked.
constexpr int KV4_PT = 128;      // prefill threads
constexpr int KV4_PROWS = 64;
constexpr int KV4_PST = 4;       // page stages

template <int D>
struct Kv4Pf {
    static constexpr int PG = KV_BLK * D / 2;            // bytes of a K or V page
    static constexpr int STAGE = 2 * PG + 2 * KV_BLK;    // K, V, key scales, value scales
    static constexpr int SMEM = KV4_PST * STAGE;
};

template <int D>
__global__ void __launch_bounds__(KV4_PT, 2) k_kv4_prefill(Kv4Args a, Kv4Attn p) {
    using C = Kv4Pf<D>;
    constexpr int KS = D / 32, NC = D / 16;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ unsigned long long full[KV4_PST];
    __shared__ int page_ok[KV4_PST];
    __shared__ int r_pos[KV4_PROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, tig = lane & 3;
    const int g = blockIdx.x;
    const int lgBQ = 6 - p.lgGp, BQ = 1 << lgBQ;
    const int t0 = p.t0 + (int)(gridDim.y - 1 - blockIdx.y) * BQ;    // later tokens tend to have more keys
    const int nt = min(BQ, p.T - t0);
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (tid == 0) {
        for (int s = 0; s < KV4_PST; ++s) mbar_init(smem_u32(&full[s]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // row r: token t0 + (r >> lgGp), q head r & (Gp - 1)
    const int rA = warp * 16 + gid, rB = rA + 8;
    if (tid < KV4_PROWS) {
        const int i = tid >> p.lgGp, hh = tid & ((1 << p.lgGp) - 1);
        int pos = -1;
        if (i < nt && hh < p.G) {
            pos = p.tok_pos[t0 + i];
            const int seq = p.tok_seq[t0 + i];
            if (pos >= 0 && (pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks)) {
                pos = -1;
                if (a.status) a.status[ST_CTX] = 1;
            }
        }
        r_pos[tid] = pos;
    }
    __syncthreads();
    Kv4Row rw[2];
    int T[2] = {KV4_NEG, KV4_NEG};
    int qf[KS][4], qo[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = x ? rB : rA;
        const int i = r >> p.lgGp, hh = r & ((1 << p.lgGp) - 1);
        int w[2 * KS];
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j) w[j] = 0;
        int mq = 0, kq = 0;
        if (i < nt && hh < p.G) {
            const size_t qi = (size_t)(t0 + i) * a.nq + g * p.G + hh;
            const int* qp = (const int*)(p.q8 + qi * D + tig * (D / 4));
#pragma unroll
            for (int j = 0; j < 2 * KS; ++j) w[j] = qp[j];
            mq = p.mq[qi];
            kq = p.kq[qi];
        }
        rw[x] = kv4_row(mq, kq, kvp[6], kvp[7]);
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
    int aL[2 * NC][4], aH[2 * NC][4];
#pragma unroll
    for (int n = 0; n < 2 * NC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) aL[n][e] = aH[n][e] = 0;
    i64 sumE[2] = {0, 0}, sumW[2] = {0, 0};

    int it = 0;                                          // pages consumed so far (ring position)
    for (int s0 = 0; s0 < nt;) {
        // a run of one sequence: tokens [s0, s1)
        const int seq = p.tok_seq[t0 + s0];
        int s1 = s0 + 1;
        while (s1 < nt && p.tok_seq[t0 + s1] == seq) ++s1;
        int kmax = -1, kmin = 0x7fffffff;
        for (int i = s0; i < s1; ++i) {
            const int pos = r_pos[i << p.lgGp];
            if (pos < 0) continue;
            kmax = max(kmax, pos);
            kmin = min(kmin, p.window > 0 ? max(0, pos + 1 - p.window) : 0);
        }
        const int iA = rA >> p.lgGp, iB = rB >> p.lgGp;
        const int hiA = iA >= s0 && iA < s1 ? r_pos[rA] : -1, hiB = iB >= s0 && iB < s1 ? r_pos[rB] : -1;
        const int loA = p.window > 0 ? max(0, hiA + 1 - p.window) : 0, loB = p.window > 0 ? max(0, hiB + 1 - p.window) : 0;
        // keys of this warp's rows, and the keys that every one of them takes
        const int wmax = __reduce_max_sync(0xffffffffu, max(hiA, hiB));
        const int wmin = __reduce_min_sync(0xffffffffu, min(hiA >= 0 ? loA : 0x7fffffff, hiB >= 0 ? loB : 0x7fffffff));
        const int cmax = __reduce_min_sync(0xffffffffu, min(hiA, hiB));
        const int cmin = __reduce_max_sync(0xffffffffu, max(loA, loB));
        s0 = s1;
        if (kmax < 0) continue;
        const int p0 = kmin >> 6, np = (kmax >> 6) - p0 + 1;
        const int32_t* bt = a.block_table + (size_t)seq * a.max_blocks + p0;
        auto issue = [&](int i) {                        // i: page of the two sweeps, 0 .. 2 np - 1
            const int st = (it + i) & (KV4_PST - 1), sweep = i >= np;
            int blk = bt[sweep ? i - np : i];
            const uint32_t bar = smem_u32(&full[st]);
            if (blk < 0 || blk >= a.n_blocks) {
                page_ok[st] = 0;
                if (a.status) a.status[ST_CTX] = 1;
                mbar_arrive(bar);
                return;
            }
            page_ok[st] = 1;
            const size_t u = (size_t)blk * a.n_kv + g;
            const uint32_t dst = smem_u32(kv4_raw + st * C::STAGE);
            mbar_arrive_expect_tx(bar, sweep ? C::STAGE : C::PG + KV_BLK);
            bulk_g2s(dst, a.k + u * C::PG, C::PG, bar);
            bulk_g2s(dst + 2 * C::PG, a.ks + u * KV_BLK, KV_BLK, bar);
            if (sweep) {
                bulk_g2s(dst + C::PG, a.v + u * C::PG, C::PG, bar);
                bulk_g2s(dst + 2 * C::PG + KV_BLK, a.vs + u * KV_BLK, KV_BLK, bar);
            }
        };
        if (tid == 0)
            for (int i = 0; i < min(KV4_PST, 2 * np); ++i) issue(i);
        for (int i = 0; i < 2 * np; ++i) {
            const int st = (it + i) & (KV4_PST - 1);
            if (!mbar_wait(smem_u32(&full[st]), ((it + i) / KV4_PST) & 1) && a.status) a.status[ST_TIMEOUT] = 1;
            const int kb = (p0 + (i >= np ? i - np : i)) << 6;
            if (page_ok[st] && kb <= wmax && kb + 63 >= wmin) {
                const unsigned char* base = kv4_raw + st * C::STAGE;
                int S[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    S[j][0] = S[j][1] = qo[0];
                    S[j][2] = S[j][3] = qo[1];
                    const unsigned char* kr = base + (16 * (gid >> 1) + 2 * j + (gid & 1)) * (D / 2) + tig * (D / 8);
                    int w[KS];
                    if (D == 128) {
                        const int4 v = *(const int4*)kr;
                        w[0] = v.x; w[1] = v.y; w[KS - 2] = v.z; w[KS - 1] = v.w;
                    } else {
                        const int2 v = *(const int2*)kr;
                        w[0] = v.x; w[1] = v.y;
                    }
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        mma_s8u8(S[j], qf[s][0], qf[s][1], qf[s][2], qf[s][3], kv4_lo(w[s]), kv4_hi(w[s]));
                }
                const uint4 ckv = *(const uint4*)(base + 2 * C::PG + 16 * tig);
                const unsigned ck[4] = {ckv.x, ckv.y, ckv.z, ckv.w};
                const bool clear = kb >= cmin && kb + 63 <= cmax;      // no key of the page is masked
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = (int)(ck[j >> 1] >> (8 * ((2 * j + e) & 3))) & 255;
                        const int key = kb + 16 * tig + 2 * j + e;
                        const bool inA = clear || (key <= hiA && key >= loA), inB = clear || (key <= hiB && key >= loB);
                        S[j][e] = inA ? S[j][e] * c : KV4_NEG;
                        S[j][2 + e] = inB ? S[j][2 + e] * c : KV4_NEG;
                    }
                }
                if (i < np) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        T[0] = max(T[0], max(S[j][0], S[j][1]));
                        T[1] = max(T[1], max(S[j][2], S[j][3]));
                    }
                } else {
                    const uint4 cvv = *(const uint4*)(base + 2 * C::PG + KV_BLK + 16 * tig);
                    const unsigned cv[4] = {cvv.x, cvv.y, cvv.z, cvv.w};
                    int wl[2][4], wh[2][4];              // [row][4 keys]
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        int te = 0, tw = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            int w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int s = S[2 * k + (e >> 1)][2 * x + (e & 1)];
                                const int E = s == KV4_NEG ? 0 : kv4_E(rw[x], s, T[x]);
                                w[e] = kv4_W(E, (int)(cv[k] >> (8 * e)) & 255);
                                te += E;
                                tw += w[e];
                            }
                            const unsigned wa = (unsigned)w[0] | ((unsigned)w[1] << 16), wb = (unsigned)w[2] | ((unsigned)w[3] << 16);
                            wl[x][k] = (int)__byte_perm(wa, wb, 0x6420);
                            wh[x][k] = (int)__byte_perm(wa, wb, 0x7531);
                        }
                        sumE[x] += te;
                        sumW[x] += tw;
                    }
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int4 v = *(const int4*)(base + C::PG + c * 512 + lane * 16);
                        const int l0 = kv4_lo(v.x), u0 = kv4_hi(v.x), l1 = kv4_lo(v.y), u1 = kv4_hi(v.y);
                        const int l2 = kv4_lo(v.z), u2 = kv4_hi(v.z), l3 = kv4_lo(v.w), u3 = kv4_hi(v.w);
                        mma_u8u8(aL[2 * c], wl[0][0], wl[1][0], wl[0][1], wl[1][1], l0, u0);
                        mma_u8u8(aH[2 * c], wh[0][0], wh[1][0], wh[0][1], wh[1][1], l0, u0);
                        mma_u8u8(aL[2 * c + 1], wl[0][0], wl[1][0], wl[0][1], wl[1][1], l2, u2);
                        mma_u8u8(aH[2 * c + 1], wh[0][0], wh[1][0], wh[0][1], wh[1][1], l2, u2);
                        mma_u8u8(aL[2 * c], wl[0][2], wl[1][2], wl[0][3], wl[1][3], l1, u1);
                        mma_u8u8(aH[2 * c], wh[0][2], wh[1][2], wh[0][3], wh[1][3], l1, u1);
                        mma_u8u8(aL[2 * c + 1], wl[0][2], wl[1][2], wl[0][3], wl[1][3], l3, u3);
                        mma_u8u8(aH[2 * c + 1], wh[0][2], wh[1][2], wh[0][3], wh[1][3], l3, u3);
                    }
                }
            }
            if (i == np - 1) {
                // the row maxima of this run are complete over the row's four lanes
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 1));
                    T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 2));
                }
            }
            __syncthreads();                             // every warp is done with the stage
            if (tid == 0 && i + KV4_PST < 2 * np) issue(i + KV4_PST);
        }
        it += 2 * np;
    }
    // ---- one deferred division per row
    const i64 MV = kvp[4];
    const int KVS = kvp[5];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        i64 e = sumE[x], w = sumW[x];
        e += __shfl_xor_sync(0xffffffffu, e, 1);
        w += __shfl_xor_sync(0xffffffffu, w, 1);
        e += __shfl_xor_sync(0xffffffffu, e, 2);
        w += __shfl_xor_sync(0xffffffffu, w, 2);
        const int r = x ? rB : rA;
        const int i = r >> p.lgGp, hh = r & ((1 << p.lgGp) - 1);
        if (i >= nt || hh >= p.G) continue;
        const int bl = bitlen_u64((u64)e);
        const i64 rs = e > 0 ? (i64)pow2_recip((u64)e, bl, 1, 23) : 0;
        int32_t* orow = p.o + (size_t)(t0 + i) * p.o_stride + (size_t)(g * p.G + hh) * D + 2 * tig;
#pragma unroll
        for (int n = 0; n < 2 * NC; ++n) {
            int2 out;
            out.x = kv4_out((i64)aL[n][2 * x] + (i64)aH[n][2 * x] * 256 - 8 * w, rs, bl, MV, KVS);
            out.y = kv4_out((i64)aL[n][2 * x + 1] + (i64)aH[n][2 * x + 1] * 256 - 8 * w, rs, bl, MV, KVS);
            *(int2*)(orow + n * 8) = out;
        }
    }
}

}  // namespace detint
