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
// Attention of a query row over its keys (arithmetic specification, section 16):
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
constexpr int KV4_NEG = -2147483647 - 1;   // maximum of no key

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

__device__ __forceinline__ unsigned max4(const int (&x)[4]) {
    const int hi = max(max(x[0], x[1]), max(x[2], x[3])), lo = min(min(x[0], x[1]), min(x[2], x[3]));
    return max((unsigned)max(hi, 0), 0u - (unsigned)min(lo, 0));
}
__device__ __forceinline__ int pack4(const int (&q)[4]) { return q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24); }
__device__ __forceinline__ short4 val4(const int (&q)[4], int c) {
    return make_short4((short)((q[0] - 8) * c), (short)((q[1] - 8) * c), (short)((q[2] - 8) * c), (short)((q[3] - 8) * c));
}

// What a row needs once. Norm: from sum x'^2 (x' the row with its largest
// magnitude brought to 24 bits, cl = clz of that magnitude), the floor square
// root r and R = floor(2^(bl + 23) / r), bl = bitlen(r).
struct Kv4Inv {
    unsigned R;
    int bl;
};
__device__ __forceinline__ Kv4Inv kv4_inv_rms(u64 ss, int lg_d, int cl, i64 eps) {
    Kv4Inv v = {0u, 20};
    if (cl < 32) {
        const int sig = 8 - cl;                              // bitlen - 24
        const u64 es = sig >= 0 ? (u64)eps >> (2 * sig) : (u64)eps << (-2 * sig);   // eps < 2^15: < 2^61
        const u64 r = isqrt_fast((ss >> lg_d) + es);
        v.bl = bitlen_u64(r);
        v.R = (unsigned)pow2_recip(r, v.bl, 1, 23);          // <= 2^24
    }
    return v;
}
// x' of one channel: |x| aligned to bit 31 and cut by 8, sign put back
__device__ __forceinline__ int kv4_cut(int x, int cl) {
    const int m = (int)((uabs32(x) << (cl & 31)) >> 8), s = x >> 31;
    return (m ^ s) - s;
}
// y = rshr(x' gamma R, bl + 21); r >= 2^23 / sqrt(d), so the shift is 41 or
// more and only the high word of the product matters; |x'| / r <= sqrt(d), so
// |y| < 2^21 and nothing that follows saturates
__device__ __forceinline__ int kv4_scale(int x, int g, unsigned R, int bl) {
    const i64 z = (i64)x * g;
    const int hi = (int)(z >> 32) * (int)R + (int)__umulhi((unsigned)z, R);
    return (hi + (1 << (bl - 12))) >> (bl - 11);
}
// without the norm: sat32(4 x)
__device__ __forceinline__ int kv4_x4(int x) {
    return x >= (1 << 29) ? 2147483647 : (x <= -(1 << 29) ? -2147483647 : 4 * x);
}
// rshr(x0 c0 + x1 c1, 14); without the norm saturating to 32 bits
template <bool NORM>
__device__ __forceinline__ int kv4_turn(int x0, int c0, int x1, int c1) {
    const i64 v = (i64)x0 * c0 + ((i64)x1 * c1 + 8192);
    const int hi = (int)(v >> 32), r = (int)__funnelshift_r((unsigned)v, (unsigned)hi, 14);
    if (NORM) return r;
    const int top = hi >> 13;                                // 0 or -1 when the result fits
    return max((unsigned)(top + 1) > 1u ? (hi < 0 ? -2147483647 : 2147483647) : r, -2147483647);
}
// the rotation of a head held as four consecutive channels per lane
template <int LPH, bool NORM>
__device__ __forceinline__ void kv4_rotate(const Kv4Append& p, int pos, int (&y)[4]) {
    const int lane = threadIdx.x & (LPH - 1), R2 = p.rot >> 1;
    if (p.inter) {
        if (4 * lane < p.rot) {
            const unsigned at = (unsigned)max(pos, 0) * R2 + 2 * lane;
            const short2 c = __ldg((const short2*)(p.cos + at)), s = __ldg((const short2*)(p.sin + at));
            const int a0 = y[0], a1 = y[1], a2 = y[2], a3 = y[3];
            y[0] = kv4_turn<NORM>(a0, c.x, a1, -s.x);
            y[1] = kv4_turn<NORM>(a1, c.x, a0, s.x);
            y[2] = kv4_turn<NORM>(a2, c.y, a3, -s.y);
            y[3] = kv4_turn<NORM>(a3, c.y, a2, s.y);
        }
    } else if (R2) {
        const int sh = R2 >> 2;                              // lanes between a pair's halves
        const bool first = lane < sh, in = lane < 2 * sh;
        const int src = (threadIdx.x & 31) + (first ? sh : (in ? -sh : 0));
        const unsigned at = (unsigned)max(pos, 0) * R2 + 4 * (first ? lane : (in ? lane - sh : 0));
        const short4 c = __ldg((const short4*)(p.cos + at)), s = __ldg((const short4*)(p.sin + at));
        const int c4[4] = {c.x, c.y, c.z, c.w};
        const int s4[4] = {first ? -s.x : s.x, first ? -s.y : s.y, first ? -s.z : s.z, first ? -s.w : s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int z = __shfl_sync(seg_mask<LPH>(), y[j], src);
            const int v = kv4_turn<NORM>(y[j], c4[j], z, s4[j]);
            y[j] = in ? v : y[j];
        }
    }
}
// query quantisation: R = floor(127 2^(e + 16) / am), e = bitlen(am), and the
// dyadic scale of am / 127: with a = am aligned to 32 bits, am 2^k / 127 is
// a / (127 2^11) or twice that, whichever is at least 2^14
__device__ __forceinline__ void kv4_qscale(unsigned am, int* R, int* m, int* k) {
    *R = *m = *k = 0;
    if (!am) return;
    const int bl = 32 - __clz(am);
    *R = (int)pow2_recip(am, bl, 127, 16);                   // < 2^24
    const unsigned al = am << (32 - bl);
    const int up = al < (127u << 25);
    *m = (int)((unsigned)((((u64)al << up) + (127u << 10)) >> 11) / 127);
    *k = 35 - bl + up;
}
// rshr(y R, e + 16): aligned by 31 - e the shift is 47, the high word's 15
__device__ __forceinline__ int kv4_q8(int y, unsigned am, int R) {
    const int al = max((int)__clz(am), 1) - 1;
    return (__mulhi(y << (al & 31), R) + (1 << 14)) >> 15;
}
// sat(rshr(v M, s), 1785) for M < 2^30, 0 <= s <= 62: past lim the result
// saturates, and clamping there keeps the shifted product in 32 bits
struct Kv4Fix {
    int M, s, lim;
};
__device__ __forceinline__ Kv4Fix kv4_fix(int M, int s) {
    Kv4Fix f = {min(max(M, 0), 1 << 27), min(max(s, 0), 62), 2147483647};
    if (f.M > 0 && f.s < 50) {
        const u64 n = (u64)(KV4_XMAX + 1) << f.s;            // < 2^61
        if (n < ((u64)f.M << 30)) f.lim = (int)udiv_small(n, (u64)f.M) + 1;
    }
    return f;
}
__device__ __forceinline__ int kv4_fixed(const Kv4Fix& f, int e, int v) {
    const int lim = f.lim == 2147483647 ? f.lim : (f.lim >> e) + 1;
    const i64 p = (i64)min(max(v, -lim), lim) * (f.M << e) + (f.s ? 1ll << (f.s - 1) : 0ll);
    const unsigned lo = (unsigned)p, hi = (unsigned)((u64)p >> 32);
    const bool far = f.s >= 32;
    const int x = (int)__funnelshift_r(far ? hi : lo, far ? (unsigned)((int)hi >> 31) : hi, f.s & 31);
    return min(max(x, -KV4_XMAX), KV4_XMAX);
}
// scale code c = max(1, ceil(max|x| / 7)) and R = floor(2^(b + 16) / c), b =
// bitlen(c): the codes are rshr(x R, b + 16), |x| / c <= 7 (no clamp needed),
// |x R| < 2^11 2^17
__device__ __forceinline__ int kv4_code_scale(unsigned am) { return max(1, (int)((am + 6) / 7)); }
__device__ __forceinline__ int kv4_code_inv(int c) { return (int)pow2_recip((u64)c, 32 - __clz(c), 1, 16); }
__device__ __forceinline__ int kv4_code(int x, int R, int c) { return rshr32(x * R, 48 - __clz(c)) + 8; }

// one k row's codes into its page
template <int LPH>
__device__ __forceinline__ void kv4_put_k(const Kv4Args& a, const Kv4Append& p, int t, int kvh, int blk, int off,
                                          const int (&q)[4], int c, bool live) {
    constexpr int D = 4 * LPH;
    const int lane = threadIdx.x & (LPH - 1);
    const int w4 = pack4(q);
    const int up = __shfl_down_sync(seg_mask<LPH>(), w4, 1);
    if (blk >= 0) {
        const size_t row = ((size_t)blk * a.n_kv + kvh) * KV_BLK + off;
        if (!(lane & 1)) *(int*)(a.k + row * (D / 2) + 2 * lane) = w4 | (up << 4);
        if (lane == 0) a.ks[row] = (uint8_t)c;
    }
    if (live && p.k_val)
        *(short4*)(p.k_val + ((size_t)t * a.n_kv + kvh) * D + 4 * lane) = blk < 0 ? make_short4(0, 0, 0, 0) : val4(q, c);
}
// the page of a token of the call, -1 where nothing is appended
__device__ __forceinline__ int kv4_page_of(const Kv4Args& a, const Kv4Append& p, int t, int pos, int* off) {
    *off = 0;
    return pos >= 0 && pos < p.max_pos ? kv4_slot(a, p.tok_seq[t], pos, off) : -1;
}

// Single tokens: q or k head `slot` of token t, every lane of the head
// repeating what the row needs once (the latency of one row is all there is).
template <int LPH, bool NORM>
__device__ __forceinline__ void kv4_qk_row(const Kv4Args& a, const Kv4Append& p, int t, int slot, bool live) {
    constexpr int D = 4 * LPH;
    const int lane = threadIdx.x & (LPH - 1);
    const bool isq = slot < a.nq;
    const int kvh = isq ? (slot * a.gmul) >> 16 : slot - a.nq;
    int pos = live ? p.tok_pos[t] : -1;
    if (pos >= p.max_pos) {
        if (lane == 0 && a.status) a.status[ST_CTX] = 1;
        pos = -1;
    }
    int4 v = make_int4(0, 0, 0, 0);
    if (pos >= 0) v = __ldg((const int4*)(p.qkv + (size_t)t * p.qkv_stride + (size_t)slot * D + 4 * lane));
    int y[4] = {v.x, v.y, v.z, v.w};
    const int32_t* kvp = a.params + (size_t)kvh * (8 + D);
    const int4 ev = __ldg((const int4*)(kvp + 8 + 4 * lane));
    const int e4[4] = {ev.x & 3, ev.y & 3, ev.z & 3, ev.w & 3};
    if (NORM) {
        const int cl = __clz(seg_max<LPH>(max4(y)));
        u64 ss = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = kv4_cut(y[j], cl);
            ss += (u64)((i64)y[j] * y[j]);
        }
#pragma unroll
        for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(seg_mask<LPH>(), ss, o);
        const Kv4Inv n = kv4_inv_rms(ss, LPH == 32 ? 7 : 6, cl, p.eps);
        const short4 gm = __ldg((const short4*)((isq ? p.q_gamma : p.k_gamma) + 4 * lane));
        const int g4[4] = {gm.x, gm.y, gm.z, gm.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = kv4_scale(y[j], g4[j], n.R, n.bl);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = kv4_x4(y[j]);
    }
    kv4_rotate<LPH, NORM>(p, pos, y);
    if (isq) {
        const int E = (int)seg_max<LPH>((unsigned)max(max(e4[0], e4[1]), max(e4[2], e4[3])));
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = NORM ? y[j] << (E - e4[j]) : sat32((i64)y[j] << (E - e4[j]));
        const unsigned am = seg_max<LPH>(max4(y));
        int R, m, k;
        kv4_qscale(am, &R, &m, &k);
        if (live) {
            const size_t qi = (size_t)t * a.nq + slot;
            *(char4*)(p.q8 + qi * D + 4 * lane) = make_char4((signed char)kv4_q8(y[0], am, R), (signed char)kv4_q8(y[1], am, R),
                                                             (signed char)kv4_q8(y[2], am, R), (signed char)kv4_q8(y[3], am, R));
            if (lane == 0) { p.mq[qi] = m; p.kq[qi] = k; }
        }
    } else {
        const Kv4Fix f = kv4_fix(kvp[0], kvp[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = kv4_fixed(f, e4[j], y[j]);
        const int c = kv4_code_scale(seg_max<LPH>(max4(y))), R = kv4_code_inv(c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = kv4_code(y[j], R, c);
        int off;
        const int blk = kv4_page_of(a, p, t, pos, &off);
        kv4_put_k<LPH>(a, p, t, kvh, blk, off, y, c, live);
    }
}

// Chunks of up to LPH tokens of one head: three passes over the rows, which
// wait in shared memory, with what a row needs once computed between the
// passes by one lane per row. (With each row's lanes repeating the square
// root, reciprocals and dyadic scale, 4 x 4096 tokens of 16 + 8 + 8 heads of
// 128 channels took 535 us, most of it that scalar code.) In a batch of 8
// rows, row i's sum ends up in lanes i LPR .. i LPR + LPR - 1 (LPR = LPH / 8);
// lane l of the head owns row 8 (l % LPR) + l / LPR.
template <int LPH>
__device__ __forceinline__ u64 rows_sum(u64 (&v)[8]) {
    const unsigned mask = seg_mask<LPH>();
    int n = 8;
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) {
        if (n > 1) {
            n >>= 1;
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h < n) {
                    const bool up = (threadIdx.x & o) != 0;
                    const u64 keep = up ? v[h + n] : v[h], give = up ? v[h] : v[h + n];
                    v[h] = keep + __shfl_xor_sync(mask, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(mask, v[0], o);
        }
    }
    return v[0];
}

template <int LPH, bool NORM>
__device__ __forceinline__ void kv4_qk_chunk(const Kv4Args& a, const Kv4Append& p, int t0, int n, int slot, bool live,
                                             int* st) {
    constexpr int D = 4 * LPH, LPR = LPH / 8;
    const unsigned mask = seg_mask<LPH>();
    const int lane = threadIdx.x & (LPH - 1), base = threadIdx.x & 31 & ~(LPH - 1);
    const bool isq = slot < a.nq;
    const int kvh = isq ? (slot * a.gmul) >> 16 : slot - a.nq;
    st += 4 * lane;                                          // row r at st + r D
    // lane l: position (and for keys the page) of token t0 + l
    int pos_l = lane < n ? p.tok_pos[t0 + lane] : -1;
    if (pos_l >= p.max_pos) {
        if (a.status) a.status[ST_CTX] = 1;
        pos_l = -1;
    }
    int blk_l = -1, off_l = 0;
    if (!isq && pos_l >= 0) blk_l = kv4_slot(a, p.tok_seq[t0 + lane], pos_l, &off_l);
    const int32_t* row = p.qkv + (size_t)t0 * p.qkv_stride + (size_t)slot * D + 4 * lane;
    const int4 ev = __ldg((const int4*)(a.params + (size_t)kvh * (8 + D) + 8 + 4 * lane));
    const int e4[4] = {ev.x & 3, ev.y & 3, ev.z & 3, ev.w & 3};
    Kv4Inv inv = {0u, 20};
    int g4[4] = {0, 0, 0, 0};
    if (NORM) {
        const short4 gm = __ldg((const short4*)((isq ? p.q_gamma : p.k_gamma) + 4 * lane));
        g4[0] = gm.x; g4[1] = gm.y; g4[2] = gm.z; g4[3] = gm.w;
        u64 ss_l = 0;
        int cl_l = 32;
        const int32_t* r = row;
#pragma unroll 1
        for (int b = 0; 8 * b < n; ++b) {
            int4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i, r += p.qkv_stride) {
                v[i] = make_int4(0, 0, 0, 0);
                if (__shfl_sync(mask, pos_l, base + 8 * b + i) >= 0) v[i] = __ldg((const int4*)r);
            }
            u64 ss[8];
            int cl[8], least = 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int y[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                cl[i] = __clz(seg_max<LPH>(max4(y)));
                least = min(least, cl[i]);
                if (lane == i * LPR + b) cl_l = cl[i];
            }
            // rows below 2^24 (nearly all there are) only shift left
            const bool small = __all_sync(0xffffffffu, least >= 8);
            if (small) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int s = (cl[i] - 8) & 31;
                    v[i] = make_int4(v[i].x << s, v[i].y << s, v[i].z << s, v[i].w << s);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = make_int4(kv4_cut(v[i].x, cl[i]), kv4_cut(v[i].y, cl[i]), kv4_cut(v[i].z, cl[i]), kv4_cut(v[i].w, cl[i]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss[i] = (u64)((i64)v[i].x * v[i].x) + (u64)((i64)v[i].y * v[i].y) + (u64)((i64)v[i].z * v[i].z) + (u64)((i64)v[i].w * v[i].w);
                *(int4*)(st + (8 * b + i) * D) = v[i];
            }
            const u64 s = rows_sum<LPH>(ss);
            if ((lane & (LPR - 1)) == b) ss_l = s;
        }
        inv = kv4_inv_rms(ss_l, LPH == 32 ? 7 : 6, cl_l, p.eps);
    }
    const int E = isq ? (int)seg_max<LPH>((unsigned)max(max(e4[0], e4[1]), max(e4[2], e4[3]))) : 0;
    Kv4Fix f = {0, 0, 0};
    if (!isq) f = kv4_fix(a.params[(size_t)kvh * (8 + D)], a.params[(size_t)kvh * (8 + D) + 1]);
    unsigned am_l = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i, row += p.qkv_stride) {
        const int own = (i & 7) * LPR + (i >> 3);
        const int pos = __shfl_sync(mask, pos_l, base + i);
        int4 v = make_int4(0, 0, 0, 0);
        if (NORM) v = *(const int4*)(st + i * D);
        else if (pos >= 0) v = __ldg((const int4*)row);
        int y[4] = {v.x, v.y, v.z, v.w};
        const unsigned R = NORM ? __shfl_sync(mask, inv.R, base + own) : 0u;
        const int bl = NORM ? __shfl_sync(mask, inv.bl, base + own) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = NORM ? kv4_scale(y[j], g4[j], R, bl) : kv4_x4(y[j]);
        kv4_rotate<LPH, NORM>(p, pos, y);
        if (isq) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = NORM ? y[j] << (E - e4[j]) : sat32((i64)y[j] << (E - e4[j]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = kv4_fixed(f, e4[j], y[j]);
        }
        const unsigned am = seg_max<LPH>(max4(y));
        if (lane == own) am_l = am;
        *(int4*)(st + i * D) = make_int4(y[0], y[1], y[2], y[3]);
    }
    // (a lane reads back only what it stored itself)
    int R_l = 0, c_l = 1;
    if (isq) {
        int m, k;
        kv4_qscale(am_l, &R_l, &m, &k);
        const int mine = 8 * (lane & (LPR - 1)) + lane / LPR;
        if (live && mine < n) {
            p.mq[(size_t)(t0 + mine) * a.nq + slot] = m;
            p.kq[(size_t)(t0 + mine) * a.nq + slot] = k;
        }
        int8_t* qd = p.q8 + ((size_t)t0 * a.nq + slot) * D + 4 * lane;
#pragma unroll 4
        for (int i = 0; i < n; ++i, qd += a.nq * D) {
            const int own = base + (i & 7) * LPR + (i >> 3);
            const int R = __shfl_sync(mask, R_l, own);
            const unsigned am = __shfl_sync(mask, am_l, own);
            const int4 y = *(const int4*)(st + i * D);
            if (live)
                *(char4*)qd = make_char4((signed char)kv4_q8(y.x, am, R), (signed char)kv4_q8(y.y, am, R),
                                         (signed char)kv4_q8(y.z, am, R), (signed char)kv4_q8(y.w, am, R));
        }
    } else {
        c_l = kv4_code_scale(am_l);
        R_l = kv4_code_inv(c_l);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const int own = base + (i & 7) * LPR + (i >> 3);
            const int R = __shfl_sync(mask, R_l, own), c = __shfl_sync(mask, c_l, own);
            const int4 y = *(const int4*)(st + i * D);
            const int q[4] = {kv4_code(y.x, R, c), kv4_code(y.y, R, c), kv4_code(y.z, R, c), kv4_code(y.w, R, c)};
            kv4_put_k<LPH>(a, p, t0 + i, kvh, __shfl_sync(mask, blk_l, base + i), __shfl_sync(mask, off_l, base + i), q, c, live);
        }
    }
}

// blockIdx.x is a tile of consecutive tokens. blockIdx.y below qk_blocks: one
// warp (half a warp for 64 channels) per q or k head; above: the values of one
// kv head, whose codes are collected in shared memory and then written by
// words of 8 keys. A run of tokens that fills a word is one store; a shorter
// run changes its own nibbles with two atomics, so that another CTA's tokens
// in the same word are kept (the nibbles are distinct, so the order of the
// atomics does not matter).
// Bound: single tokens by latency (one warp's dependent chain, 3.7 us with the
// launch); many by integer instructions, 67 per channel: 4 x 4096 tokens of 16 +
// 8 + 8 heads of 128 channels take 199 us, 2.0 TB/s of the 389 MB they move, at
// 52 % of the ALU pipe and 0.58 instructions per cycle and scheduler. Chunks
// of 16 rows and 6 CTAs per SM: 32 rows took 332 us, 8 or 4 rows held in
// registers 334 and 248 us, 7 CTAs (fewer registers) 212 us; bringing the next
// chunk to L2 ahead changed nothing.
constexpr int KV4_APT = 128;     // append threads
constexpr int KV4_VTILE = 32;    // most tokens in a tile: a lane each
constexpr int KV4_CH = 16;       // rows of a chunk (at most the lanes of a head)

template <int LPH, bool NORM, bool CHUNK>
__global__ void __launch_bounds__(KV4_APT, CHUNK ? 6 : 4) k_kv4_append(Kv4Args a, Kv4Append p) {
    constexpr int D = 4 * LPH, HPW = 32 / LPH, HPB = (KV4_APT / 32) * HPW;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    const int t0 = (int)blockIdx.x * p.tile, nt = min(p.tile, p.T - t0);
    const int lane = threadIdx.x & (LPH - 1), hd = (int)threadIdx.x / LPH;
    if ((int)blockIdx.y < p.qk_blocks) {
        const int slot = (int)blockIdx.y * HPB + hd;
        const bool live = slot < a.nq + a.n_kv;
        if (CHUNK) {
            for (int i = 0; i < nt; i += KV4_CH)
                kv4_qk_chunk<LPH, NORM>(a, p, t0 + i, min(KV4_CH, nt - i), live ? slot : 0, live, (int*)kv4_raw + hd * (KV4_CH * D));
        } else {
            for (int i = 0; i < nt; ++i) kv4_qk_row<LPH, NORM>(a, p, t0 + i, live ? slot : 0, live);
        }
        return;
    }
    __shared__ int page[KV4_VTILE], offs[KV4_VTILE], code[KV4_VTILE], cinv[KV4_VTILE];
    __shared__ unsigned lead_m;
    short4* xs = (short4*)kv4_raw;                           // [nt][LPH] cached integers before coding
    int* cw = (int*)(xs + p.tile * LPH);                     // [nt][LPH] four codes each
    const int g = (int)blockIdx.y - p.qk_blocks;
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    const Kv4Fix f = kv4_fix(kvp[2], kvp[3]);
    if ((int)threadIdx.x < nt) {
        int off;
        page[threadIdx.x] = kv4_page_of(a, p, t0 + (int)threadIdx.x, p.tok_pos[t0 + threadIdx.x], &off);
        offs[threadIdx.x] = off;
    }
    __syncthreads();
    const int32_t* row = p.qkv + (size_t)t0 * p.qkv_stride + (size_t)(a.nq + a.n_kv + g) * D + 4 * lane;
    const int rounds = (nt + HPB - 1) / HPB;
#pragma unroll 4
    for (int k = 0; k < rounds; ++k) {
        const int i = k * HPB + hd;
        int4 v = make_int4(0, 0, 0, 0);
        if (i < nt && page[i] >= 0) v = __ldg((const int4*)(row + (size_t)i * p.qkv_stride));
        const int x[4] = {kv4_fixed(f, 0, v.x), kv4_fixed(f, 0, v.y), kv4_fixed(f, 0, v.z), kv4_fixed(f, 0, v.w)};
        const unsigned am = seg_max<LPH>(max4(x));
        if (i < nt) {
            xs[i * LPH + lane] = make_short4((short)x[0], (short)x[1], (short)x[2], (short)x[3]);
            if (lane == 0) code[i] = (int)am;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < nt) {
        const int c = kv4_code_scale((unsigned)code[threadIdx.x]), blk = page[threadIdx.x];
        code[threadIdx.x] = c;
        cinv[threadIdx.x] = kv4_code_inv(c);
        if (blk >= 0) a.vs[((size_t)blk * a.n_kv + g) * KV_BLK + offs[threadIdx.x]] = (uint8_t)c;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < rounds; ++k) {
        const int i = k * HPB + hd;
        if (i >= nt) break;
        const short4 x = xs[i * LPH + lane];
        const int R = cinv[i], c = code[i];
        const int q[4] = {kv4_code(x.x, R, c), kv4_code(x.y, R, c), kv4_code(x.z, R, c), kv4_code(x.w, R, c)};
        cw[i * LPH + lane] = pack4(q);
        if (p.v_val)
            *(short4*)(p.v_val + ((size_t)(t0 + i) * a.n_kv + g) * D + 4 * lane) =
                page[i] < 0 ? make_short4(0, 0, 0, 0) : val4(q, c);
    }
    __syncthreads();
    // words: a head's lanes take a run of tokens, each its four channels. A run
    // starts where the word changes or the positions stop ascending.
    if ((int)threadIdx.x < KV4_VTILE) {
        const int i = threadIdx.x, blk = i < nt ? page[i] : -1, off = i < nt ? offs[i] : 0;
        const bool lead = blk >= 0 && !(i > 0 && page[i - 1] == blk && (offs[i - 1] >> 3) == (off >> 3) && offs[i - 1] < off);
        const unsigned m = __ballot_sync(0xffffffffu, lead);
        if (i == 0) lead_m = m;
    }
    __syncthreads();
    unsigned todo = lead_m;
    for (int k = 0; todo; ++k, todo &= todo - 1) {
        if ((k & (HPB - 1)) != hd) continue;
        const int i = __ffs((int)todo) - 1;
        const int blk = page[i], off = offs[i];
        int w[8];                                            // codes of the word's keys
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 0;
        unsigned have = 0;
        int last = -1;
        for (int j = i; j < nt && page[j] == blk && (offs[j] >> 3) == (off >> 3) && offs[j] > last; ++j) {
            last = offs[j];
            have |= 1u << (last & 7);
            const int v = cw[j * LPH + lane];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if ((last & 7) == k) w[k] = v;
        }
        // nibbles: key k and k + 4 share a byte; then a 4 x 4 byte transpose
        const int b0 = w[0] | (w[4] << 4), b1 = w[1] | (w[5] << 4), b2 = w[2] | (w[6] << 4), b3 = w[3] | (w[7] << 4);
        const unsigned p01 = __byte_perm(b0, b1, 0x5140), q01 = __byte_perm(b0, b1, 0x7362);
        const unsigned p23 = __byte_perm(b2, b3, 0x5140), q23 = __byte_perm(b2, b3, 0x7362);
        const unsigned o[4] = {__byte_perm(p01, p23, 0x5410), __byte_perm(p01, p23, 0x7632),
                               __byte_perm(q01, q23, 0x5410), __byte_perm(q01, q23, 0x7632)};
        uint32_t* vp = (uint32_t*)(a.v + ((size_t)blk * a.n_kv + g) * (D * KV_BLK / 2)) + (off >> 4) * 4 + ((off >> 3) & 1);
        unsigned keep = 0;                                   // nibbles of keys that are not in the run
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (!(have >> k & 1)) keep |= 15u << (8 * (k & 3) + (k & 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int ch = 4 * lane + j;
            uint32_t* d = vp + (ch >> 4) * 128 + (ch & 7) * 16 + ((ch >> 3) & 1) * 2;
            if (!keep) {
                *d = o[j];
            } else {
                atomicAnd(d, keep);
                atomicOr(d, o[j]);
            }
        }
    }
}

// ------------------------------------------------------------ attention
// a bounded wait for a phase of a bulk copy's barrier, recorded when it runs
// out (the polls come as an argument: with an immediate, some of the kernels
// counted fp16-class instructions)
__device__ __forceinline__ void kv4_wait(unsigned long long* bar, int parity, int polls, int32_t* status) {
    const uint32_t b = smem_u32(bar);
    for (int i = polls; i > 0; --i)
        if (mbar_try_wait(b, (uint32_t)parity)) return;
    if (status) status[ST_TIMEOUT] = 1;
}
// What a query row's scores become: E = exp2q(rshr(d M, sh)) with d = t - T
// <= 0. M is brought to [2^29, 2^30] (and sh with it), and d to a multiple
// that makes the shift at least 33, so that the shifted sum is the high word
// of one 32 x 32 product plus a rounding constant: rshr(d M, sh) = (hi(d mul M)
// + 2^(s2 - 1)) >> s2. From dmin on the result is zero; clamping there keeps
// d mul in 32 bits. (A shift below 3 gives zero for every d < 0, as 3 does.)
struct Kv4Row {
    int M, mul, dmin, s2;
};
__device__ __forceinline__ Kv4Row kv4_row(int mq, int kq, int cstm, int cstk) {
    Kv4Row r = {0, 1, 0, 1};                            // M = 0: every kept key has delta 0
    const i64 m = (i64)mq * cstm;
    if (m <= 0 || m > (1ll << 30)) return r;
    const int z = max(__clz((int)m) - 2, 0);
    const int sh = max(min(max(kq + cstk - 10, 0), 62) + z, 3);
    const int s1 = max(33 - sh, 0);
    if (sh + s1 - 32 >= 28) return r;                   // |d M| < 2^57: rounds to 0
    r.M = (int)(m << z);
    r.mul = 1 << s1;
    r.s2 = sh + s1 - 32;
    r.dmin = -(1 << 27);                                // |t - T| < 2^26
    if (sh < 44) r.dmin = max(r.dmin, -(int)udiv_small(24577ull << sh, (u64)r.M) - 1);
    return r;
}
__device__ __forceinline__ unsigned shr_clamp(unsigned x, int n) {   // 0 for n >= 32
    unsigned y;
    asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(n));
    return y;
}
// 15-bit probability of score t against the row maximum T: exp2q with the
// constants of its Horner steps inside the shifted sums
__device__ __forceinline__ int kv4_E(const Kv4Row& r, int t, int T) {
    const int delta = (__mulhi(max(t - T, r.dmin) * r.mul, r.M) + (1 << (r.s2 - 1))) >> r.s2;
    const int f = delta & 1023;
    const int v1 = (2562 * f + (512 + (7419 << 10))) >> 10;
    const int v2 = (f * v1 + (512 + (22787 << 10))) >> 10;
    const int p2 = (f * v2 + (512 + (32768 << 10))) >> 10;
    return (int)min((shr_clamp(2u * (unsigned)p2, -(delta >> 10)) + 1) >> 1, 32767u);
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
// settle the maximum, and later the sums, among themselves as one thread-block
// cluster (S <= 16, distributed shared memory).
//   scores: a warp takes a page. A lane holds 32 channels of a key and the
//     matching 8 words of every q head in registers; dp4a, then a
//     reduce-scatter over the key's lanes leaves each lane its own heads (a
//     lane keeps its heads in an order of its own, so that no select is
//     needed to pick what it keeps);
//   probabilities: four keys of a head per thread, split into the two bytes
//     of W, tiles of 8 pages in shared memory;
//   P V: mma.sync, V^T codes as the 16-row operand and the bytes of W as its
//     columns 2 h + limb; a warp owns 16 channels. Low and high nibbles have
//     accumulators of their own, the high ones 16 times the sum (no shift).
// Each warp streams what it alone reads, whole K pages and then its 512-byte
// slices of the V pages, through a ring of its own by bulk copies: no barrier
// between warps while scores are formed, and the first V slices travel while
// the unit settles its maximum. dp4a and mma.sync run on different pipes (a
// loop of one does not slow the other).
// Bound: latency, of the launch, the table, one page and two exchanges in the
// cluster (1 token of 65 keys 5.7 us, 8 of 17..767 8.2 us, 16 + 8 heads of 128; 32
// of 1025..1536 keys, 32 + 8 heads of 64, 13 us or 1.7 TB/s of K and V).
constexpr int KV4_DT = 256;      // decode threads
constexpr int KV4_TP = 8;        // pages per probability tile

template <int D>
struct Kv4Ring {
    static constexpr int PG = KV_BLK * D / 2;            // bytes of a K or V page
    static constexpr int SLOT = PG + KV_BLK;             // a K page and its scale codes, or a tile's V slices
    static constexpr int NST = D == 128 ? 2 : 4;         // slots per warp
    static constexpr int BYTES = 8 * NST * SLOT;
};

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

// q heads of a lane: register head i is head HPL (i / HPL ^ subh) + i % HPL,
// subh the lane's place among the lanes that keep heads apart
template <int D, int GT>
struct Kv4Q {
    static constexpr int LPK = D / 32, KPL = 32 / LPK;               // lanes per key, keys per load
    static constexpr int HPL = GT >= LPK ? GT / LPK : 1;             // heads a lane ends up with
    static constexpr int LPG = GT >= LPK ? 1 : LPK / GT;             // lanes that end up with the same head
    int w[GT][8], off[GT];

    __device__ __forceinline__ void load(const int8_t* q8, int nh) { // q8: the unit's first head
        const int sub = threadIdx.x & (LPK - 1), subh = sub / LPG;
#pragma unroll
        for (int i = 0; i < GT; ++i) {
            const int h = HPL * ((i / HPL) ^ subh) + (i & (HPL - 1));
            int4 u = make_int4(0, 0, 0, 0), v = u;
            if (h < nh) {
                const int4* qp = (const int4*)(q8 + (size_t)h * D + sub * 32);
                u = __ldg(qp);
                v = __ldg(qp + 1);
            }
            w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
            w[i][4] = v.x; w[i][5] = v.y; w[i][6] = v.z; w[i][7] = v.w;
            int sq = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = __dp4a(w[i][j], 0x01010101, sq);
            off[i] = -8 * sq;                                        // the codes are values + 8
        }
    }
    // scores of a page in shared memory (K codes, then 64 scale codes): this
    // lane's heads [HPL] of key i KPL + lane / LPK go to out[x * pitch + i KPL];
    // keys outside [lo, hi) do not count for the maxima tm
    __device__ __forceinline__ void page(const unsigned char* base, int* out, int pitch, bool clear, int lo, int hi, int (&tm)[HPL]) const {
        const int lane = threadIdx.x & 31, sub = lane & (LPK - 1), kl = lane / LPK;
        const unsigned char* kr = base + kl * (D / 2) + sub * 16;
        const unsigned char* cr = base + KV_BLK * D / 2 + kl;
        const bool writer = (sub & (LPG - 1)) == 0;
#pragma unroll 4
        for (int i = 0; i < KV_BLK / KPL; ++i) {
            const int4 kv = *(const int4*)(kr + i * (KPL * D / 2));
            const int ck = cr[i * KPL];
            const int ww[4] = {kv.x, kv.y, kv.z, kv.w};
            int acc[GT];
#pragma unroll
            for (int h = 0; h < GT; ++h) acc[h] = off[h];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int l = kv4_lo(ww[x]), u = kv4_hi(ww[x]);
#pragma unroll
                for (int h = 0; h < GT; ++h) acc[h] = __dp4a(l, w[h][2 * x], acc[h]);
#pragma unroll
                for (int h = 0; h < GT; ++h) acc[h] = __dp4a(u, w[h][2 * x + 1], acc[h]);
            }
            // reduce over the key's lanes; the upper half of a lane's registers
            // is its partner's lower half
            int n = GT;
#pragma unroll
            for (int o = LPK / 2; o; o >>= 1) {
                if (n > 1) {
                    n >>= 1;
#pragma unroll
                    for (int h = 0; h < GT / 2; ++h)
                        if (h < n) acc[h] += __shfl_xor_sync(0xffffffffu, acc[h + n], o);
                } else {
                    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
                }
            }
            const int j = i * KPL + kl;
            const bool in = clear || (j >= lo && j < hi);
#pragma unroll
            for (int x = 0; x < HPL; ++x) {
                const int tv = acc[x] * ck;
                if (in) tm[x] = max(tm[x], tv);
                if (writer) out[x * pitch + i * KPL] = tv;
            }
        }
    }
};

// the probabilities of four keys of one head: W's low and high bytes, packed,
// and their sums
__device__ __forceinline__ void kv4_probs(const Kv4Row& rw, int T, const int4& tv, uint32_t cvw, bool clear, int lo, int hi,
                                          uint32_t* wl, uint32_t* wh, unsigned* sumE, unsigned* sumW) {
    const int t4[4] = {tv.x, tv.y, tv.z, tv.w};
    int e[4], w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = kv4_E(rw, t4[k], T);
    if (!clear) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < lo || k >= hi) e[k] = 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = kv4_W(e[k], (int)(cvw >> (8 * k)) & 255);
    *sumE += (unsigned)(e[0] + e[1] + e[2] + e[3]);
    *sumW += (unsigned)(w[0] + w[1] + w[2] + w[3]);
    const unsigned wa = (unsigned)w[0] + ((unsigned)w[1] << 16), wb = (unsigned)w[2] + ((unsigned)w[3] << 16);
    *wl = __byte_perm(wa, wb, 0x6420);
    *wh = __byte_perm(wa, wb, 0x7531);
}
// one page's P V of a warp's 16 channels: vb its 512-byte slice (+ lane * 16),
// wp the page's probability bytes [2 GT][16 words]
template <int GT, int NT>
__device__ __forceinline__ void kv4_pv_page(int (&acc)[NT][2][4], const unsigned char* vb, const uint32_t (*wp)[16]) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int4 v = *(const int4*)vb;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        int4 b = make_int4(0, 0, 0, 0);
        if (8 * n + gid < 2 * GT) b = *(const int4*)&wp[8 * n + gid][4 * tig];
        mma_u8u8(acc[n][0], kv4_lo(v.x), kv4_lo(v.z), kv4_lo(v.y), kv4_lo(v.w), b.x, b.z);
        mma_u8u8(acc[n][1], v.x & 0xf0f0f0f0, v.z & 0xf0f0f0f0, v.y & 0xf0f0f0f0, v.w & 0xf0f0f0f0, b.y, b.w);
    }
}

template <int D, int GT>
__global__ void __launch_bounds__(KV4_DT, 2) k_kv4_decode(Kv4Args a, Kv4Attn p) {
    using C = Kv4Ring<D>;
    using Q = Kv4Q<D, GT>;
    constexpr int LPK = Q::LPK, HPL = Q::HPL;
    constexpr int NG = D / 16, WPG = 8 / NG, NV = KV4_TP / WPG;
    constexpr int NT = (2 * GT + 7) / 8, NPASS = (GT + 1) / 2;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ Kv4DecSm<GT> sm;
    __shared__ unsigned long long full[8][C::NST];
    i64* num_s = (i64*)(kv4_raw + C::BYTES);             // [GT][D]
    int* pg = (int*)(num_s + GT * D);                    // [cap / 64]
    const int pitch = p.cap + 8;                         // 8 banks between heads
    int* ts = pg + (((p.cap >> 6) + 3) & ~3);            // [GT][pitch]

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

    // ---- this warp's stream: its K pages (warp, warp + 8, ...), then its
    // channel group's slices of the V pages, a tile of KV4_TP pages at a time
    const int cg = warp & (NG - 1), ph = warp / NG;
    const int nk = np > warp ? (np - warp + 7) >> 3 : 0, ntile = (np + KV4_TP - 1) / KV4_TP;
    unsigned char* ring = kv4_raw + warp * (C::NST * C::SLOT);
    auto issue = [&](int q) {                            // whole warp
        if (q >= nk + ntile) return;
        const int st = q & (C::NST - 1);
        const uint32_t bar = smem_u32(&full[warp][st]), dst = smem_u32(ring + st * C::SLOT);
        if (q < nk) {
            const int blk = pg[warp + 8 * q];
            if (lane == 0) {
                if (blk < 0) {
                    mbar_arrive(bar);
                } else {
                    const size_t u = (size_t)blk * a.n_kv + g;
                    mbar_arrive_expect_tx(bar, C::PG + KV_BLK);
                    bulk_g2s(dst, a.k + u * C::PG, C::PG, bar);
                    bulk_g2s(dst + C::PG, a.ks + u * KV_BLK, KV_BLK, bar);
                }
            }
        } else {
            const int pi = (q - nk) * KV4_TP + lane * WPG + ph;
            const int blk = lane < NV && pi < np ? pg[pi] : -1;
            const unsigned m = __ballot_sync(0xffffffffu, blk >= 0);
            if (lane == 0) {
                if (m) mbar_arrive_expect_tx(bar, 512 * __popc(m));
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (blk >= 0) bulk_g2s(dst + lane * 512, a.v + ((size_t)blk * a.n_kv + g) * C::PG + cg * 512, 512, bar);
        }
    };
    auto wait = [&](int q) {
        kv4_wait(&full[warp][q & (C::NST - 1)], (q / C::NST) & 1, p.polls, a.status);
    };
#pragma unroll
    for (int q = 0; q < C::NST; ++q) issue(q);

    // ---- scores
    int tm[HPL];
#pragma unroll
    for (int x = 0; x < HPL; ++x) tm[x] = KV4_NEG;
    const int sub = lane & (LPK - 1), hb = sub / Q::LPG * HPL;
    for (int q = 0; q < nk; ++q) {
        const int pi = warp + 8 * q, jb = (pg0 + pi) << 6;
        const bool ok = pg[pi] >= 0;
        wait(q);
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
        for (unsigned r = lane; r < S; r += 32)
            m = max(m, S > 1 ? cl_ld32(&sm.cmax[h], r) : sm.cmax[h]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) sm.tmax[h] = m;
    }
    __syncthreads();

    // ---- probabilities and P V, tiles of KV4_TP pages
    int acc[NT][2][4];                                   // low nibbles; high nibbles, times 16
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][0][e] = acc[n][1][e] = 0;
    unsigned sumE[NPASS], sumW[NPASS];
#pragma unroll
    for (int x = 0; x < NPASS; ++x) sumE[x] = sumW[x] = 0;
    const int qd = tid & 127;                            // this thread's four keys of a tile
    auto load_cv = [&](int tile) -> uint32_t {
        const int pi = tile * KV4_TP + (qd >> 4);
        const int blk = pi < np ? pg[pi] : -1;
        return blk >= 0 ? __ldg((const uint32_t*)(a.vs + ((size_t)blk * a.n_kv + g) * KV_BLK) + (qd & 15)) : 0u;
    };
    uint32_t cv_next = load_cv(0);
    for (int tile = 0; tile < ntile; ++tile) {
        const int buf = tile & 1;
        const uint32_t cvw = cv_next;
        cv_next = load_cv(tile + 1);
        {
            const int pi = tile * KV4_TP + (qd >> 4), jb = ((pg0 + pi) << 6) + 4 * (qd & 15);
            const bool ok = pi < np && pg[pi] >= 0;
            const bool clear = ok && jb >= j0 && jb + 4 <= j1;
#pragma unroll
            for (int x = 0; x < NPASS; ++x) {
                const int h = 2 * x + (tid >> 7);
                if (h < GT) {
                    uint32_t wl = 0, wh = 0;
                    if (ok)
                        kv4_probs(sm.row[h], sm.tmax[h], *(const int4*)(ts + h * pitch + pi * KV_BLK + 4 * (qd & 15)), cvw,
                                  clear, j0 - jb, j1 - jb, &wl, &wh, &sumE[x], &sumW[x]);
                    sm.wp[buf][qd >> 4][2 * h][qd & 15] = wl;
                    sm.wp[buf][qd >> 4][2 * h + 1][qd & 15] = wh;
                }
            }
        }
        __syncthreads();
        wait(nk + tile);
        const unsigned char* vb = ring + ((nk + tile) & (C::NST - 1)) * C::SLOT + lane * 16;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int pt = i * WPG + ph;
            if (tile * KV4_TP + pt >= np) break;         // (a page outside the pool has W = 0)
            kv4_pv_page<GT, NT>(acc, vb + i * 512, sm.wp[buf][pt]);
        }
        __syncwarp();
        issue(nk + tile + C::NST);
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
                const int h = 4 * n + (lane & 3);
                if (h < GT) {
                    i64* d0 = num_s + h * D + cg * 16 + (lane >> 2);
                    int c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = acc[n][0][e] + (acc[n][1][e] >> 4);
                    const i64 v0 = (i64)c[0] + (i64)c[1] * 256, v1 = (i64)c[2] + (i64)c[3] * 256;
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
    }
    if (S > 1) cl_sync();
    else __syncthreads();
    // ---- the row sums, then this CTA's share of the outputs
    if (warp < GT) {
        for (int h = warp; h < GT; h += 8) {
            u64 e = 0, w = 0;
            for (unsigned r = lane; r < S; r += 32) {
                e += (unsigned)(S > 1 ? cl_ld32((const int*)&sm.csum[0][h], r) : (int)sm.csum[0][h]);
                w += (unsigned)(S > 1 ? cl_ld32((const int*)&sm.csum[1][h], r) : (int)sm.csum[1][h]);
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
            num += S > 1 ? cl_ld64(num_s + i, r) : num_s[i];
        orow[i] = kv4_out(num, sm.tot[0][h], (int)sm.tot[1][h], MV, KVS);
    }
    if (S > 1) cl_sync();      // no CTA leaves while another reads its shared memory
}

// ---- the same in two launches, for contexts that keep the whole device busy.
// k_kv4_scores: a warp takes up to 8 pages of one unit by itself and writes
// their scores and its maxima to the workspace. k_kv4_pv: a warp takes pages
// again by itself, forms their probabilities in the registers of its own P V
// operand and runs P V over all channels; the CTA adds its warps' sums in
// shared memory, then to the unit's by 64-bit integer atomics (exact, so their
// order does not matter), and the unit's last CTA divides. Nothing waits for
// another warp in either stream. (With a barrier per tile of 8 pages and a
// warp per 16 channels the second launch took 115 us over 64 contexts of 4 k to
// 16 k keys, 32 + 8 heads of 128, whose tensor time is 67 us; handing half of the
// channels to the dp4a pipe made the barriers longer, 135 us. One cooperative
// launch drawing both kinds of work from a counter took 67 and 180 us where the
// two took 48 and 176: 1 token of 131071 keys, and those 64.) Scores cost 8 bytes of
// traffic per key and head, mostly in L2; K and V are read once, with an
// evict-first policy.
// Bound: at 64 x 4k-16k the score launch takes 66 us, 5.2 TB/s of K with the ALU
// pipe (which runs dp4a's nibble masks and the maxima) half busy; P V takes 110
// us, its tensor work 67, the rest the sums at a chunk's end and the last wave.
// Chunks of 8 pages per warp: 4 and 16 pages were slower. CTAs per SM of P V: 5 (3
// or 4 with 8 heads) cost a few spilled registers and hide a chunk's ends (64 x
// 4k-16k 171 us, with 4 176; with 6, 64 tokens of 8000 keys took 134 us, not 119).
template <int D, int GT>
__global__ void __launch_bounds__(128) k_kv4_scores(Kv4Args a, Kv4Attn p) {
    using C = Kv4Ring<D>;
    using Q = Kv4Q<D, GT>;
    constexpr int LPK = Q::LPK, HPL = Q::HPL, NST = C::NST;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ unsigned long long full[4][NST];
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.z + p.t0, c = blockIdx.x * 4 + warp;
    int g = blockIdx.y, hg = 0;
    while (g >= a.n_kv) { g -= a.n_kv; ++hg; }
    const int nh = min(GT, p.G - hg * GT), h0 = g * p.G + hg * GT;
    const int pos = p.tok_pos[t], seq = p.tok_seq[t];
    if (pos < 0 || pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks) return;
    const int j1 = pos + 1, j0 = p.window > 0 ? max(0, j1 - p.window) : 0;
    const int b0 = j0 >> 6, nb = ((j1 + 63) >> 6) - b0;
    const size_t unit = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (c == 0) {
        for (int i = lane; i < GT * D; i += 32) p.ws_num[unit * (GT * D) + i] = 0;
        for (int i = lane; i < 2 * GT; i += 32) p.ws_sum[unit * (2 * GT) + i] = 0;
        if (lane == 0) p.ws_cnt[unit] = 0;
    }
    const int k0 = c * p.pw, n = min(p.pw, nb - k0);     // pages b0 + k0 ..
    if (n <= 0) return;
    int blk_l = -1;
    if (lane < n) {
        blk_l = a.block_table[(size_t)seq * a.max_blocks + b0 + k0 + lane];
        if (blk_l < 0 || blk_l >= a.n_blocks) {
            blk_l = -1;
            if (a.status) a.status[ST_CTX] = 1;
        }
    }
    if (lane == 0)
        for (int i = 0; i < NST; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    unsigned char* ring = kv4_raw + warp * (NST * C::SLOT);
    const uint64_t pol = l2_evict_first();
    auto issue = [&](int q) {
        if (q >= n) return;
        const int blk = __shfl_sync(0xffffffffu, blk_l, q);
        if (lane == 0) {
            const uint32_t bar = smem_u32(&full[warp][q & (NST - 1)]), dst = smem_u32(ring + (q & (NST - 1)) * C::SLOT);
            if (blk < 0) {
                mbar_arrive(bar);
            } else {
                const size_t u = (size_t)blk * a.n_kv + g;
                mbar_arrive_expect_tx(bar, C::PG + KV_BLK);
                bulk_g2s_hint(dst, a.k + u * C::PG, C::PG, bar, pol);
                bulk_g2s(dst + C::PG, a.ks + u * KV_BLK, KV_BLK, bar);
            }
        }
    };
#pragma unroll
    for (int q = 0; q < NST; ++q) issue(q);
    Q qr;
    qr.load(p.q8 + ((size_t)t * a.nq + h0) * D, nh);
    int tm[HPL];
#pragma unroll
    for (int x = 0; x < HPL; ++x) tm[x] = p.none;
    const int sub = lane & (LPK - 1), hb = sub / Q::LPG * HPL;
    int* out = p.ws_t + (unit * GT + hb) * p.ts_pitch + (size_t)k0 * KV_BLK + lane / LPK;
    for (int q = 0; q < n; ++q, out += KV_BLK) {
        const bool ok = __shfl_sync(0xffffffffu, blk_l, q) >= 0;
        const int jb = (b0 + k0 + q) << 6;
        kv4_wait(&full[warp][q & (NST - 1)], (q / NST) & 1, p.polls, a.status);
        qr.page(ring + (q & (NST - 1)) * C::SLOT, out, p.ts_pitch, ok && jb >= j0 && jb + 64 <= j1, j0 - jb,
                ok ? j1 - jb : -1, tm);
        __syncwarp();
        issue(q + NST);
    }
#pragma unroll
    for (int x = 0; x < HPL; ++x) {
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) tm[x] = max(tm[x], __shfl_xor_sync(0xffffffffu, tm[x], o));
        if (lane < LPK && (sub & (Q::LPG - 1)) == 0) p.ws_max[(unit * p.n_sw + c) * GT + hb + x] = tm[x];
    }
}

template <int D, int GT>
__global__ void __launch_bounds__(128, GT == 8 ? (D == 64 ? 4 : 3) : 5) k_kv4_pv(Kv4Args a, Kv4Attn p) {
    using C = Kv4Ring<D>;
    constexpr int NST = C::NST, NG = D / 16, NT = (2 * GT + 7) / 8;
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ int num[2][GT][D];                        // low and high limb sums of the CTA
    __shared__ int tmax[GT];
    __shared__ unsigned sums[2][GT];
    __shared__ Kv4Row row[GT];
    __shared__ i64 tot[3][GT];
    __shared__ int last;
    __shared__ unsigned long long full[4][NST];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.z + p.t0;
    int g = blockIdx.y, hg = 0;
    while (g >= a.n_kv) { g -= a.n_kv; ++hg; }
    const int nh = min(GT, p.G - hg * GT), h0 = g * p.G + hg * GT;
    const int pos = p.tok_pos[t], seq = p.tok_seq[t];
    int32_t* orow = p.o + (size_t)t * p.o_stride + (size_t)h0 * D;
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (pos < 0 || pos >= p.max_len || seq < 0 || seq >= a.n_seq || (pos >> 6) >= a.max_blocks) {
        if (blockIdx.x == 0) {                           // no key: a zero row
            for (int i = tid; i < nh * D; i += 128) orow[i] = 0;
            if (pos >= 0 && tid == 0 && a.status) a.status[ST_CTX] = 1;
        }
        pdl_wait();                                      // this launch ends after the first, whatever its CTAs do
        return;
    }
    const int j1 = pos + 1, j0 = p.window > 0 ? max(0, j1 - p.window) : 0;
    const int b0 = j0 >> 6, nb = ((j1 + 63) >> 6) - b0;
    const size_t unit = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    // the CTA's pages k0 .. k0 + 2^lg_cp - 1, this warp's every fourth
    const int k0 = (int)blockIdx.x << p.lg_cp, np = min(1 << p.lg_cp, nb - k0);
    if (np <= 0) {
        pdl_wait();
        return;
    }
    const int n = (np - warp + 3) >> 2;
    int blk_l = -1;
    if (lane < n) {
        const int blk = a.block_table[(size_t)seq * a.max_blocks + b0 + k0 + warp + 4 * lane];
        blk_l = blk < a.n_blocks ? max(blk, -1) : -1;    // (recorded by the first launch)
    }
    if (lane == 0)
        for (int i = 0; i < NST; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    unsigned char* ring = kv4_raw + warp * (NST * C::SLOT);
    const uint64_t pol = l2_evict_first();
    auto issue = [&](int q) {
        if (q >= n) return;
        const int blk = __shfl_sync(0xffffffffu, blk_l, q);
        if (lane == 0) {
            const uint32_t bar = smem_u32(&full[warp][q & (NST - 1)]), dst = smem_u32(ring + (q & (NST - 1)) * C::SLOT);
            if (blk < 0) {
                mbar_arrive(bar);
            } else {
                const size_t u = (size_t)blk * a.n_kv + g;
                mbar_arrive_expect_tx(bar, C::PG + KV_BLK);
                bulk_g2s_hint(dst, a.v + u * C::PG, C::PG, bar, pol);
                bulk_g2s(dst + C::PG, a.vs + u * KV_BLK, KV_BLK, bar);
            }
        }
    };
#pragma unroll
    for (int q = 0; q < NST; ++q) issue(q);
    for (int i = tid; i < 2 * GT * D; i += 128) (&num[0][0][0])[i] = 0;
    if (tid < GT) {
        const size_t qi = (size_t)t * a.nq + h0 + min(tid, nh - 1);
        row[tid] = kv4_row(p.mq[qi], p.kq[qi], kvp[6], kvp[7]);
        sums[0][tid] = sums[1][tid] = 0;
    }
    pdl_wait();                                          // the scores are complete
    const int nw = (int)(((u64)(nb + p.pw - 1) * p.pwmul) >> 32);        // ceil(nb / pw) warps wrote maxima
    for (int h = warp; h < GT; h += 4) {
        int m = KV4_NEG;
        for (int r = lane; r < nw; r += 32) m = max(m, __ldcg(p.ws_max + (unit * p.n_sw + r) * GT + h));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) tmax[h] = m;
    }
    __syncthreads();
    // A lane's probabilities: head 4 x + lane / 8, keys 16 tig + 8 limb + 0..7 of
    // a page; its operand column is that head's byte `limb`, keys 16 tig + 0..15:
    // the pair of lanes of a head exchanges the bytes it does not need itself.
    const int tig = lane & 3, limb = (lane >> 2) & 1, koff = 16 * tig + 8 * limb;
    Kv4Row rw[NT];
    int T[NT];
    const int* tsrc[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const int h = min(4 * x + (lane >> 3), GT - 1);
        rw[x] = row[h];
        T[x] = tmax[h];
        tsrc[x] = p.ws_t + (unit * GT + h) * p.ts_pitch + (size_t)(k0 + warp) * KV_BLK + koff;
    }
    const bool mine0 = (lane >> 3) < GT;                 // GT < 4: the other lanes' columns are zero
    int4 tn[NT][2];
    auto load_t = [&](int q) {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            tn[x][0] = tn[x][1] = make_int4(0, 0, 0, 0);
            if (q < n) {
                tn[x][0] = __ldcg((const int4*)(tsrc[x] + q * (4 * KV_BLK)));
                tn[x][1] = __ldcg((const int4*)(tsrc[x] + q * (4 * KV_BLK)) + 1);
            }
        }
    };
    load_t(0);
    int acc[NG][NT][2][4];                               // low nibbles; high nibbles, times 16
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][x][0][e] = acc[c][x][1][e] = 0;
    unsigned sumE[NT], sumW[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) sumE[x] = sumW[x] = 0;
#pragma unroll 1
    for (int q = 0; q < n; ++q) {
        const bool ok = __shfl_sync(0xffffffffu, blk_l, q) >= 0;
        const int jb = ((b0 + k0 + warp + 4 * q) << 6) + koff;
        const bool clear = jb >= j0 && jb + 8 <= j1;
        kv4_wait(&full[warp][q & (NST - 1)], (q / NST) & 1, p.polls, a.status);
        const unsigned char* base = ring + (q & (NST - 1)) * C::SLOT;
        const uint2 cv = *(const uint2*)(base + C::PG + koff);
        int4 b[NT];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            uint32_t l0 = 0, l1 = 0, u0 = 0, u1 = 0;
            if (ok && mine0) {
                kv4_probs(rw[x], T[x], tn[x][0], cv.x, clear, j0 - jb, j1 - jb, &l0, &u0, &sumE[x], &sumW[x]);
                kv4_probs(rw[x], T[x], tn[x][1], cv.y, clear, j0 - jb - 4, j1 - jb - 4, &l1, &u1, &sumE[x], &sumW[x]);
            }
            const uint32_t r0 = __shfl_xor_sync(0xffffffffu, limb ? l0 : u0, 4), r1 = __shfl_xor_sync(0xffffffffu, limb ? l1 : u1, 4);
            b[x] = limb ? make_int4((int)r0, (int)r1, (int)u0, (int)u1) : make_int4((int)l0, (int)l1, (int)r0, (int)r1);
        }
        load_t(q + 1);
        const unsigned char* vb = base + lane * 16;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            const int4 v = *(const int4*)(vb + c * 512);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma_u8u8(acc[c][x][0], kv4_lo(v.x), kv4_lo(v.z), kv4_lo(v.y), kv4_lo(v.w), b[x].x, b[x].z);
                mma_u8u8(acc[c][x][1], v.x & 0xf0f0f0f0, v.z & 0xf0f0f0f0, v.y & 0xf0f0f0f0, v.w & 0xf0f0f0f0, b[x].y, b[x].w);
            }
        }
        __syncwarp();
        issue(q + NST);
    }
    // ---- add up: the CTA's warps, then the unit's CTAs; the last one divides
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            sumE[x] += __shfl_xor_sync(0xffffffffu, sumE[x], o);
            sumW[x] += __shfl_xor_sync(0xffffffffu, sumW[x], o);
        }
        const int h = 4 * x + (lane >> 3);
        if ((lane & 7) == 0 && h < GT) {
            atomicAdd(&sums[0][h], sumE[x]);
            atomicAdd(&sums[1][h], sumW[x]);
        }
        const int hc = 4 * x + tig;                      // the accumulators' head: columns 2 tig, 2 tig + 1
        if (hc < GT) {
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                const int ch = c * 16 + (lane >> 2);
                atomicAdd(&num[0][hc][ch], acc[c][x][0][0] + (acc[c][x][1][0] >> 4));
                atomicAdd(&num[1][hc][ch], acc[c][x][0][1] + (acc[c][x][1][1] >> 4));
                atomicAdd(&num[0][hc][ch + 8], acc[c][x][0][2] + (acc[c][x][1][2] >> 4));
                atomicAdd(&num[1][hc][ch + 8], acc[c][x][0][3] + (acc[c][x][1][3] >> 4));
            }
        }
    }
    __syncthreads();
    unsigned long long* un = (unsigned long long*)p.ws_num + unit * (GT * D);
    unsigned long long* us = p.ws_sum + unit * (2 * GT);
    for (int i = tid; i < nh * D; i += 128)
        atomicAdd(un + i, (unsigned long long)((i64)(&num[0][0][0])[i] + (i64)(&num[1][0][0])[i] * 256));
    if (tid < 2 * GT) atomicAdd(us + tid, (unsigned long long)(&sums[0][0])[tid]);
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        const unsigned chunks = (unsigned)((nb + (1 << p.lg_cp) - 1) >> p.lg_cp);
        last = atomicAdd(p.ws_cnt + unit, 1u) == chunks - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (tid < GT) {
        const u64 e = __ldcg(us + tid), w = __ldcg(us + GT + tid);
        const int bl = bitlen_u64(e);
        tot[0][tid] = e ? (i64)pow2_recip(e, bl, 1, 23) : 0;
        tot[1][tid] = bl;
        tot[2][tid] = -8 * (i64)w;
    }
    __syncthreads();
    for (int i = tid; i < nh * D; i += 128) {
        const int h = i / D;
        orow[i] = kv4_out((i64)__ldcg(un + i) + tot[2][h], tot[0][h], (int)tot[1][h], kvp[4], kvp[5]);
    }
}

// -------------------------------------------- attention of token blocks
// A CTA takes 32 (or 64) query rows (32 / Gp consecutive tokens times the G q
// heads of one kv head, Gp the power of two >= G) and sweeps its keys twice, as the
// maximum has to be known first: sweep 1 scores and maxima, sweep 2 scores,
// probabilities and P V. Two warps share 16 rows: each scores half of a page's
// keys and sums half of the channels. Column n of score tile j is key
// 16 (n / 2) + 2 j + (n & 1), so that the scores a lane holds are the keys of
// its own P V operand for one 32-key step (j / 4, the warp's half); the other
// step's operand comes from the partner through shared memory. (One warp per
// 16 rows with all keys and channels needs no exchange, but its accumulators
// leave 8 warps on an SM: 4 x 4096 tokens of 16 + 8 heads of 128 channels took
// 4336 us, and 4716 us with sweep 1 on the dp4a pipe.) Bound: the int8 tensor
// pipe, 92 % busy over those 4 x 4096 tokens (3840 us; 3480 us would be its
// measured rate for two score sweeps and two limbs), 71 % over 1 x 1024 (99 us),
// where the SMs' causal blocks do not come out even. The tokens of a block may
// belong to several sequences: each run of one sequence is swept by itself
// with the other rows masked. Where there are few blocks, a thread-block cluster
// takes one: its CTAs share a run's pages, settle the maxima between the
// sweeps and add up their sums at the end through distributed shared memory.
constexpr int KV4_PST = 4;       // page stages

template <int D, int NW>
struct Kv4Pf {
    static constexpr int ROWS = 8 * NW;                  // query rows of a CTA of NW warps
    static constexpr int PG = KV_BLK * D / 2;            // bytes of a K or V page
    static constexpr int STAGE = 2 * PG + 2 * KV_BLK;    // K, V, key scales, value scales
    static constexpr int O_W = KV4_PST * STAGE;          // probability operands: 2 buffers x 1 KB per warp
    static constexpr int SMEM = O_W + 2 * NW * 1024;
};

template <int D, int NW>
__global__ void __launch_bounds__(32 * NW, 16 / NW) k_kv4_prefill(Kv4Args a, Kv4Attn p) {
    using C = Kv4Pf<D, NW>;
    constexpr int ROWS = C::ROWS;
    constexpr int KS = D / 32, NC = D / 32;              // 32-channel steps; 16-channel groups of a warp's half
    extern __shared__ __align__(16) unsigned char kv4_raw[];
    __shared__ unsigned long long full[KV4_PST];
    __shared__ int page_ok[KV4_PST];
    __shared__ int r_pos[ROWS], r_top[2][2][ROWS];       // r_top: by runs in turn, by halves
    __shared__ i64 r_sum[2][2][ROWS], tot[3][ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rg = warp >> 1, hf = warp & 1;             // 16-row group; half of the keys and channels
    const int gid = lane >> 2, tig = lane & 3;
    const int g = (int)blockIdx.x >> p.lgC, rank = (int)blockIdx.x & ((1 << p.lgC) - 1);
    const int lgBQ = (NW == 8 ? 6 : 5) - p.lgGp, BQ = 1 << lgBQ;
    const int t0 = p.t0 + (int)(gridDim.y - 1 - blockIdx.y) * BQ;    // later tokens tend to have more keys
    const int nt = min(BQ, p.T - t0);
    const int32_t* kvp = a.params + (size_t)g * (8 + D);
    if (tid == 0) {
        for (int s = 0; s < KV4_PST; ++s) mbar_init(smem_u32(&full[s]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // row r: token t0 + (r >> lgGp), q head r & (Gp - 1)
    const int rA = rg * 16 + gid, rB = rA + 8;
    if (tid < ROWS) {
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
    unsigned sumE[2] = {0, 0}, sumW[2] = {0, 0};         // an eighth of 2^19 keys: below 2^32
    const int k_lane = 16 * tig + 8 * hf;                // first of this lane's eight keys of a page

    int it = 0, wbuf = 0, run = 0;                       // pages consumed so far (ring position); operand and maxima buffers
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
        // the run's pages, and this CTA's share of them
        const int all = (kmax >> 6) - (kmin >> 6) + 1, per = (all + (1 << p.lgC) - 1) >> p.lgC;
        const int p0 = (kmin >> 6) + rank * per, np = min(per, max(0, all - rank * per));
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
        // the row maxima of this run over the row's lanes, both halves and every CTA
        auto settle = [&]() {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 1));
                T[x] = max(T[x], __shfl_xor_sync(0xffffffffu, T[x], 2));
                if (tig == 0) r_top[run][hf][x ? rB : rA] = T[x];
            }
            if (p.lgC) cl_sync();
            else bar_named(1 + rg, 64);
            for (int r = 0; r < (1 << p.lgC); ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int row = x ? rB : rA;
                    const int u = p.lgC ? cl_ld32(&r_top[run][0][row], r) : r_top[run][0][row];
                    const int v = p.lgC ? cl_ld32(&r_top[run][1][row], r) : r_top[run][1][row];
                    T[x] = max(T[x], max(u, v));
                }
            run ^= 1;
        };
        if (np == 0) settle();
        for (int i = 0; i < 2 * np; ++i) {
            if (i == np) settle();
            const int st = (it + i) & (KV4_PST - 1);
            kv4_wait(&full[st], ((it + i) / KV4_PST) & 1, p.polls, a.status);
            const int kb = (p0 + (i >= np ? i - np : i)) << 6;
            if (page_ok[st] && kb <= wmax && kb + 63 >= wmin) {
                const unsigned char* base = kv4_raw + st * C::STAGE;
                const bool clear = kb >= cmin && kb + 63 <= cmax;      // no key of the page is masked
                const uint2 ckv = *(const uint2*)(base + 2 * C::PG + k_lane);
                int S[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    S[j][0] = S[j][1] = qo[0];
                    S[j][2] = S[j][3] = qo[1];
                    const unsigned char* kr = base + (16 * (gid >> 1) + 8 * hf + 2 * j + (gid & 1)) * (D / 2) + tig * (D / 8);
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
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = (int)((j < 2 ? ckv.x : ckv.y) >> (8 * ((2 * j + e) & 3))) & 255;
                        S[j][e] *= c;
                        S[j][2 + e] *= c;
                    }
                if (i < np) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = kb + k_lane + 2 * j + e;
                            if (clear || (key <= hiA && key >= loA)) T[0] = max(T[0], S[j][e]);
                            if (clear || (key <= hiB && key >= loB)) T[1] = max(T[1], S[j][2 + e]);
                        }
                } else {
                    const uint2 cv = *(const uint2*)(base + 2 * C::PG + KV_BLK + k_lane);
                    uint32_t wl[2][2], wh[2][2];         // [row][4 keys]
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int hi = x ? hiB : hiA, lo = x ? loB : loA;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            kv4_probs(rw[x], T[x], make_int4(S[2 * k][2 * x], S[2 * k][2 * x + 1], S[2 * k + 1][2 * x], S[2 * k + 1][2 * x + 1]),
                                      k ? cv.y : cv.x, clear, lo - (kb + k_lane + 4 * k), hi + 1 - (kb + k_lane + 4 * k),
                                      &wl[x][k], &wh[x][k], &sumE[x], &sumW[x]);
                    }
                    // this warp's step of the operand, and the partner's
                    int4* wx = (int4*)(kv4_raw + C::O_W + wbuf * (NW * 1024));
                    wx[(2 * warp) * 32 + lane] = make_int4((int)wl[0][0], (int)wl[1][0], (int)wl[0][1], (int)wl[1][1]);
                    wx[(2 * warp + 1) * 32 + lane] = make_int4((int)wh[0][0], (int)wh[1][0], (int)wh[0][1], (int)wh[1][1]);
                    bar_named(1 + rg, 64);
                    const int4 l0 = wx[(4 * rg) * 32 + lane], u0 = wx[(4 * rg + 1) * 32 + lane];
                    const int4 l1 = wx[(4 * rg + 2) * 32 + lane], u1 = wx[(4 * rg + 3) * 32 + lane];
                    wbuf ^= 1;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int4 v = *(const int4*)(base + C::PG + (hf * NC + c) * 512 + lane * 16);
                        const int a0 = kv4_lo(v.x), b0 = kv4_hi(v.x), a1 = kv4_lo(v.y), b1 = kv4_hi(v.y);
                        const int a2 = kv4_lo(v.z), b2 = kv4_hi(v.z), a3 = kv4_lo(v.w), b3 = kv4_hi(v.w);
                        mma_u8u8(aL[2 * c], l0.x, l0.y, l0.z, l0.w, a0, b0);
                        mma_u8u8(aH[2 * c], u0.x, u0.y, u0.z, u0.w, a0, b0);
                        mma_u8u8(aL[2 * c + 1], l0.x, l0.y, l0.z, l0.w, a2, b2);
                        mma_u8u8(aH[2 * c + 1], u0.x, u0.y, u0.z, u0.w, a2, b2);
                        mma_u8u8(aL[2 * c], l1.x, l1.y, l1.z, l1.w, a1, b1);
                        mma_u8u8(aH[2 * c], u1.x, u1.y, u1.z, u1.w, a1, b1);
                        mma_u8u8(aL[2 * c + 1], l1.x, l1.y, l1.z, l1.w, a3, b3);
                        mma_u8u8(aH[2 * c + 1], u1.x, u1.y, u1.z, u1.w, a3, b3);
                    }
                }
            }
            __syncthreads();                             // every warp is done with the stage
            if (tid == 0 && i + KV4_PST < 2 * np) issue(i + KV4_PST);
        }
        it += 2 * np;
    }
    // ---- the row sums over both halves, then one deferred division per row
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        i64 e = sumE[x], w = sumW[x];
        e += __shfl_xor_sync(0xffffffffu, e, 1);
        w += __shfl_xor_sync(0xffffffffu, w, 1);
        e += __shfl_xor_sync(0xffffffffu, e, 2);
        w += __shfl_xor_sync(0xffffffffu, w, 2);
        if (tig == 0) {
            r_sum[hf][0][x ? rB : rA] = e;
            r_sum[hf][1][x ? rB : rA] = w;
        }
    }
    const i64 MV = kvp[4];
    const int KVS = kvp[5];
    if (p.lgC) {
        // limb sums [row][channel] of every CTA where its pages were; each CTA
        // divides its share of the rows
        int2* nm = (int2*)kv4_raw;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < 2 * NC; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    nm[(x ? rB : rA) * D + hf * (D / 2) + 8 * n + 2 * tig + e] = make_int2(aL[n][2 * x + e], aH[n][2 * x + e]);
        cl_sync();
        const int share = ROWS >> p.lgC;
        if (tid < share) {
            const int r = rank * share + tid;
            i64 e = 0, w = 0;
            for (int q = 0; q < (1 << p.lgC); ++q) {
                e += cl_ld64(&r_sum[0][0][r], q) + cl_ld64(&r_sum[1][0][r], q);
                w += cl_ld64(&r_sum[0][1][r], q) + cl_ld64(&r_sum[1][1][r], q);
            }
            const int bl = bitlen_u64((u64)e);
            tot[0][tid] = e > 0 ? (i64)pow2_recip((u64)e, bl, 1, 23) : 0;
            tot[1][tid] = bl;
            tot[2][tid] = -8 * w;
        }
        __syncthreads();
#pragma unroll 2
        for (int k = tid; k < share * D; k += 32 * NW) {
            const int j = k / D, r = rank * share + j, c = k & (D - 1);
            const int i = r >> p.lgGp, hh = r & ((1 << p.lgGp) - 1);
            if (i >= nt || hh >= p.G) continue;
            i64 num = tot[2][j];
            for (int q = 0; q < (1 << p.lgC); ++q) {
                const i64 v = cl_ld64((const i64*)(nm + r * D + c), q);
                num += (i64)(int)v + (v >> 32) * 256;
            }
            p.o[(size_t)(t0 + i) * p.o_stride + (size_t)(g * p.G + hh) * D + c] = kv4_out(num, tot[0][j], (int)tot[1][j], MV, KVS);
        }
        cl_sync();                                       // no CTA leaves while another reads its shared memory
        return;
    }
    bar_named(1 + rg, 64);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = x ? rB : rA;
        const i64 e = r_sum[0][0][r] + r_sum[1][0][r], w = r_sum[0][1][r] + r_sum[1][1][r];
        const int i = r >> p.lgGp, hh = r & ((1 << p.lgGp) - 1);
        if (i >= nt || hh >= p.G) continue;
        const int bl = bitlen_u64((u64)e);
        const i64 rs = e > 0 ? (i64)pow2_recip((u64)e, bl, 1, 23) : 0;
        int32_t* orow = p.o + (size_t)(t0 + i) * p.o_stride + (size_t)(g * p.G + hh) * D + hf * (D / 2) + 2 * tig;
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
