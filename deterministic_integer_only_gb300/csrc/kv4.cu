// Host side of the 4-bit paged K/V cache: launch shapes, argument checks and
// the C entry points detint_kv4_*. Kernel code lives in k_kv4.cuh.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <mutex>

#include "../../include/detint.h"
#include "k_kv4.cuh"

namespace detint {

namespace {

constexpr int KV4_MAX_LEN = 1 << 19;       // keys: the limb sums stay in int32
constexpr int KV4_CHUNK_MIN = 4;           // tokens of a tile from which append takes chunks

struct DevInfo {
    bool ready = false;
    int sms = 0;
    int max_cluster = 8;                   // CTAs of a cluster at full shared memory
};
DevInfo g_dev[64];
std::mutex g_mu;

DevInfo* dev_info() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    return &g_dev[dev];
}

using DecFn = void (*)(Kv4Args, Kv4Attn);
int lg2(int n) { return n >= 8 ? 3 : n >= 4 ? 2 : n >= 2 ? 1 : 0; }
// [head_dim 128][log2 heads per CTA]: one launch; scores; probabilities and P V
const DecFn DEC_FUSED[2][4] = {{k_kv4_decode<64, 1>, k_kv4_decode<64, 2>, k_kv4_decode<64, 4>, k_kv4_decode<64, 8>},
                               {k_kv4_decode<128, 1>, k_kv4_decode<128, 2>, k_kv4_decode<128, 4>, k_kv4_decode<128, 8>}};
const DecFn DEC_SCORES[2][4] = {{k_kv4_scores<64, 1>, k_kv4_scores<64, 2>, k_kv4_scores<64, 4>, k_kv4_scores<64, 8>},
                                {k_kv4_scores<128, 1>, k_kv4_scores<128, 2>, k_kv4_scores<128, 4>, k_kv4_scores<128, 8>}};
const DecFn DEC_PV[2][4] = {{k_kv4_pv<64, 1>, k_kv4_pv<64, 2>, k_kv4_pv<64, 4>, k_kv4_pv<64, 8>},
                            {k_kv4_pv<128, 1>, k_kv4_pv<128, 2>, k_kv4_pv<128, 4>, k_kv4_pv<128, 8>}};
int scores_smem(int d) { return (d == 128 ? Kv4Ring<128>::BYTES : Kv4Ring<64>::BYTES) / 2; }   // 4 of 8 warps

using AppFn = void (*)(Kv4Args, Kv4Append);
AppFn append_kernel(int d, bool norm, bool chunk) {
    static const AppFn f[2][2][2] = {
        {{k_kv4_append<16, false, false>, k_kv4_append<16, false, true>}, {k_kv4_append<16, true, false>, k_kv4_append<16, true, true>}},
        {{k_kv4_append<32, false, false>, k_kv4_append<32, false, true>}, {k_kv4_append<32, true, false>, k_kv4_append<32, true, true>}}};
    return f[d == 128][norm][chunk];
}

struct Pf {
    DecFn fn;
    int threads, smem;
};
const Pf PREFILL[2][2] = {{{k_kv4_prefill<64, 4>, 128, Kv4Pf<64, 4>::SMEM}, {k_kv4_prefill<64, 8>, 256, Kv4Pf<64, 8>::SMEM}},
                          {{k_kv4_prefill<128, 4>, 128, Kv4Pf<128, 4>::SMEM}, {k_kv4_prefill<128, 8>, 256, Kv4Pf<128, 8>::SMEM}}};

// values: 3 bytes per channel and token; chunks: KV4_CH rows of integers per head
size_t append_smem(int d, int tile) {
    const size_t values = (size_t)tile * d * 3, heads = KV4_APT / (d / 4);
    return tile < KV4_CHUNK_MIN ? values : std::max(values, heads * KV4_CH * d * 4);
}

size_t dec_smem(int d, int gt, int cap) {
    const size_t ring = d == 128 ? Kv4Ring<128>::BYTES : Kv4Ring<64>::BYTES;
    return ring + (size_t)gt * d * 8 + (size_t)(((cap >> 6) + 3) & ~3) * 4 + (size_t)gt * (cap + 8) * 4;
}

// dynamic shared memory up to which two decode CTAs share an SM (228 KB, 1 KB
// of it reserved for each CTA)
size_t dec_smem2(int gt) {
    const size_t fixed = gt == 8 ? sizeof(Kv4DecSm<8>) : gt == 4 ? sizeof(Kv4DecSm<4>) : gt == 2 ? sizeof(Kv4DecSm<2>) : sizeof(Kv4DecSm<1>);
    return 114 * 1024 - 1024 - 1024 - fixed;
}

// how a decode call is split
struct DecPlan {
    int gt, hg;
    bool two;                // two launches
    int S, cap;              // one launch: CTAs per unit, keys per CTA
    size_t smem;
    int pw, n_sw, lg_cp, pitch;
};

// no_ws: one launch wherever it fits
DecPlan dec_plan(const DevInfo& di, const Kv4Args& a, int d, int T, int max_len, int window, bool no_ws) {
    DecPlan p{};
    const int G = a.nq / a.n_kv;
    int mp = (max_len + 63) >> 6;                                   // pages a token can have
    if (window > 0) mp = std::min(mp, ((window + 62) >> 6) + 1);
    p.gt = G >= 5 ? 8 : (G >= 3 ? 4 : G);
    p.hg = (G + p.gt - 1) / p.gt;
    const long long units = (long long)T * a.n_kv * p.hg;
    // One launch: the clusters' CTAs fit the SMs once, two on each, with at
    // least 4 pages each (32 tokens of 1025..1536 keys, 32 + 8 heads of 64: 12.8
    // us split so, 19.8 us as two waves of half the size; 3 tokens of 300 keys, 16
    // + 8 heads of 128: 6.3 us, 7.6 with 2 pages each; 1 of 2000: 8.2 and 7.8). Where the scores of
    // such a CTA do not fit its shared memory, two launches (64 tokens of 4 k
    // to 16 k keys, 32 + 8 heads of 128: 171 us, against 276 us in larger
    // clusters; at 38 tokens of 4000 keys 50 and 53 us, at 76 of 2000, where
    // the scores fit, 51 and 48 us).
    int S = 1;
    while (S < di.max_cluster && units * 2 * S <= 2 * di.sms && mp >= 8 * S) S <<= 1;
    p.S = S;
    p.cap = ((mp + S - 1) / S) << 6;
    p.smem = dec_smem(d, p.gt, p.cap);
    p.two = p.smem > dec_smem2(p.gt);
    // Two as well where CTAs of more than 32 pages leave over a quarter of their
    // places on the SMs empty (16 + 8 heads of 128: 1 token of 120000 keys 33 us,
    // 49 in one launch, 40 of 4000 45 and 50; 100 of 3000, which fill 88 % of
    // them, 78 and 73 us).
    const long long n = units * S, places = 2 * di.sms, waves = (n + places - 1) / places;
    if (!no_ws && p.cap > 32 * KV_BLK && 4 * n < 3 * waves * places) p.two = true;
    if (p.two) {
        // pages of a score warp: 32 warps per SM, of which 6 CTAs of 4 fit at a
        // time (16 tokens of 12000 keys, 32 + 8 heads of 128: 55 us; with 16 warps
        // 58, with 48 55)
        p.pw = 8;
        while (p.pw > 1 && units * ((mp + p.pw - 1) / p.pw) < 32LL * di.sms) p.pw >>= 1;
        p.n_sw = (mp + p.pw - 1) / p.pw;
        // pages of a P V CTA: 6 CTAs per SM (3 tokens of 20000 keys, 32 + 8 heads of
        // 128: 28 us; with 10 32; 40 of 4000, heads of 64: 34, 40; with 4 as with 6)
        p.lg_cp = 5;                                                // up to 8 pages a warp
        while (p.lg_cp > 2 && units * ((mp + (1 << p.lg_cp) - 1) >> p.lg_cp) < 6LL * di.sms) --p.lg_cp;
        p.pitch = ((mp + 7) & ~7) << 6;                             // whole tiles
    }
    return p;
}

size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }
struct WsLayout { size_t t, mx, sum, num, cnt, total; };
WsLayout ws_layout(const DecPlan& p, long long units, int d) {
    WsLayout w{};
    size_t o = 0;
    const size_t n = (size_t)units * p.gt;
    w.t = o; o += a256(n * p.pitch * 4);
    w.mx = o; o += a256(n * p.n_sw * 4);
    w.sum = o; o += a256(n * 16);
    w.num = o; o += a256(n * d * 8);
    w.cnt = o; o += a256((size_t)units * 4);
    w.total = o;
    return w;
}

}  // namespace

cudaError_t kv4_init() {
    DevInfo* di = dev_info();
    if (!di) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    if (di->ready) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&di->sms, cudaDevAttrMultiProcessorCount, dev);
    int mc = 16;
    for (int d : {64, 128})
        for (int l = 0; l < 4; ++l) {
            const DecFn f = DEC_FUSED[d == 128][l];
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dec_smem2(1 << l));
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(DEC_SCORES[d == 128][l], cudaFuncAttributeMaxDynamicSharedMemorySize, scores_smem(d));
            if (e == cudaSuccess) e = cudaFuncSetAttribute(DEC_PV[d == 128][l], cudaFuncAttributeMaxDynamicSharedMemorySize, scores_smem(d));
            if (e != cudaSuccess) continue;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 16;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(KV4_DT);
            cfg.dynamicSmemBytes = dec_smem2(1 << l);
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, f, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                mc = 8;
            }
        }
    for (int d : {64, 128})
        for (int norm = 0; norm < 2; ++norm)
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(append_kernel(d, norm, true), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)append_smem(d, KV4_VTILE));
    for (const Pf& f : {PREFILL[0][0], PREFILL[0][1], PREFILL[1][0], PREFILL[1][1]})
        for (int i = 0; i < 2 && e == cudaSuccess; ++i)
            e = i ? cudaFuncSetAttribute(f.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)
                  : cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem);
    if (e == cudaSuccess) {
        di->max_cluster = mc;
        di->ready = true;
    }
    return e;
}

cudaError_t launch_kv4_append(const Kv4Args& a, const Kv4Append& p0, int d, cudaStream_t s) {
    Kv4Append p = p0;
    DevInfo* di = dev_info();
    if (!di || !di->ready) return cudaErrorInvalidDevice;
    const int hpb = d == 128 ? 4 : 8;
    p.qk_blocks = (a.nq + a.n_kv + hpb - 1) / hpb;
    // Tokens per CTA: up to 32 (of 64, 10000 tokens of 16 + 8 + 8 heads of 128 made
    // 2.4 waves and took 170 us, not 131), as many as still make 6 CTAs per SM
    // (with 4, 1400 and 2800 tokens took 31 and 75 us, not 22 and 44; with 8, 300
    // took 11.5, not 8.8). Below 4 each row's lanes repeat what the row needs once:
    // the chunk's three passes have too few rows (300 tokens in tiles of 2: 12.6
    // us in chunks, 11.5 us by rows; in tiles of 4: 8.9 and 13.6 us).
    const int per_tile = p.qk_blocks + a.n_kv;
    p.tile = KV4_VTILE;
    while (p.tile > 1 && (long long)((p.T + p.tile - 1) / p.tile) * per_tile < 6LL * di->sms) p.tile >>= 1;
    const dim3 grid((p.T + p.tile - 1) / p.tile, per_tile);
    const size_t smem = append_smem(d, p.tile);
    append_kernel(d, p.q_gamma != nullptr, p.tile >= KV4_CHUNK_MIN)<<<grid, KV4_APT, smem, s>>>(a, p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_prefill(const Kv4Args& a, const Kv4Attn& p0, int d, cudaStream_t s) {
    Kv4Attn p = p0;
    p.polls = SG_SPIN;
    p.none = KV4_NEG;
    DevInfo* di = dev_info();
    if (!di || !di->ready) return cudaErrorInvalidDevice;
    // so few tokens that the single-token form takes them all in one wave: the
    // same rows, with every key split over CTAs (3 x 13 tokens after 4000 keys,
    // 2 + 1 heads of 128: 14.5 us, 53 us in blocks; 20 after 1000, 16 + 8 heads: 13
    // and 22 us)
    const DecPlan dp = dec_plan(*di, a, d, p.T, p.max_len, p.window, true);
    if (!dp.two && (long long)p.T * a.n_kv * dp.hg <= 2LL * di->sms) return launch_kv4_decode(a, p0, d, nullptr, s);
    p.lgGp = 0;
    while ((1 << p.lgGp) < p.G) ++p.lgGp;
    // 32 rows per CTA and four CTAs on an SM balance causal blocks better than
    // 64 rows and two (4 x 4096 tokens 3840 us, not 3951; 1 x 1024 99 us, not 117);
    // only a group of more than 32 heads needs 64
    const bool wide = p.lgGp > 5;
    const int bq = (wide ? 64 : 32) >> p.lgGp;
    const int tiles = (p.T + bq - 1) / bq;
    // few blocks: clusters whose CTAs share a block's pages, while they fit the
    // SMs once (four CTAs on each) and a CTA keeps 2 pages (60 tokens after 4000
    // keys, 16 + 8 heads of 128: 52 us, one CTA per block 302 us; 1 x 512: 38 and
    // 47 us)
    const int mp = (p.max_len + 63) >> 6;
    p.lgC = 0;
    while (!wide && p.lgC < 4 && (1 << (p.lgC + 1)) <= di->max_cluster &&
           ((long long)tiles * a.n_kv << (p.lgC + 1)) <= 4LL * di->sms && mp >= 4 << p.lgC)
        ++p.lgC;
    const Pf f = PREFILL[d == 128][wide];
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1 << p.lgC;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.lgC ? 1 : 0;
    cfg.blockDim = dim3(f.threads);
    cfg.dynamicSmemBytes = f.smem;
    cfg.stream = s;
    for (int b0 = 0; b0 < tiles; b0 += 65535) {
        p.t0 = b0 * bq;
        cfg.gridDim = dim3(a.n_kv << p.lgC, std::min(65535, tiles - b0));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, f.fn, a, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Bytes for a call of two launches, whatever its window: fewer keys take less
// of each array, but may need more warps and CTAs per page, which only the
// maxima depend on. Fewer tokens or keys take less.
static size_t ws_bytes(const Kv4Args& a, int d, int T, int max_len, DecPlan pl) {
    pl.n_sw = (max_len + 63) >> 6;
    return ws_layout(pl, (long long)T * a.n_kv * pl.hg, d).total;
}
// The most that a call of T tokens or fewer may ask for. Two launches depend on
// how the CTAs fill the SMs, so fewer tokens may take them where T take one (16 +
// 8 heads of 128, 3000 keys: 20 and 40 tokens do, 38, 64 and 100 do not); for a
// number of tokens, more keys never turn two launches into one. Past three waves
// of one CTA per unit a wave is never a quarter empty and shared memory alone
// decides, for every number of tokens alike.
size_t kv4_decode_ws(const Kv4Args& a, int d, int T, int max_len) {
    DevInfo* di = dev_info();
    if (!di || !di->ready) return 0;
    for (int n = std::min(T, 65535); n > 0; --n) {
        const DecPlan pl = dec_plan(*di, a, d, n, max_len, 0, false);
        if (pl.two) return ws_bytes(a, d, n, max_len, pl);
        n = std::min(n, 6 * di->sms / (a.n_kv * pl.hg) + 1);
    }
    return 0;
}
size_t kv4_decode_need(const Kv4Args& a, int d, int T, int max_len, int window) {
    DevInfo* di = dev_info();
    if (!di || !di->ready) return 0;
    const int Tc = std::min(T, 65535);
    if (!dec_plan(*di, a, d, Tc, max_len, window, false).two) return 0;
    return ws_bytes(a, d, Tc, max_len, dec_plan(*di, a, d, Tc, max_len, 0, false));
}

cudaError_t launch_kv4_decode(const Kv4Args& a, const Kv4Attn& p0, int d, void* ws, cudaStream_t s) {
    DevInfo* di = dev_info();
    if (!di || !di->ready) return cudaErrorInvalidDevice;
    Kv4Attn p = p0;
    p.polls = SG_SPIN;
    p.none = KV4_NEG;
    const DecPlan pl = dec_plan(*di, a, d, std::min(p.T, 65535), p.max_len, p.window, !ws);
    const int d128 = d == 128, l = lg2(pl.gt);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.stream = s;
    cfg.attrs = at;
    for (int t0 = 0; t0 < p.T; t0 += 65535) {
        const int nt = std::min(65535, p.T - t0);
        p.t0 = t0;
        cudaError_t e;
        if (!pl.two) {
            p.cap = pl.cap;
            p.smul = ((1ull << 32) + pl.S - 1) / pl.S;
            cfg.gridDim = dim3(pl.S, a.n_kv * pl.hg, nt);
            cfg.blockDim = dim3(KV4_DT);
            cfg.dynamicSmemBytes = pl.smem;
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = pl.S;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.numAttrs = pl.S > 1 ? 1 : 0;
            e = cudaLaunchKernelEx(&cfg, DEC_FUSED[d128][l], a, p);
        } else {
            const WsLayout w = ws_layout(pl, (long long)nt * a.n_kv * pl.hg, d);
            unsigned char* b = (unsigned char*)ws;
            p.ws_t = (int32_t*)(b + w.t);
            p.ws_max = (int32_t*)(b + w.mx);
            p.ws_sum = (unsigned long long*)(b + w.sum);
            p.ws_num = (long long*)(b + w.num);
            p.ws_cnt = (unsigned*)(b + w.cnt);
            p.pw = pl.pw;
            p.pwmul = ((1ull << 32) + pl.pw - 1) / pl.pw;
            p.n_sw = pl.n_sw;
            p.lg_cp = pl.lg_cp;
            p.ts_pitch = pl.pitch;
            cfg.gridDim = dim3((pl.n_sw + 3) / 4, a.n_kv * pl.hg, nt);
            cfg.blockDim = dim3(128);
            cfg.dynamicSmemBytes = scores_smem(d);
            cfg.numAttrs = 0;
            e = cudaLaunchKernelEx(&cfg, DEC_SCORES[d128][l], a, p);
            if (e != cudaSuccess) return e;
            // starts while the first launch drains: its V slices travel before it waits
            cfg.gridDim = dim3((pl.pitch / 64 + (1 << pl.lg_cp) - 1) >> pl.lg_cp, a.n_kv * pl.hg, nt);
            at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, DEC_PV[d128][l], a, p);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace detint

using namespace detint;

namespace {

int failed(int code, const char* where, const char* what) {
    char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", where, what);
    return set_last_error(code, msg);
}
// (the error is reported here and not left for the check of the next launch)
int cuda_fail(const char* where, cudaError_t e) {
    cudaGetLastError();
    return failed(DETINT_E_CUDA, where, cudaGetErrorString(e));
}
bool mis(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; }

// the checks every entry point shares; fills the kernels' view of the cache
int check_cache(const char* where, const detint_kv4_t* c, Kv4Args* a) {
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    if (!c) return err(DETINT_E_ARG, "null cache");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->params) return err(DETINT_E_ARG, "null pointer in the cache");
    if (c->head_dim != 64 && c->head_dim != 128) return err(DETINT_E_SHAPE, "head_dim must be 64 or 128");
    if (c->n_kv < 1 || c->n_q < 1 || c->n_q > 1024 || c->n_q % c->n_kv || c->n_q / c->n_kv > 64)
        return err(DETINT_E_SHAPE, "n_q must be n_kv times 1..64, at most 1024");
    if (c->n_blocks < 1 || c->n_seq < 1 || c->max_blocks < 1) return err(DETINT_E_ARG, "n_blocks, n_seq and max_blocks must be positive");
    if (mis(c->k, 16) || mis(c->v, 16) || mis(c->k_scale, 16) || mis(c->v_scale, 16) || mis(c->params, 16))
        return err(DETINT_E_ARG, "pages, scale codes and parameters must be 16-byte aligned");
    if (mis(c->block_table, 4) || mis(c->status, 4)) return err(DETINT_E_ARG, "block_table and status must be 4-byte aligned");
    a->nq = c->n_q; a->n_kv = c->n_kv; a->n_blocks = c->n_blocks; a->n_seq = c->n_seq; a->max_blocks = c->max_blocks;
    a->gmul = (65536 + c->n_q / c->n_kv - 1) / (c->n_q / c->n_kv);
    a->k = c->k; a->v = c->v; a->ks = c->k_scale; a->vs = c->v_scale;
    a->block_table = c->block_table; a->params = c->params; a->status = c->status;
    return DETINT_OK;
}

int check_attn(const char* where, const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
               const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window, int32_t* o,
               long long o_stride, Kv4Args* a, Kv4Attn* p) {
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    const int rc = check_cache(where, c, a);
    if (rc) return rc;
    if (!q8 || !mq || !kq || !tok_seq || !tok_pos || !o) return err(DETINT_E_ARG, "null pointer");
    if (n_tok < 1) return err(DETINT_E_ARG, "n_tok must be positive");
    if (max_len < 1 || max_len > KV4_MAX_LEN) return err(DETINT_E_ARG, "max_len must be in 1..524288");
    if (window < 0) return err(DETINT_E_ARG, "window must not be negative");
    if (mis(tok_seq, 4) || mis(tok_pos, 4) || mis(mq, 4) || mis(kq, 4)) return err(DETINT_E_ARG, "tokens and scales must be 4-byte aligned");
    if (mis(q8, 16) || mis(o, 8)) return err(DETINT_E_ARG, "q8 must be 16-byte and o 8-byte aligned");
    if (o_stride < (long long)c->n_q * c->head_dim || (o_stride & 1)) return err(DETINT_E_ARG, "o_stride must be even and hold a row");
    *p = Kv4Attn{};
    p->q8 = q8; p->mq = mq; p->kq = kq; p->tok_seq = tok_seq; p->tok_pos = tok_pos; p->o = o; p->o_stride = (size_t)o_stride;
    p->T = n_tok; p->G = c->n_q / c->n_kv; p->max_len = max_len;
    p->window = window < max_len ? window : 0;      // a window that every key is in: none (any int, so no sum with it may overflow)
    return DETINT_OK;
}

}  // namespace

extern "C" {

int detint_kv4_append(const detint_kv4_t* c, const detint_rope_t* r, const int32_t* qkv, long long qkv_stride,
                      const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int8_t* q8, int32_t* mq, int32_t* kq,
                      int16_t* k_val, int16_t* v_val, detint_stream_t sp) {
    const char* where = "detint_kv4_append";
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    Kv4Args a{};
    const int rc = check_cache(where, c, &a);
    if (rc) return rc;
    const int d = c->head_dim;
    if (!r || !qkv || !tok_seq || !tok_pos || !q8 || !mq || !kq) return err(DETINT_E_ARG, "null pointer");
    if (n_tok < 1) return err(DETINT_E_ARG, "n_tok must be positive");
    if (r->rot_dim < 0 || r->rot_dim > d || (r->rot_dim & 7)) return err(DETINT_E_SHAPE, "rot_dim must be a multiple of 8 up to head_dim");
    if (r->max_pos < 1 || (r->rot_dim && (!r->cos || !r->sin))) return err(DETINT_E_ARG, "rotation tables missing");
    if (r->interleaved != 0 && r->interleaved != 1) return err(DETINT_E_ARG, "interleaved must be 0 or 1");
    if (!r->q_gamma != !r->k_gamma) return err(DETINT_E_ARG, "both gammas or none");
    if (r->eps < 0 || r->eps > 32767) return err(DETINT_E_ARG, "eps must be in 0..32767");
    if (mis(r->cos, 8) || mis(r->sin, 8) || mis(r->q_gamma, 8) || mis(r->k_gamma, 8)) return err(DETINT_E_ARG, "tables and gammas must be 8-byte aligned");
    if ((long long)r->max_pos * r->rot_dim > 0x7fffffffLL) return err(DETINT_E_SHAPE, "rotation tables too large");
    if (qkv_stride < (long long)(c->n_q + 2 * c->n_kv) * d || (qkv_stride & 3) || mis(qkv, 16))
        return err(DETINT_E_ARG, "qkv rows must be 16-byte aligned and hold every head");
    if (mis(tok_seq, 4) || mis(tok_pos, 4) || mis(mq, 4) || mis(kq, 4)) return err(DETINT_E_ARG, "tokens and scales must be 4-byte aligned");
    if (mis(q8, 16) || mis(k_val, 8) || mis(v_val, 8)) return err(DETINT_E_ARG, "outputs misaligned");
    Kv4Append p{};
    p.qkv = qkv; p.qkv_stride = (size_t)qkv_stride; p.tok_seq = tok_seq; p.tok_pos = tok_pos; p.T = n_tok;
    p.cos = r->cos; p.sin = r->sin; p.max_pos = r->max_pos; p.rot = r->rot_dim; p.inter = r->interleaved;
    p.q_gamma = r->q_gamma; p.k_gamma = r->k_gamma; p.eps = r->eps;
    p.q8 = q8; p.mq = mq; p.kq = kq; p.k_val = k_val; p.v_val = v_val;
    cudaError_t e = kv4_init();
    if (e == cudaSuccess) e = launch_kv4_append(a, p, d, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

int detint_kv4_workspace(const detint_kv4_t* c, int n_tok, int max_len, long long* bytes) {
    Kv4Args a{};
    const int rc = check_cache("detint_kv4_workspace", c, &a);
    if (rc) return rc;
    if (!bytes || n_tok < 1 || max_len < 1 || max_len > KV4_MAX_LEN)
        return set_last_error(DETINT_E_ARG, "detint_kv4_workspace: bad arguments");
    const cudaError_t e = kv4_init();
    if (e != cudaSuccess) return cuda_fail("detint_kv4_workspace", e);
    *bytes = (long long)kv4_decode_ws(a, c->head_dim, n_tok, max_len);
    return DETINT_OK;
}

int detint_kv4_decode(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
                      const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window, int32_t* o,
                      long long o_stride, void* workspace, long long workspace_bytes, detint_stream_t sp) {
    const char* where = "detint_kv4_decode";
    Kv4Args a{};
    Kv4Attn p{};
    const int rc = check_attn(where, c, q8, mq, kq, tok_seq, tok_pos, n_tok, max_len, window, o, o_stride, &a, &p);
    if (rc) return rc;
    cudaError_t e = kv4_init();
    if (e != cudaSuccess) return cuda_fail(where, e);
    const size_t need = kv4_decode_need(a, c->head_dim, n_tok, max_len, p.window);
    if (need && (!workspace || workspace_bytes < (long long)need || mis(workspace, 16)))
        return failed(DETINT_E_ARG, where, "a 16-byte aligned workspace of detint_kv4_workspace bytes is needed");
    e = launch_kv4_decode(a, p, c->head_dim, workspace, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

int detint_kv4_prefill(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
                       const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window, int32_t* o,
                       long long o_stride, detint_stream_t sp) {
    const char* where = "detint_kv4_prefill";
    Kv4Args a{};
    Kv4Attn p{};
    const int rc = check_attn(where, c, q8, mq, kq, tok_seq, tok_pos, n_tok, max_len, window, o, o_stride, &a, &p);
    if (rc) return rc;
    cudaError_t e = kv4_init();
    if (e == cudaSuccess) e = launch_kv4_prefill(a, p, c->head_dim, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

}  // extern "C"
