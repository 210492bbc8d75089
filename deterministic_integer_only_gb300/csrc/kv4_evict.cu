// Host side of the cached keys' weights, eviction and page copies: launch
// shapes, argument checks and the C entry points. Kernel code: k_kv4_evict.cuh.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "../../include/detint.h"
#include "k_kv4_evict.cuh"
#include "kv4_check.h"

namespace detint {

namespace {

struct DevInfo {
    bool ready = false;
    int sms = 0;
    int max_cluster = 8;
};
DevInfo g_dev[64];
std::mutex g_mu;

constexpr int SMEM_MAX = 227 * 1024;
constexpr int EV_HELD = 192 * 1024;          // bytes of keys that select holds in shared memory

using WeighFn = void (*)(Kv4Args, Kv4Attn, Kv4Weigh);
constexpr int NGT = 3;                       // 1, 2 or 4 heads of a CTA
const WeighFn WEIGH[2][NGT] = {{k_kv4_weigh<64, 1>, k_kv4_weigh<64, 2>, k_kv4_weigh<64, 4>},
                               {k_kv4_weigh<128, 1>, k_kv4_weigh<128, 2>, k_kv4_weigh<128, 4>}};
const WeighFn WEIGH_BLOCK[2][2] = {{k_kv4_weigh_block<64, 2>, k_kv4_weigh_block<64, 3>}, {k_kv4_weigh_block<128, 2>, k_kv4_weigh_block<128, 3>}};   // 4 or 8 warps
void (*const EV_SELECT[2])(Kv4Args, Kv4Evict) = {k_kv4_evict_select<256>, k_kv4_evict_select<512>};
int lg2(int n) { return n >= 4 ? 2 : n >= 2 ? 1 : 0; }
size_t weigh_fixed(int gt) { return gt == 4 ? sizeof(Kv4WeighSm<4>) : gt == 2 ? sizeof(Kv4WeighSm<2>) : sizeof(Kv4WeighSm<1>); }
size_t weigh_smem(int gt, int cap) {
    return (size_t)(((cap >> 6) + 3) & ~3) * 4 + (size_t)gt * (cap + 8) * 4;
}
// dynamic shared memory of one CTA on an SM, and of two
size_t weigh_room(int gt, int ctas) { return (ctas == 1 ? SMEM_MAX : 113 * 1024) - 1024 - weigh_fixed(gt); }

// CTAs of the largest cluster that can run, 16 or 8
int cluster_of(const void* f, int threads, size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 16;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, f, &cfg) == cudaSuccess && n >= 1) return 16;
    cudaGetLastError();
    return 8;
}

// sets the kernels' attributes once per device (no call that a stream capture forbids)
cudaError_t init(DevInfo** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    DevInfo* di = *out = &g_dev[dev];
    std::lock_guard<std::mutex> lk(g_mu);
    if (di->ready) return cudaSuccess;
    e = cudaDeviceGetAttribute(&di->sms, cudaDevAttrMultiProcessorCount, dev);
    int mc = 16;
    for (int d : {0, 1})
        for (int l = 0; l < NGT && e == cudaSuccess; ++l) {
            const size_t room = weigh_room(1 << l, 1);
            e = cudaFuncSetAttribute(WEIGH[d][l], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(WEIGH[d][l], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) mc = std::min(mc, cluster_of((const void*)WEIGH[d][l], KV4_DT, room));
        }
    for (int d : {0, 1})
        for (int l = 0; l < 2 && e == cudaSuccess; ++l) {
            const WeighFn f = WEIGH_BLOCK[d][l];
            const int bytes = (WB_SMEM + 16 * WB_EXCH) * (4 << l);
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) mc = std::min(mc, cluster_of((const void*)f, 128 << l, bytes));
        }
    for (int w : {0, 1}) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(EV_SELECT[w], cudaFuncAttributeMaxDynamicSharedMemorySize, EV_HELD);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(EV_SELECT[w], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) mc = std::min(mc, cluster_of((const void*)EV_SELECT[w], 256 << w, EV_HELD));
    }
    if (e == cudaSuccess) {
        di->max_cluster = mc;
        di->ready = true;
    }
    return e;
}

cudaError_t launch_weigh(const DevInfo& di, const Kv4Args& a, Kv4Attn p, const Kv4Weigh& w, int d, cudaStream_t s) {
    p.none = KV4_NEG;
    int mp = (p.max_len + 63) >> 6;                                 // pages a token can have
    if (p.window > 0) mp = std::min(mp, ((p.window + 62) >> 6) + 1);
    int gt = p.G >= 3 ? 4 : p.G, S = 1;
    const int Tc = std::min(p.T, 65535);
    auto units = [&]() { return (long long)Tc * a.n_kv * ((p.G + gt - 1) / gt); };
    auto cap = [&]() { return ((mp + S - 1) / S) << 6; };
    while (S < di.max_cluster && units() * 2 * S <= 2 * di.sms && mp >= 8 * S) S <<= 1;
    while (S < di.max_cluster && weigh_smem(gt, cap()) > weigh_room(gt, 2)) S <<= 1;
    while (gt > 1 && weigh_smem(gt, cap()) > weigh_room(gt, 1)) gt >>= 1;
    p.cap = cap();
    if (weigh_smem(gt, p.cap) > weigh_room(gt, 1)) return cudaErrorNotSupported;
    p.smul = ((1ull << 32) + S - 1) / S;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 1 : 0;
    cfg.stream = s;
    cfg.blockDim = dim3(KV4_DT);
    cfg.dynamicSmemBytes = weigh_smem(gt, p.cap);
    for (p.t0 = 0; p.t0 < p.T; p.t0 += 65535) {
        cfg.gridDim = dim3(S, a.n_kv * ((p.G + gt - 1) / gt), std::min(65535, p.T - p.t0));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, WEIGH[d == 128][lg2(gt)], a, p, w);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_weigh_block(const DevInfo& di, const Kv4Args& a, Kv4Attn p, const Kv4Weigh& w, int d, cudaStream_t s) {
    p.none = KV4_NEG;
    // few tokens: one wave of the single-token form, whose keys are spread over more
    // CTAs (4 sequences of 16 tokens after 1000, 16 + 8 heads of 128: 13.3 us, 18.7 in
    // blocks; 32 after 4000 17.0 and 19.7; 183 after 8000, 32 + 8 of 64: 143 and 118)
    if ((long long)p.T * a.n_kv * ((p.G + 3) / 4) <= 4LL * di.sms) return launch_weigh(di, a, p, w, d, s);
    int mp = (p.max_len + 63) >> 6;                                 // pages a token can have, and one for its neighbours
    if (p.window > 0) mp = std::min(mp, ((p.window + 62) >> 6) + 2);
    // CTAs of 4 warps while 16 of them hold the pages (1 x 4096 tokens, 16 + 8 heads
    // of 128: 463 us, with 8 warps 477, with 16 524; 1 x 1000 34, 44 and 66), then of
    // 8 (512 after 16000 631, with 16 737); past a bound of 32768 keys the scores are
    // not kept at once, and each token goes by itself (512 after 30000 972 us, after
    // 40000 1780)
    p.lgC = 0;
    int nw = 4;
    while (mp > (nw * WB_PG) << p.lgC && (2 << p.lgC) <= di.max_cluster) ++p.lgC;
    if (mp > (nw * WB_PG) << p.lgC) nw = 8;
    if (mp > (nw * WB_PG) << p.lgC) return launch_weigh(di, a, p, w, d, s);
    p.lgGp = 0;
    while (p.lgGp < 4 && (1 << p.lgGp) < p.G) ++p.lgGp;
    const int bq = WB_ROWS >> p.lgGp, hg = (p.G + (1 << p.lgGp) - 1) >> p.lgGp, tiles = (p.T + bq - 1) / bq;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1 << p.lgC;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.lgC ? 1 : 0;
    cfg.stream = s;
    cfg.blockDim = dim3(32 * nw);
    cfg.dynamicSmemBytes = (WB_SMEM + (WB_EXCH << p.lgC)) * nw;      // (a round may have more pages than a token)
    for (int b0 = 0; b0 < tiles; b0 += 65535) {
        p.t0 = b0 * bq;
        cfg.gridDim = dim3(1 << p.lgC, a.n_kv * hg, std::min(65535, tiles - b0));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, WEIGH_BLOCK[d == 128][nw == 8], a, p, w);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_evict(const DevInfo& di, const Kv4Args& a, Kv4Evict p, int n, int d, cudaStream_t s) {
    const int mp = (p.max_len + 63) >> 6;
    int lg = 0;
    auto pages = [&]() { return (mp + (1 << lg) - 1) >> lg; };
    // CTAs of 32 pages or less while there are few of them (4 sequences of 8192
    // keys, 8 kv heads: 22.4 us, with 8 CTAs 23.4; 16 of up to 32768 98 with 4, with
    // 2 112, with 8 107; 32 of 4096 48 with 2, with one 45), 16 of them only for long
    // contexts (1 of 32768: 27.8 with 8, with 16 32)
    while ((2 << lg) <= di.max_cluster &&
           (pages() > EV_PAGES || (pages() > (lg < 3 ? 32 : 128) && ((long long)n * a.n_kv << (lg + 1)) * 2 <= 7LL * di.sms)))
        ++lg;
    p.lg_s = lg;
    const size_t bytes = (size_t)pages() * KV_BLK * 8;
    p.held = bytes <= EV_HELD;
    if (pages() > EV_PAGES) return cudaErrorNotSupported;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1 << lg;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = lg ? 1 : 0;
    cfg.stream = s;
    cfg.gridDim = dim3(n << lg, a.n_kv);
    // 256 threads where two CTAs of 512 per SM would not hold all and a CTA has few
    // pages, as the phases' latencies then overlap (8 sequences of 16384 keys, 8 kv
    // heads: 42 us, with 512 48; 256 of 700 78 and 87; 16 of up to 32768, 128 pages
    // a CTA: 104, with 512 98). The move starts while the selection drains only where
    // an SM has one CTA of it: past that its CTAs would find the SMs set to much
    // shared memory and little L1 (16 of up to 32768: 98 us, then 123; 1 of 4097:
    // 16.3, after it 16.7)
    const long long ctas = (long long)n * a.n_kv << lg;
    const bool small = pages() <= 32 && ctas > 2LL * di.sms;
    cfg.blockDim = dim3(small ? 256 : 512);
    cfg.dynamicSmemBytes = p.held ? bytes : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, EV_SELECT[!small], a, p);
    if (e != cudaSuccess) return e;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = ctas <= di.sms;
    cfg.gridDim = dim3(p.new_blocks, a.n_kv, n);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, d == 128 ? k_kv4_evict_move<128> : k_kv4_evict_move<64>, a, p);
}

}  // namespace
}  // namespace detint

using namespace detint;

namespace {

int weigh(const char* where, bool block, const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
          const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window, int64_t* weight, detint_stream_t sp) {
    Kv4Args a{};
    Kv4Attn p{};
    if (!weight || mis(weight, 16)) return failed(DETINT_E_ARG, where, "a 16-byte aligned weight array is needed");
    // (no output rows: the weights stand in for them in the shared checks)
    const int rc = check_attn(where, c, q8, mq, kq, tok_seq, tok_pos, n_tok, max_len, window, (int32_t*)weight,
                              c ? (long long)c->n_q * c->head_dim : 0, &a, &p);
    if (rc) return rc;
    Kv4Weigh w{};
    w.weight = (long long*)weight;
    DevInfo* di = nullptr;
    cudaError_t e = init(&di);
    if (e == cudaSuccess) e = (block ? launch_weigh_block : launch_weigh)(*di, a, p, w, c->head_dim, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

}  // namespace

extern "C" {

int detint_kv4_weigh(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq, const int32_t* tok_seq,
                     const int32_t* tok_pos, int n_tok, int max_len, int window, int64_t* weight, detint_stream_t sp) {
    return weigh("detint_kv4_weigh", false, c, q8, mq, kq, tok_seq, tok_pos, n_tok, max_len, window, weight, sp);
}

int detint_kv4_weigh_block(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq, const int32_t* tok_seq,
                           const int32_t* tok_pos, int n_tok, int max_len, int window, int64_t* weight, detint_stream_t sp) {
    return weigh("detint_kv4_weigh_block", true, c, q8, mq, kq, tok_seq, tok_pos, n_tok, max_len, window, weight, sp);
}

int detint_kv4_evict(const detint_kv4_t* c, int64_t* weight, const int32_t* seq, const int32_t* lens, int n, int max_len,
                     int keep, int sinks, int recent, const int32_t* new_table, int32_t* kept, detint_stream_t sp) {
    const char* where = "detint_kv4_evict";
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    Kv4Args a{};
    const int rc = check_cache(where, c, &a);
    if (rc) return rc;
    if (!weight || !seq || !lens || !new_table || !kept) return err(DETINT_E_ARG, "null pointer");
    if (n < 1 || n > 65535) return err(DETINT_E_ARG, "n must be in 1..65535");
    if (max_len < 1 || max_len > KV4_MAX_LEN) return err(DETINT_E_ARG, "max_len must be in 1..524288");
    if (keep < 1 || keep > KV4_MAX_LEN) return err(DETINT_E_ARG, "keep must be in 1..524288");
    if (sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks) return err(DETINT_E_ARG, "sinks and recent must fit keep");
    if (mis(weight, 16) || mis(seq, 4) || mis(lens, 4) || mis(new_table, 4) || mis(kept, 4))
        return err(DETINT_E_ARG, "weights must be 16-byte, the other arrays 4-byte aligned");
    Kv4Evict p{};
    p.weight = (long long*)weight;
    p.seq = seq; p.lens = lens; p.new_table = new_table; p.kept = kept;
    p.max_len = max_len; p.keep = keep; p.sinks = sinks; p.recent = recent;
    p.new_blocks = (keep + KV_BLK - 1) / KV_BLK;
    DevInfo* di = nullptr;
    cudaError_t e = init(&di);
    if (e == cudaSuccess) e = launch_evict(*di, a, p, n, c->head_dim, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

int detint_kv4_copy(const detint_kv4_t* c, const int32_t* src, const int32_t* dst, int n, int64_t* weight, detint_stream_t sp) {
    const char* where = "detint_kv4_copy";
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    Kv4Args a{};
    const int rc = check_cache(where, c, &a);
    if (rc) return rc;
    if (!src || !dst) return err(DETINT_E_ARG, "null pointer");
    if (n < 1) return err(DETINT_E_ARG, "n must be positive");
    if (mis(src, 4) || mis(dst, 4) || mis(weight, 16)) return err(DETINT_E_ARG, "lists must be 4-byte, weights 16-byte aligned");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;       // starts while detint_beam_reorder drains
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.stream = (cudaStream_t)sp;
    cfg.gridDim = dim3(n, a.n_kv);
    cfg.blockDim = dim3(256);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv4_copy, a, src, dst, KV_BLK * c->head_dim / 2, (long long*)weight);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

}  // extern "C"
