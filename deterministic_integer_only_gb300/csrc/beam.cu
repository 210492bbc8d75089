// Host side of beam search: launch shapes, argument checks and the C entry
// points detint_beam_*. Kernel code lives in k_beam.cuh.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "../../include/detint.h"
#include "k_beam.cuh"
#include "kv4_check.h"

namespace detint {

namespace {

struct DevInfo {
    bool ready = false;
    int sms = 0;
    int lg_max = 3;                      // log2 of the CTAs of the largest cluster
};
DevInfo g_dev[64];
std::mutex g_mu;

using RowsFn = void (*)(BeamArgs);
constexpr int NQ = 6;
constexpr int QUADS[NQ] = {1, 2, 4, 5, 8, 10};
template <bool VEC>
RowsFn rows_of(int i) {
    static const RowsFn f[NQ + 1] = {k_beam_rows<1, true, VEC>, k_beam_rows<2, true, VEC>, k_beam_rows<4, true, VEC>,
                                     k_beam_rows<5, true, VEC>, k_beam_rows<8, true, VEC>, k_beam_rows<10, true, VEC>,
                                     k_beam_rows<8, false, VEC>};
    return f[i];
}

cudaError_t init(DevInfo** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    DevInfo* di = *out = &g_dev[dev];
    std::lock_guard<std::mutex> lk(g_mu);
    if (di->ready) return cudaSuccess;
    e = cudaDeviceGetAttribute(&di->sms, cudaDevAttrMultiProcessorCount, dev);
    int lg = 4;
    for (int i = 0; i <= NQ; ++i)
        for (int v = 0; v < 2 && e == cudaSuccess; ++v) {
            const RowsFn f = v ? rows_of<true>(i) : rows_of<false>(i);
            e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 16;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(BM_THREADS);
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (e == cudaSuccess && (cudaOccupancyMaxActiveClusters(&n, f, &cfg) != cudaSuccess || n < 1)) {
                cudaGetLastError();
                lg = 3;
            }
        }
    if (e == cudaSuccess) {
        di->lg_max = lg;
        di->ready = true;
    }
    return e;
}

size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

cudaError_t launch_select(const DevInfo& di, BeamArgs a, int groups, cudaStream_t s) {
    const int quads = (a.n + 3) / 4;
    int lg = 0;
    while (lg < di.lg_max && quads > BM_THREADS << lg && ((long long)a.rows << (lg + 1)) <= 4LL * di.sms) ++lg;
    while (lg < di.lg_max && quads > (QUADS[NQ - 1] * BM_THREADS) << lg) ++lg;
    int i = 0;
    while (i < NQ && quads > (QUADS[i] * BM_THREADS) << lg) ++i;
    const int entries = BM_WARPS << lg;
    a.lg_cl = lg;
    a.lg_groups = 0;
    while ((1 << a.lg_groups) < a.n_out && (1 << a.lg_groups) < entries) ++a.lg_groups;
    a.per_warp = (a.n_out + entries - 1) / entries;
    const bool vec = !(a.stride & 3) && !mis(a.logits, 16);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.attrs = at;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1 << lg;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(a.rows << lg);
    cfg.blockDim = dim3(BM_THREADS);
    cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? rows_of<true>(i) : rows_of<false>(i), a);
    if (e != cudaSuccess) return e;
    // starts while the rows' launch drains
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(groups);
    cfg.blockDim = dim3(BM_MERGE_THREADS);
    cfg.dynamicSmemBytes = (size_t)a.beams * a.n_out * 8;
    return cudaLaunchKernelEx(&cfg, k_beam_merge, a);
}

constexpr int MAX_VOCAB = 1 << 24;           // the sum of a row's exponentials stays below 2^55
constexpr int MAX_ROWS = 1 << 20;

}  // namespace
}  // namespace detint

using namespace detint;

extern "C" {

int detint_beam_workspace(int rows, int n, int n_out, long long* bytes) {
    if (!bytes || rows < 1 || rows > MAX_ROWS || n < 1 || n > MAX_VOCAB || n_out < 1 || n_out > BM_MAX_OUT)
        return failed(DETINT_E_ARG, "detint_beam_workspace", "bad arguments");
    *bytes = (long long)(a256((size_t)rows * n_out * 8) + a256((size_t)rows * n_out * 4));
    return DETINT_OK;
}

int detint_beam_select(const int32_t* logits, long long stride, int n, const int64_t* scores, const int32_t* done,
                       int groups, int beams, int end_id, int n_out, int32_t* parent, int32_t* token, int64_t* score,
                       int32_t* done_out, void* workspace, long long workspace_bytes, detint_stream_t sp) {
    const char* where = "detint_beam_select";
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    if (!logits || !scores || !parent || !token || !score || !done_out) return err(DETINT_E_ARG, "null pointer");
    if (groups < 1 || beams < 1 || beams > BM_MAX_OUT) return err(DETINT_E_ARG, "groups must be positive, beams in 1..64");
    if (n_out < 1 || n_out > BM_MAX_OUT) return err(DETINT_E_ARG, "n_out must be in 1..64");
    if ((long long)groups * beams > MAX_ROWS) return err(DETINT_E_ARG, "more than 2^20 rows");
    if (n < 1 || n > MAX_VOCAB) return err(DETINT_E_SHAPE, "a row must have 1..2^24 logits");
    if (stride < n) return err(DETINT_E_ARG, "the stride must hold a row");
    if (end_id < -1 || end_id >= n || (done && end_id < 0)) return err(DETINT_E_ARG, "end_id must be a token, or -1 without done");
    if (mis(logits, 4) || mis(done, 4) || mis(parent, 4) || mis(token, 4) || mis(done_out, 4) || mis(scores, 8) || mis(score, 8))
        return err(DETINT_E_ARG, "misaligned array");
    long long need = 0;
    const int rc = detint_beam_workspace(groups * beams, n, n_out, &need);
    if (rc) return rc;
    if (!workspace || workspace_bytes < need || mis(workspace, 16))
        return err(DETINT_E_ARG, "a 16-byte aligned workspace of detint_beam_workspace bytes is needed");
    BeamArgs a{};
    a.logits = logits; a.stride = (size_t)stride; a.scores = (const long long*)scores; a.done = done;
    a.rows = groups * beams; a.n = n; a.n_out = n_out; a.end_id = end_id; a.beams = beams;
    a.ws_score = (long long*)workspace;
    a.ws_tok = (int32_t*)((unsigned char*)workspace + a256((size_t)a.rows * n_out * 8));
    a.parent = parent; a.token = token; a.done_out = done_out; a.score_out = (long long*)score;
    DevInfo* di = nullptr;
    cudaError_t e = init(&di);
    if (e == cudaSuccess) e = launch_select(*di, a, groups, (cudaStream_t)sp);
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

int detint_beam_reorder(const int32_t* block_table, int32_t* out, int max_blocks, const int32_t* parent, const int32_t* lens,
                        int groups, int beams, int32_t* src, int32_t* dst, detint_stream_t sp) {
    const char* where = "detint_beam_reorder";
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    if (!block_table || !out || !parent || !lens || !src || !dst) return err(DETINT_E_ARG, "null pointer");
    if (groups < 1 || groups > 65535 || beams < 1 || beams > BM_MAX_OUT) return err(DETINT_E_ARG, "groups must be in 1..65535, beams in 1..64");
    if (max_blocks < 1) return err(DETINT_E_ARG, "max_blocks must be positive");
    if (mis(block_table, 4) || mis(out, 4) || mis(parent, 4) || mis(lens, 4) || mis(src, 4) || mis(dst, 4))
        return err(DETINT_E_ARG, "arrays must be 4-byte aligned");
    k_beam_reorder<<<dim3((max_blocks + BR_COLS - 1) / BR_COLS, groups), BR_THREADS, 0, (cudaStream_t)sp>>>(
        block_table, out, parent, lens, beams, max_blocks, src, dst);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

}  // extern "C"
