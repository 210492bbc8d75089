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

int g_sms[64];                               // 0: not set up yet
std::mutex g_mu;

// scores and tokens of the beams' lists, then a list per warp
size_t merge_smem(int beams, int n_out) { return (((size_t)beams * n_out * 12 + 15) & ~(size_t)15) + (size_t)std::min(beams, BM_MERGE_NW) * BM_CAP * 8; }

// sets the kernels' attributes once per device (no call that a stream capture forbids)
cudaError_t init(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    if ((*sms = g_sms[dev])) return cudaSuccess;
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_beam_merge, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)merge_smem(BM_MAX_OUT, BM_MAX_OUT));
    if (e == cudaSuccess) *sms = g_sms[dev] = n;
    return e;
}

size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

struct WsLayout { size_t part_key, key, sum, list, top, most, count, total; };
WsLayout ws_layout(size_t rows) {
    // (of the most parts that a row can have: enough for shorter rows too)
    WsLayout w{};
    size_t o = 0;
    w.part_key = o; o += a256(rows * BM_PARTS * 8);
    w.key = o; o += a256(rows * BM_PARTS * BM_NW * 8);
    w.sum = o; o += a256(rows * BM_PARTS * 8);
    w.list = o; o += a256(rows * BM_CAP * 8);
    w.top = o; o += a256(rows * BM_PARTS * 4);
    w.most = o; o += a256(rows * 4);
    w.count = o; o += a256(rows * 4);
    w.total = o;
    return w;
}

cudaError_t launch_select(BeamArgs a, int groups, int sms, cudaStream_t s) {
    const int all = (a.n + BM_ROUND - 1) / BM_ROUND;
    // parts: up to 6 CTAs per SM, of which 4 of k_beam_sum run at a time, so that
    // what a CTA does once is not done too often (24 x 5 rows of 128256 logits:
    // 28.7 us, with 12 30.6, with 24 39; with 4 29.7)
    int most = BM_PARTS;
    while (most > 1 && (long long)groups * a.beams * std::min(most, all) > 6LL * sms) --most;
    a.rounds = (all + most - 1) / most;
    a.parts = (all + a.rounds - 1) / a.rounds;
    // entries that the n_out-th largest value is looked for among: twice as many
    // as continuations, so that the bound is well above their least
    a.per_part = a.parts >= 2 * a.n_out ? a.n_out : 0;
    a.lanes = std::min(32, (2 * a.n_out + a.parts * BM_NW - 1) / (a.parts * BM_NW));
    a.per_warp = (a.n_out + a.lanes - 1) / a.lanes;
    const bool vec = !(a.stride & 3) && !mis(a.logits, 16);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.stream = s;
    cfg.gridDim = dim3(a.parts, groups * a.beams);
    cfg.blockDim = dim3(BM_NT);
    cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? k_beam_top<true> : k_beam_top<false>, a);
    cfg.numAttrs = 1;                                    // the others start while the one before drains
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, vec ? k_beam_sum<true> : k_beam_sum<false>, a);
    cfg.gridDim = dim3(groups);
    cfg.blockDim = dim3(BM_MERGE);
    cfg.dynamicSmemBytes = merge_smem(a.beams, a.n_out);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k_beam_merge, a);
    return e;
}

constexpr int MAX_VOCAB = 1 << 24;           // the sum of a row's exponentials stays below 2^55
constexpr int MAX_ROWS = 65535;

}  // namespace

cudaError_t launch_copy_blocks(const BlockParts& b, const int* src, const int* dst, int n, cudaStream_t s) {
    for (int i = 0; i < n; i += CB_PAIRS) {
        BlockPairs p{};
        const int m = std::min(n - i, CB_PAIRS);
        std::copy(src + i, src + i + m, p.src);
        std::copy(dst + i, dst + i + m, p.dst);
        k_copy_blocks<<<dim3(m, b.parts * b.layers), 256, 0, s>>>(b, p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace detint

using namespace detint;

extern "C" {

int detint_beam_workspace(int rows, int n, int n_out, long long* bytes) {
    if (!bytes || rows < 1 || rows > MAX_ROWS || n < 1 || n > MAX_VOCAB || n_out < 1 || n_out > BM_MAX_OUT)
        return failed(DETINT_E_ARG, "detint_beam_workspace", "bad arguments");
    *bytes = (long long)ws_layout((size_t)rows).total;
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
    if ((long long)groups * beams > MAX_ROWS) return err(DETINT_E_ARG, "more than 65535 rows");
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
    // (a group's outputs are written while others' inputs are still read)
    const size_t rows = (size_t)groups * beams, outs = (size_t)groups * n_out;
    const Span written[] = {{parent, outs * 4}, {token, outs * 4}, {score, outs * 8}, {done_out, outs * 4}, {workspace, (size_t)need}};
    const Span read[] = {{logits, ((rows - 1) * (size_t)stride + n) * 4}, {scores, rows * 8}, {done, rows * 4}};
    if (clash(written, read)) return err(DETINT_E_ARG, "an output or the workspace overlaps another array of the call");
    BeamArgs a{};
    a.logits = logits; a.stride = (size_t)stride; a.scores = (const long long*)scores; a.done = done;
    a.n = n; a.n_out = n_out; a.end_id = end_id; a.beams = beams;
    unsigned char* ws = (unsigned char*)workspace;
    const WsLayout w = ws_layout((size_t)groups * beams);
    a.part_key = (unsigned long long*)(ws + w.part_key);
    a.key = (unsigned long long*)(ws + w.key);
    a.sum = (unsigned long long*)(ws + w.sum);
    a.list = (unsigned long long*)(ws + w.list);
    a.top = (int32_t*)(ws + w.top);
    a.most = (int32_t*)(ws + w.most);
    a.count = (unsigned*)(ws + w.count);
    a.parent = parent; a.token = token; a.done_out = done_out; a.score_out = (long long*)score;
    int sms = 0;
    cudaError_t e = init(&sms);
    if (e == cudaSuccess) e = launch_select(a, groups, sms, (cudaStream_t)sp);
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
    const size_t rows = (size_t)groups * beams, cells = rows * (size_t)max_blocks;
    const Span written[] = {{out, cells * 4}, {src, rows * 4}, {dst, rows * 4}};
    const Span read[] = {{out == block_table ? nullptr : block_table, cells * 4}, {parent, rows * 4}, {lens, (size_t)groups * 4}};
    if (clash(written, read)) return err(DETINT_E_ARG, "out (unless it is block_table itself), src or dst overlaps another array of the call");
    k_beam_reorder<<<dim3((max_blocks + BR_COLS - 1) / BR_COLS, groups), BR_THREADS, 0, (cudaStream_t)sp>>>(
        block_table, out, parent, lens, beams, max_blocks, src, dst);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DETINT_OK : cuda_fail(where, e);
}

}  // extern "C"
