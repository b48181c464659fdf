// Host side of the MegaMoE C ABI: argument checks, workspace carving and the
// launch order of the stages on one stream.  The order is the stage overview
// of the pto-isa MegaMoE overview page: FrontReorder, (Dispatch), GMM1,
// SwiGLU, GMM2, (Combine), Unpermute.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "../../include/megamoe.h"
#include "../../include/megamoe/half.h"
#include "half.hpp"
#include "kernels.hpp"


using namespace megamoe;

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kErrBytes = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// The four large intermediates start on 2 MiB boundaries, as separate device
// allocations of their size would.
constexpr size_t kBigAlign = 2u << 20;
size_t align_big(size_t v) { return (v + kBigAlign - 1) / kBigAlign * kBigAlign; }

bool aligned16(const void *p) { return p && ((uintptr_t)p & 15u) == 0; }

// CU count of the current device, queried once per device.  It only sizes the
// persistent GEMM grid, so a failed query falls back to MI355X's 256.  The
// cache is filled with relaxed atomics: concurrent first calls store the same
// value.
int cu_count_current() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Scratch of megamoe_permute_noalloc: the sort's per-block expert counts.
// The sort uses at most 256 blocks of routes and at most 256 experts, so
// 256 x 256 counts cover every shape megamoe_check_dims accepts.  Each GPU the
// library runs on holds its own copy until the process ends.  In host code
// the name `scratch` is only a stand-in for the symbol: its device address
// comes from hipGetSymbolAddress (scratch_device_ptr below).
constexpr size_t kNoAllocScratchBytes = 256u * 256u * sizeof(int32_t);
static __device__ __align__(256) int32_t scratch[kNoAllocScratchBytes / sizeof(int32_t)];

// Device address of `scratch` on the current device, looked up once per
// device with that device current (concurrent first calls store the same
// value).  nullptr if the HIP calls fail.
int32_t *scratch_device_ptr() {
    static std::atomic<int32_t *> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
    int32_t *p = cached[dev].load(std::memory_order_acquire);
    if (p == nullptr) {
        void *addr = nullptr;
        if (hipGetSymbolAddress(&addr, HIP_SYMBOL(scratch)) != hipSuccess || addr == nullptr)
            return nullptr;
        p = static_cast<int32_t *>(addr);
        cached[dev].store(p, std::memory_order_release);
    }
    return p;
}

struct Layout {
    size_t err, bcnt, tscale, tsync, tdone, eri, sorted, counts, cumsum, pts1, pts2, prow, gmA,
        gmC, q2, g2, ks, total;
};

// permute workspace: error word, the sort's per-block expert counts, then the
// per-token scales of the token-major path
size_t permute_ws_bytes(const megamoe_dims &d) {
    return align_up(kErrBytes) + align_up(route_sort_workspace_bytes(d.M * d.top_k, d.E)) +
           align_up((size_t)d.M * 4);
}

// GMM1's K-split buffer (megamoe_gmm1_gather_split): the tile counters, then
// the partial tiles
constexpr size_t kSplitCountBytes = (kKsCounters * 4 + 255) / 256 * 256;
size_t split_ws_bytes() { return kSplitCountBytes + (size_t)kKsMaxTiles * 4 * kKsPartBytes; }

// bytes of q2 in the row-paired layout: each expert's rows padded to an even
// count, at most R + E rows
size_t paired_q2_bytes(const megamoe_dims &d) {
    return ((size_t)d.M * d.top_k + d.E + 1) * d.I;
}

Layout forward_layout(const megamoe_dims &d) {
    const size_t R = (size_t)d.M * d.top_k;
    Layout L;
    size_t o = 0;
    L.err = o;    o += align_up(kErrBytes);
    L.bcnt = o;   o += align_up(route_sort_workspace_bytes((int)R, d.E));
    L.tscale = o; o += align_up((size_t)d.M * 4);
    L.tsync = o;  o += align_up(kSyncWords * 4);
    L.tdone = o;  o += align_up(R);
    L.eri = o;    o += align_up(R * 4);
    L.sorted = o; o += align_up(R * 4);
    L.counts = o; o += align_up((size_t)d.E * 4);
    L.cumsum = o; o += align_up((size_t)d.E * 4);
    L.pts1 = o;   o += align_up(R * 4);
    L.pts2 = o;   o += align_up(R * 4);
    L.prow = o;   o += align_up(R * 4);
    o = align_big(o);
    L.gmA = o;    o = align_big(o + (size_t)d.M * d.K);   // token-major quantised x
    L.gmC = o;    o = align_big(o + R * 2 * d.I * 2);
    // q2, row-paired when GMM2 uses the 256-row tiles: each expert's rows are
    // padded to an even count, at most R + E rows
    L.q2 = o;     o = align_big(o + paired_q2_bytes(d));
    L.g2 = o;     o = align_big(o + R * d.K * 2);
    // GMM1's partial tiles when its sparse last round splits tiles over K
    L.ks = o;     o += (size_t)kKsMaxTiles * 4 * kKsPartBytes;
    L.total = o;
    return L;
}

int hip_status(hipError_t e) { return e == hipSuccess ? MEGAMOE_OK : MEGAMOE_EHIP; }

#define MEGAMOE_TRY(expr)                         \
    do {                                          \
        const int _rc = (expr);                   \
        if (_rc != MEGAMOE_OK) return _rc;        \
    } while (0)

// token_major: gmA is [M, K] (row t = quantised token t) rather than the
// expert-sorted [R, K]; the fused forward reads it through the route list.
// tscale [M] (token_major only): scratch for the per-token scales when the
// quantisation runs beside the sort's first pass.
// tail_done / tail_sync (nullable, forward only): flags of the GMM1 that
// follows, cleared by the permute's kernels.
int run_permute(const megamoe_dims &d, const uint16_t *x, const int32_t *expert_idx, int8_t *gmA,
                float *pts1, int32_t *eri, int32_t *sorted, int32_t *counts, int32_t *cumsum,
                int32_t *err_word, int32_t *block_counts, bool token_major, hipStream_t s,
                float *tscale = nullptr, uint8_t *tail_done = nullptr,
                uint32_t *tail_sync = nullptr, int32_t *prow = nullptr) {
    const int R = d.M * d.top_k;
    if (permute_fused_ok(R, d.top_k))
        return hip_status(launch_permute_fused(x, expert_idx, d.M, d.K, d.E, d.top_k, gmA, pts1, eri,
                                               sorted, counts, cumsum, err_word, token_major, s,
                                               tail_done, tail_sync, prow));
    if (token_major && tscale)
        return hip_status(launch_permute_tokens_2pass(x, expert_idx, d.M, d.K, d.E, d.top_k, gmA,
                                                      pts1, eri, sorted, counts, cumsum, err_word,
                                                      block_counts, tscale, s, tail_done,
                                                      tail_sync, prow));
    MEGAMOE_TRY(hip_status(launch_route_sort(expert_idx, R, d.E, sorted, eri, counts, cumsum,
                                             err_word, block_counts, s)));
    return hip_status(
        launch_quant_scatter(x, eri, d.M, d.K, d.top_k, gmA, pts1, token_major, s));
}

// a_route (nullable): A row d is token a_route[d] / top_k of a token-major A.
// tail (nullable, GMM1 only): SwiGLU in GMM1's last round (tail_*) or the
// K-split last round (ks_*), see gmm.hip.
// a_pair: A is in the row-paired layout (GmmParams::a_pair).
int run_gmm(const megamoe_dims &d, const int8_t *A, const int32_t *cumsum, const int8_t *Bp,
            const float *scale, uint16_t *C, int32_t *dbg, int N, int Kred, hipStream_t s,
            const int32_t *a_route = nullptr, const GmmParams *tail = nullptr,
            bool a_pair = false) {
    const int R = d.M * d.top_k;
    GmmParams prm{A, Bp, scale, cumsum, C, dbg, d.E, N, Kred, a_route, d.top_k};
    prm.a_pair = a_pair ? 1 : 0;
    if (tail) {
        prm.tail_q2 = tail->tail_q2;
        prm.tail_pts2 = tail->tail_pts2;
        prm.tail_pts1 = tail->tail_pts1;
        prm.tail_sync = tail->tail_sync;
        prm.tail_done = tail->tail_done;
        prm.tail_I = tail->tail_I;
        prm.tail_spin = tail->tail_spin;
        prm.tail_prow = tail->tail_prow;
        prm.ks_part = tail->ks_part;
        prm.ks_count = tail->ks_count;
    }
    return hip_status(launch_gmm(gmm_pick_variant(R, d.E), prm, R, cu_count_current(), s));
}

// megamoe_set_overlap: 0 (default) GMM1 then SwiGLU; 1 SwiGLU overlaps
// GMM1's last round; 2 as 1, with every waiting workgroup giving up at once.
// Measured on MI355X the overlap is slower (the device-scope L2 write-back it
// needs, and its HBM traffic beside the last-round tiles, cost more than the
// SwiGLU time it hides), so it is off unless asked for.
std::atomic<int> g_overlap{0};
// poll limit of the wait (each poll is a device-scope load and a short
// sleep): a workgroup gives up after milliseconds, long after every resident
// workgroup has arrived (one tile takes at most a few hundred microseconds)
constexpr int kTailSpin = 8192;

int permute_entry(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                  int8_t *gmA, float *pts1, int32_t *eri, int32_t *sorted_route,
                  int32_t *tokens_per_expert, int32_t *expert_cumsum, void *ws, size_t ws_bytes,
                  bool token_major, void *stream, int32_t *prow = nullptr) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, expert_idx, gmA, pts1, eri, sorted_route, tokens_per_expert,
                          expert_cumsum, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (prow && !aligned16(prow)) return MEGAMOE_EINVAL;
    if (ws_bytes < permute_ws_bytes(*d)) return MEGAMOE_EWORKSPACE;
    char *w = (char *)ws;
    const size_t bcnt = align_up(kErrBytes);
    const size_t tsc = bcnt + align_up(route_sort_workspace_bytes(d->M * d->top_k, d->E));
    return run_permute(*d, x, expert_idx, gmA, pts1, eri, sorted_route, tokens_per_expert,
                       expert_cumsum, (int32_t *)w, (int32_t *)(w + bcnt), token_major,
                       (hipStream_t)stream, (float *)(w + tsc), nullptr, nullptr, prow);
}

static_assert(kFp32 == MEGAMOE_FP32 && kFp16 == MEGAMOE_FP16 && kBf16 == MEGAMOE_BF16,
              "the kernels' element types are the header's");

bool type_ok(int type) {
    return type == MEGAMOE_FP32 || type == MEGAMOE_FP16 || type == MEGAMOE_BF16;
}

// workspace of the few-token layer: the dropped-route word, y, its 16-column maxima
struct FewLayout {
    size_t y, ymax, total;
};
FewLayout few_layout(const megamoe_dims &d) {
    const size_t R = (size_t)d.M * d.top_k;
    FewLayout L;
    L.y = align_up(kErrBytes);
    L.ymax = L.y + align_up(R * d.I * 4);
    L.total = L.ymax + align_up(R * (d.I / 16) * 4);
    return L;
}

int check_few(const megamoe_dims *d) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    return few_ok(d->M, d->top_k) ? MEGAMOE_OK : MEGAMOE_EUNSUPPORTED;
}

// workspace of the MXFP4 forward
struct Mxfp4Layout {
    size_t err, bcnt, eri, sorted, counts, cumsum, xq, xs, yq, ys, g2, total;
};
Mxfp4Layout mxfp4_layout(const megamoe_dims &d) {
    const size_t M = d.M, K = d.K, I = d.I, R = M * d.top_k;
    Mxfp4Layout L;
    size_t o = 0;
    L.err = o;    o += align_up(kErrBytes);
    L.bcnt = o;   o += align_up(route_sort_workspace_bytes((int)R, d.E));
    L.eri = o;    o += align_up(R * 4);
    L.sorted = o; o += align_up(R * 4);
    L.counts = o; o += align_up((size_t)d.E * 4);
    L.cumsum = o; o += align_up((size_t)d.E * 4);
    L.xq = o;     o += align_up(M * (K / 2));
    L.xs = o;     o += align_up(M * (K / 32));
    L.yq = o;     o += align_up(R * (I / 2));
    L.ys = o;     o += align_up(R * (I / 32));
    L.g2 = o;     o += align_up(R * K * 2);
    L.total = o;
    return L;
}

int run_mxfp4_gmm(const megamoe_dims &d, const uint8_t *a, const uint8_t *as, const int32_t *route,
                  const int32_t *cumsum, const uint8_t *w, const uint8_t *ws, uint16_t *c,
                  uint8_t *cq, uint8_t *cs, bool first, hipStream_t s) {
    const MxGmmParams p{a, as, w, ws, route, cumsum, c, cq, cs, d.M * d.top_k, d.E,
                        first ? d.I : d.K, first ? d.K : d.I, d.top_k,
                        // the high product exceeds route / top_k by route * e / (top_k 2^32) with
                        // e < top_k <= 256 and route < 2^24: by less than a step of 1 / top_k
                        (uint32_t)(((1ull << 32) + d.top_k - 1) / d.top_k)};
    return hip_status(launch_mxfp4_gmm(p, first, cu_count_current(), s));
}

// rows of MXFP4: whole blocks, and a grid below 2^32 threads
int check_mxfp4_rows(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1) return MEGAMOE_EINVAL;
    if (cols % 32 != 0 || cols > (1ll << 24) || rows > (1ll << 36) / cols)
        return MEGAMOE_EUNSUPPORTED;
    return MEGAMOE_OK;
}

bool half_type(int type) { return type == MEGAMOE_FP16 || type == MEGAMOE_BF16; }

// gather: 0, or which operand's rows are token rows read through `route`.
int run_half_gmm(const megamoe_dims &d, int kind, bool first, const uint16_t *a, const uint16_t *b,
                 int type, const int32_t *route, int gather, const int32_t *cumsum,
                 const float *probs, bool swiglu, void *c, int c_type, bool accumulate,
                 hipStream_t s) {
    const int inner = first && !swiglu ? 2 * d.I : d.I, wide = first ? 2 * d.I : d.I;
    // the reciprocal: see run_mxfp4_gmm
    HalfGmmParams p{a, b, route, cumsum, probs, c, d.M * d.top_k, d.E, 0, 0, 0, d.top_k,
                    d.top_k == 1 ? 0 : (uint32_t)(((1ull << 32) + d.top_k - 1) / d.top_k),
                    d.top_k == 1 ? ~0u : 0u, gather, swiglu, accumulate, c_type};
    if (kind == kHalfWeights) {
        p.M = first ? wide : d.K;
        p.N = first ? d.K : wide;
    } else {  // the first product and the second's row gradient end in the inner columns
        const bool to_inner = first == (kind == kHalfProduct);
        p.N = to_inner ? inner : d.K;
        p.K = to_inner ? d.K : inner;
    }
    return hip_status(launch_half_gmm(p, kind, type, cu_count_current(), s));
}

// The weights' gradients look past a group's end by less than 64 rows, at byte offsets below 2^32.
bool half_wgrad_ok(const megamoe_dims &d) {
    const long long wide = d.K > 2 * d.I ? d.K : 2 * d.I;
    return ((long long)d.M * d.top_k + 64) * wide < (1ll << 31);
}

// workspace of the 16-bit forward
struct HalfLayout {
    size_t err, bcnt, eri, sorted, counts, cumsum, y, g2, total;
};
HalfLayout half_layout(const megamoe_dims &d) {
    const size_t M = d.M, R = M * d.top_k;
    HalfLayout L;
    size_t o = 0;
    L.err = o;    o += align_up(kErrBytes);
    L.bcnt = o;   o += align_up(route_sort_workspace_bytes((int)R, d.E));
    L.eri = o;    o += align_up(R * 4);
    L.sorted = o; o += align_up(R * 4);
    L.counts = o; o += align_up((size_t)d.E * 4);
    L.cumsum = o; o += align_up((size_t)d.E * 4);
    L.y = o;      o += align_up(R * d.I * 2);
    L.g2 = o;     o += align_up(R * d.K * 2);
    L.total = o;
    return L;
}

bool gate_ok(const megamoe_dims &d, int64_t rows, int64_t cols) {
    return (rows == 1 || rows == d.M) && (cols == 1 || cols == d.K);
}
// a pointer that has to be there and aligned, or has to be missing
bool given(const void *p, bool wanted) { return wanted ? aligned16(p) : p == nullptr; }

}  // namespace

extern "C" {

const char *megamoe_strerror(int status) {
    switch (status) {
        case MEGAMOE_OK: return "ok";
        case MEGAMOE_EINVAL: return "invalid argument (null or misaligned pointer, bad dims)";
        case MEGAMOE_EUNSUPPORTED: return "dims outside the supported limits";
        case MEGAMOE_EWORKSPACE: return "workspace too small";
        case MEGAMOE_EHIP: return "HIP runtime or launch failure";
        case MEGAMOE_EDEVICE: return "routes with an expert id outside [0, E) were dropped";
        default: return "unknown status";
    }
}

int megamoe_check_dims(const megamoe_dims *d) {
    if (!d) return MEGAMOE_EINVAL;
    if (d->M < 1 || d->K < 1 || d->E < 1 || d->top_k < 1 || d->I < 1) return MEGAMOE_EINVAL;
    if (d->top_k > d->E || d->E > 256) return MEGAMOE_EUNSUPPORTED;
    if (d->K % 128 != 0 || d->K > 32768) return MEGAMOE_EUNSUPPORTED;
    if (d->I % 128 != 0 || d->I > 16384) return MEGAMOE_EUNSUPPORTED;
    const long long R = (long long)d->M * d->top_k;
    const long long wide = d->K > 2 * d->I ? d->K : 2 * d->I;
    if (R * wide >= (1ll << 31)) return MEGAMOE_EUNSUPPORTED;
    return MEGAMOE_OK;
}

int megamoe_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = forward_layout(*d).total;
    return MEGAMOE_OK;
}

int megamoe_permute_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = permute_ws_bytes(*d);
    return MEGAMOE_OK;
}

int megamoe_packed_weight_bytes(const megamoe_dims *d, size_t *w1p, size_t *w2p) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!w1p || !w2p) return MEGAMOE_EINVAL;
    *w1p = packed_weight_bytes(d->E, d->K, 2 * d->I);
    *w2p = packed_weight_bytes(d->E, d->I, d->K);
    return MEGAMOE_OK;
}

int megamoe_prepack_w1(const megamoe_dims *d, const int8_t *w1, int8_t *w1p, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!aligned16(w1) || !aligned16(w1p)) return MEGAMOE_EINVAL;
    return hip_status(launch_pack(w1, w1p, d->E, d->K, 2 * d->I, (hipStream_t)stream));
}

int megamoe_prepack_w2(const megamoe_dims *d, const int8_t *w2, int8_t *w2p, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!aligned16(w2) || !aligned16(w2p)) return MEGAMOE_EINVAL;
    return hip_status(launch_pack(w2, w2p, d->E, d->I, d->K, (hipStream_t)stream));
}

int megamoe_permute(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                    int8_t *gmA, float *pts1, int32_t *eri, int32_t *sorted_route,
                    int32_t *tokens_per_expert, int32_t *expert_cumsum, void *ws,
                    size_t ws_bytes, void *stream) {
    return permute_entry(d, x, expert_idx, gmA, pts1, eri, sorted_route, tokens_per_expert,
                         expert_cumsum, ws, ws_bytes, false, stream);
}

int megamoe_permute_noalloc(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                            int8_t *gmA, float *pts1, int32_t *eri, int32_t *sorted_route,
                            int32_t *tokens_per_expert, int32_t *expert_cumsum,
                            int32_t *dropped, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, expert_idx, gmA, pts1, eri, sorted_route, tokens_per_expert,
                          expert_cumsum, dropped};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (route_sort_workspace_bytes(d->M * d->top_k, d->E) > kNoAllocScratchBytes)
        return MEGAMOE_EUNSUPPORTED;
    int32_t *block_counts = scratch_device_ptr();
    if (block_counts == nullptr) return MEGAMOE_EHIP;
    // every count the sort reads is written by the same call first, so the
    // scratch needs no clearing between calls
    return run_permute(*d, x, expert_idx, gmA, pts1, eri, sorted_route, tokens_per_expert,
                       expert_cumsum, dropped, block_counts, false, (hipStream_t)stream);
}

int megamoe_permute_tokens(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                           int8_t *qx, float *pts1, int32_t *eri, int32_t *sorted_route,
                           int32_t *tokens_per_expert, int32_t *expert_cumsum, void *ws,
                           size_t ws_bytes, void *stream) {
    return permute_entry(d, x, expert_idx, qx, pts1, eri, sorted_route, tokens_per_expert,
                         expert_cumsum, ws, ws_bytes, true, stream);
}

int megamoe_gmm1(const megamoe_dims *d, const int8_t *gmA, const int32_t *expert_cumsum,
                 const int8_t *w1p, const float *scale1, uint16_t *gmC, int32_t *acc_dbg,
                 void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {gmA, expert_cumsum, w1p, scale1, gmC};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (acc_dbg && !aligned16(acc_dbg)) return MEGAMOE_EINVAL;
    return run_gmm(*d, gmA, expert_cumsum, w1p, scale1, gmC, acc_dbg, 2 * d->I, d->K,
                   (hipStream_t)stream);
}

int megamoe_gmm1_gather(const megamoe_dims *d, const int8_t *qx, const int32_t *sorted_route,
                        const int32_t *expert_cumsum, const int8_t *w1p, const float *scale1,
                        uint16_t *gmC, int32_t *acc_dbg, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {qx, sorted_route, expert_cumsum, w1p, scale1, gmC};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (acc_dbg && !aligned16(acc_dbg)) return MEGAMOE_EINVAL;
    return run_gmm(*d, qx, expert_cumsum, w1p, scale1, gmC, acc_dbg, 2 * d->I, d->K,
                   (hipStream_t)stream, sorted_route);
}

int megamoe_swiglu_quant(const megamoe_dims *d, const uint16_t *gmC, const float *pts1,
                         const int32_t *expert_cumsum, int8_t *q2, float *pts2, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {gmC, pts1, expert_cumsum, q2, pts2};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    return hip_status(launch_swiglu_quant(gmC, pts1, expert_cumsum, d->M * d->top_k, d->E, d->I,
                                          q2, pts2, (hipStream_t)stream));
}

int megamoe_gmm2(const megamoe_dims *d, const int8_t *q2, const int32_t *expert_cumsum,
                 const int8_t *w2p, const float *scale2, uint16_t *gmm2_out, int32_t *acc_dbg,
                 void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {q2, expert_cumsum, w2p, scale2, gmm2_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (acc_dbg && !aligned16(acc_dbg)) return MEGAMOE_EINVAL;
    return run_gmm(*d, q2, expert_cumsum, w2p, scale2, gmm2_out, acc_dbg, d->K, d->I,
                   (hipStream_t)stream);
}

int megamoe_gmm1_split_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = split_ws_bytes();
    return MEGAMOE_OK;
}

int megamoe_gmm1_gather_split(const megamoe_dims *d, const int8_t *qx,
                              const int32_t *sorted_route, const int32_t *expert_cumsum,
                              const int8_t *w1p, const float *scale1, uint16_t *gmC,
                              void *split_ws, size_t split_ws_bytes_, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {qx, sorted_route, expert_cumsum, w1p, scale1, gmC, split_ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (split_ws_bytes_ < split_ws_bytes()) return MEGAMOE_EWORKSPACE;
    GmmParams kp{};
    kp.ks_count = (uint32_t *)split_ws;
    kp.ks_part = (int32_t *)((char *)split_ws + kSplitCountBytes);
    return run_gmm(*d, qx, expert_cumsum, w1p, scale1, gmC, nullptr, 2 * d->I, d->K,
                   (hipStream_t)stream, sorted_route, &kp);
}

int megamoe_paired_q2_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = paired_q2_bytes(*d);
    return MEGAMOE_OK;
}

int megamoe_permute_tokens_paired(const megamoe_dims *d, const uint16_t *x,
                                  const int32_t *expert_idx, int8_t *qx, float *pts1,
                                  int32_t *eri, int32_t *sorted_route, int32_t *tokens_per_expert,
                                  int32_t *expert_cumsum, int32_t *prow, void *ws,
                                  size_t ws_bytes, void *stream) {
    if (!prow) return MEGAMOE_EINVAL;
    return permute_entry(d, x, expert_idx, qx, pts1, eri, sorted_route, tokens_per_expert,
                         expert_cumsum, ws, ws_bytes, true, stream, prow);
}

int megamoe_swiglu_quant_paired(const megamoe_dims *d, const uint16_t *gmC, const float *pts1,
                                const int32_t *expert_cumsum, const int32_t *prow, int8_t *q2p,
                                float *pts2, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {gmC, pts1, expert_cumsum, prow, q2p, pts2};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    return hip_status(launch_swiglu_quant(gmC, pts1, expert_cumsum, d->M * d->top_k, d->E, d->I,
                                          q2p, pts2, (hipStream_t)stream, nullptr, prow));
}

int megamoe_gmm2_paired(const megamoe_dims *d, const int8_t *q2p, const int32_t *expert_cumsum,
                        const int8_t *w2p, const float *scale2, uint16_t *gmm2_out,
                        int32_t *acc_dbg, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {q2p, expert_cumsum, w2p, scale2, gmm2_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (acc_dbg && !aligned16(acc_dbg)) return MEGAMOE_EINVAL;
    return run_gmm(*d, q2p, expert_cumsum, w2p, scale2, gmm2_out, acc_dbg, d->K, d->I,
                   (hipStream_t)stream, nullptr, nullptr, true);
}

int megamoe_unpermute(const megamoe_dims *d, const uint16_t *gmm2_out, const float *pts2,
                      const int32_t *eri, const float *probs, uint16_t *out, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {gmm2_out, pts2, eri, probs, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    return hip_status(launch_unpermute(gmm2_out, pts2, eri, probs, d->M, d->K, d->top_k, out,
                                       (hipStream_t)stream));
}

int megamoe_forward(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                    const float *probs, const int8_t *w1p, const float *scale1,
                    const int8_t *w2p, const float *scale2, uint16_t *out, void *ws,
                    size_t ws_bytes, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, expert_idx, probs, w1p, scale1, w2p, scale2, out, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    const Layout L = forward_layout(*d);
    if (ws_bytes < L.total) return MEGAMOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    char *base = (char *)ws;
    int32_t *err = (int32_t *)(base + L.err);
    int32_t *eri = (int32_t *)(base + L.eri);
    int32_t *sorted = (int32_t *)(base + L.sorted);
    int32_t *counts = (int32_t *)(base + L.counts);
    int32_t *cumsum = (int32_t *)(base + L.cumsum);
    float *pts1 = (float *)(base + L.pts1);
    float *pts2 = (float *)(base + L.pts2);
    int8_t *gmA = (int8_t *)(base + L.gmA);
    uint16_t *gmC = (uint16_t *)(base + L.gmC);
    int8_t *q2 = (int8_t *)(base + L.q2);
    uint16_t *g2 = (uint16_t *)(base + L.g2);

    int32_t *bcnt = (int32_t *)(base + L.bcnt);
    uint32_t *tsync = (uint32_t *)(base + L.tsync);
    uint8_t *tdone = (uint8_t *)(base + L.tdone);
    const int R = d->M * d->top_k;
    const int overlap = g_overlap.load(std::memory_order_relaxed);
    const bool tail = overlap != 0 && gmm_tail_ok(R, d->E, d->I);
    // GMM2 reads q2 in the row-paired layout: the 64-byte K slices of two
    // rows share each 128-byte line, so its A copies read whole lines (the
    // sort writes each row's paired place to prow)
    int32_t *prow = (int32_t *)(base + L.prow);
    // the quantised tokens are written once, token-major; GMM1 gathers its
    // expert-sorted rows from them through the route list, so the top_k
    // copies of each token are never written to or re-read from HBM
    MEGAMOE_TRY(run_permute(*d, x, expert_idx, gmA, pts1, eri, sorted, counts, cumsum, err, bcnt,
                            true, s, (float *)(base + L.tscale), tail ? tdone : nullptr, tsync,
                            prow));
    // SwiGLU: the rows whose GMM1 output is complete before GMM1's last round
    // are done by the workgroups left idle in that round; the SwiGLU kernel
    // does the rest (all rows without the overlap)
    GmmParams tp{};
    tp.tail_q2 = q2;
    tp.tail_pts2 = pts2;
    tp.tail_pts1 = pts1;
    tp.tail_sync = tsync;
    tp.tail_done = tdone;
    tp.tail_I = d->I;
    tp.tail_spin = overlap == 2 ? -1 : kTailSpin;
    tp.tail_prow = prow;
    // without the overlap, GMM1's sparse last round splits its tiles over K
    // (the permute zeroes the counters after the overlap's three words)
    GmmParams kp{};
    kp.ks_part = (int32_t *)(base + L.ks);
    kp.ks_count = tsync + 3;
    MEGAMOE_TRY(run_gmm(*d, gmA, cumsum, w1p, scale1, gmC, nullptr, 2 * d->I, d->K, s, sorted,
                        tail ? &tp : &kp));
    MEGAMOE_TRY(hip_status(launch_swiglu_quant(gmC, pts1, cumsum, R, d->E, d->I, q2, pts2, s,
                                               tail ? tdone : nullptr, prow)));
    MEGAMOE_TRY(run_gmm(*d, q2, cumsum, w2p, scale2, g2, nullptr, d->K, d->I, s, nullptr, nullptr,
                        true));
    return hip_status(launch_unpermute(g2, pts2, eri, probs, d->M, d->K, d->top_k, out, s));
}

int megamoe_route(const megamoe_dims *d, const void *logits, int logits_type, const float *bias,
                  int renormalize, int32_t *expert_idx, float *probs, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {logits, expert_idx, probs};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if ((bias && !aligned16(bias)) || !type_ok(logits_type)) return MEGAMOE_EINVAL;
    return hip_status(launch_route(logits, logits_type, bias, d->M, d->E, d->top_k,
                                   renormalize != 0, expert_idx, probs, (hipStream_t)stream));
}

int megamoe_few_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(check_few(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = few_layout(*d).total;
    return MEGAMOE_OK;
}

int megamoe_forward_few(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                        const float *probs, const int8_t *w1p, const float *scale1,
                        const int8_t *w2p, const float *scale2, uint16_t *out, void *ws,
                        size_t ws_bytes, void *stream) {
    MEGAMOE_TRY(check_few(d));
    const void *ptrs[] = {x, expert_idx, probs, w1p, scale1, w2p, scale2, out, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    const FewLayout L = few_layout(*d);
    if (ws_bytes < L.total) return MEGAMOE_EWORKSPACE;
    char *base = (char *)ws;
    const FewParams p{x, expert_idx, probs, w1p, w2p, scale1, scale2, out, (int32_t *)base,
                      (float *)(base + L.y), (float *)(base + L.ymax), d->M, d->K, d->E, d->top_k,
                      d->I};
    return hip_status(launch_few(p, (hipStream_t)stream));
}

int megamoe_mxfp4_quant(const void *x, int type, int64_t rows, int64_t cols,
                        const int32_t *valid_rows, uint8_t *q, uint8_t *scale, void *stream) {
    MEGAMOE_TRY(check_mxfp4_rows(rows, cols));
    const void *ptrs[] = {x, q, scale};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (((uintptr_t)valid_rows & 3u) != 0 || !type_ok(type)) return MEGAMOE_EINVAL;
    return hip_status(
        launch_mxfp4_quant(x, type, rows, cols, valid_rows, q, scale, (hipStream_t)stream));
}

int megamoe_mxfp4_dequant(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                          const int32_t *valid_rows, void *x, int type, void *stream) {
    MEGAMOE_TRY(check_mxfp4_rows(rows, cols));
    const void *ptrs[] = {q, scale, x};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (((uintptr_t)valid_rows & 3u) != 0 || !type_ok(type)) return MEGAMOE_EINVAL;
    return hip_status(
        launch_mxfp4_dequant(q, scale, rows, cols, valid_rows, x, type, (hipStream_t)stream));
}

int megamoe_mxfp4_gmm1(const megamoe_dims *d, const uint8_t *xq, const uint8_t *xs,
                       const int32_t *sorted_route, const int32_t *expert_cumsum,
                       const uint8_t *w1q, const uint8_t *w1s, uint16_t *y, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {xq, xs, sorted_route, expert_cumsum, w1q, w1s, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    return run_mxfp4_gmm(*d, xq, xs, sorted_route, expert_cumsum, w1q, w1s, y, nullptr, nullptr,
                         true, (hipStream_t)stream);
}

int megamoe_mxfp4_gmm2(const megamoe_dims *d, const uint8_t *yq, const uint8_t *ys,
                       const int32_t *expert_cumsum, const uint8_t *w2q, const uint8_t *w2s,
                       uint16_t *gmm2_out, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {yq, ys, expert_cumsum, w2q, w2s, gmm2_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    return run_mxfp4_gmm(*d, yq, ys, nullptr, expert_cumsum, w2q, w2s, gmm2_out, nullptr, nullptr,
                         false, (hipStream_t)stream);
}

int megamoe_mxfp4_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = mxfp4_layout(*d).total;
    return MEGAMOE_OK;
}

int megamoe_forward_mxfp4(const megamoe_dims *d, const uint16_t *x, const int32_t *expert_idx,
                          const float *probs, const uint8_t *w1q, const uint8_t *w1s,
                          const uint8_t *w2q, const uint8_t *w2s, uint16_t *out, void *ws,
                          size_t ws_bytes, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, expert_idx, probs, w1q, w1s, w2q, w2s, out, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    const Mxfp4Layout L = mxfp4_layout(*d);
    if (ws_bytes < L.total) return MEGAMOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    char *base = (char *)ws;
    int32_t *eri = (int32_t *)(base + L.eri);
    int32_t *sorted = (int32_t *)(base + L.sorted);
    int32_t *cumsum = (int32_t *)(base + L.cumsum);
    uint8_t *xq = (uint8_t *)(base + L.xq), *xs = (uint8_t *)(base + L.xs);
    uint16_t *g2 = (uint16_t *)(base + L.g2);
    uint8_t *yq = (uint8_t *)(base + L.yq), *ys = (uint8_t *)(base + L.ys);
    const int R = d->M * d->top_k;
    MEGAMOE_TRY(hip_status(launch_route_sort(expert_idx, R, d->E, sorted, eri,
                                             (int32_t *)(base + L.counts), cumsum,
                                             (int32_t *)(base + L.err),
                                             (int32_t *)(base + L.bcnt), s)));
    MEGAMOE_TRY(hip_status(launch_mxfp4_quant(x, kFp16, d->M, d->K, nullptr, xq, xs, s)));
    MEGAMOE_TRY(run_mxfp4_gmm(*d, xq, xs, sorted, cumsum, w1q, w1s, nullptr, yq, ys, true, s));
    MEGAMOE_TRY(run_mxfp4_gmm(*d, yq, ys, nullptr, cumsum, w2q, w2s, g2, nullptr, nullptr, false, s));
    return hip_status(launch_unpermute(g2, nullptr, eri, probs, d->M, d->K, d->top_k, out, s));
}

int megamoe_sort_routes(const megamoe_dims *d, const int32_t *expert_idx, int32_t *eri,
                        int32_t *sorted_route, int32_t *tokens_per_expert, int32_t *expert_cumsum,
                        void *ws, size_t ws_bytes, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {expert_idx, eri, sorted_route, tokens_per_expert, expert_cumsum, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (ws_bytes < permute_ws_bytes(*d)) return MEGAMOE_EWORKSPACE;
    char *w = (char *)ws;
    return hip_status(launch_route_sort(expert_idx, d->M * d->top_k, d->E, sorted_route, eri,
                                        tokens_per_expert, expert_cumsum, (int32_t *)w,
                                        (int32_t *)(w + align_up(kErrBytes)), (hipStream_t)stream));
}

int megamoe_half_gmm1(const megamoe_dims *d, const uint16_t *x, int type,
                      const int32_t *sorted_route, const int32_t *expert_cumsum,
                      const uint16_t *w1, uint16_t *c, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, sorted_route, expert_cumsum, w1, c};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type)) return MEGAMOE_EINVAL;
    return run_half_gmm(*d, kHalfProduct, true, x, w1, type, sorted_route, 1, expert_cumsum,
                        nullptr, false, c, type, false, (hipStream_t)stream);
}

int megamoe_half_gmm1_swiglu(const megamoe_dims *d, const uint16_t *x, int type,
                             const int32_t *sorted_route, const int32_t *expert_cumsum,
                             const float *probs, const uint16_t *w1, uint16_t *y, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, sorted_route, expert_cumsum, w1, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if ((probs && !aligned16(probs)) || !half_type(type)) return MEGAMOE_EINVAL;
    return run_half_gmm(*d, kHalfProduct, true, x, w1, type, sorted_route, 1, expert_cumsum, probs,
                        true, y, type, false, (hipStream_t)stream);
}

int megamoe_half_gmm2(const megamoe_dims *d, const uint16_t *y, int type,
                      const int32_t *expert_cumsum, const uint16_t *w2, uint16_t *gmm2_out,
                      void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {y, expert_cumsum, w2, gmm2_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type)) return MEGAMOE_EINVAL;
    return run_half_gmm(*d, kHalfProduct, false, y, w2, type, nullptr, 0, expert_cumsum, nullptr,
                        false, gmm2_out, type, false, (hipStream_t)stream);
}

int megamoe_half_gmm1_dgrad(const megamoe_dims *d, const uint16_t *dc, int type,
                            const int32_t *expert_cumsum, const uint16_t *w1, uint16_t *dx_rows,
                            void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {dc, expert_cumsum, w1, dx_rows};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type)) return MEGAMOE_EINVAL;
    return run_half_gmm(*d, kHalfRows, true, dc, w1, type, nullptr, 0, expert_cumsum, nullptr,
                        false, dx_rows, type, false, (hipStream_t)stream);
}

int megamoe_half_gmm2_dgrad(const megamoe_dims *d, const uint16_t *dout, int type,
                            const int32_t *sorted_route, const int32_t *expert_cumsum,
                            const uint16_t *w2, uint16_t *dy, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {dout, sorted_route, expert_cumsum, w2, dy};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type)) return MEGAMOE_EINVAL;
    return run_half_gmm(*d, kHalfRows, false, dout, w2, type, sorted_route, 1, expert_cumsum,
                        nullptr, false, dy, type, false, (hipStream_t)stream);
}

int megamoe_half_gmm1_wgrad(const megamoe_dims *d, const uint16_t *dc, const uint16_t *x, int type,
                            const int32_t *sorted_route, const int32_t *expert_cumsum, void *dw1,
                            int dw_type, int accumulate, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {dc, x, sorted_route, expert_cumsum, dw1};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type) || (dw_type != type && dw_type != MEGAMOE_FP32)) return MEGAMOE_EINVAL;
    if (!half_wgrad_ok(*d)) return MEGAMOE_EUNSUPPORTED;
    return run_half_gmm(*d, kHalfWeights, true, dc, x, type, sorted_route, 2, expert_cumsum,
                        nullptr, false, dw1, dw_type, accumulate != 0, (hipStream_t)stream);
}

int megamoe_half_gmm2_wgrad(const megamoe_dims *d, const uint16_t *dout, const uint16_t *y,
                            int type, const int32_t *sorted_route, const int32_t *expert_cumsum,
                            void *dw2, int dw_type, int accumulate, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {dout, y, sorted_route, expert_cumsum, dw2};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type) || (dw_type != type && dw_type != MEGAMOE_FP32)) return MEGAMOE_EINVAL;
    if (!half_wgrad_ok(*d)) return MEGAMOE_EUNSUPPORTED;
    return run_half_gmm(*d, kHalfWeights, false, dout, y, type, sorted_route, 1, expert_cumsum,
                        nullptr, false, dw2, dw_type, accumulate != 0, (hipStream_t)stream);
}

int megamoe_half_swiglu(const megamoe_dims *d, const uint16_t *c, int type,
                        const int32_t *sorted_route, const int32_t *expert_cumsum,
                        const float *probs, uint16_t *y, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {c, sorted_route, expert_cumsum, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if ((probs && !aligned16(probs)) || !half_type(type)) return MEGAMOE_EINVAL;
    HalfSwigluParams p{};
    p.c = c;
    p.route = sorted_route;
    p.cumsum = expert_cumsum;
    p.probs = probs;
    p.y = y;
    p.R = d->M * d->top_k;
    p.E = d->E;
    p.I = d->I;
    return hip_status(launch_half_swiglu(p, type, false, (hipStream_t)stream));
}

int megamoe_half_swiglu_grad(const megamoe_dims *d, const uint16_t *c, const uint16_t *dy,
                             int type, const int32_t *sorted_route,
                             const int32_t *expanded_row_idx, const int32_t *expert_cumsum,
                             const float *probs, uint16_t *dc, float *dprobs, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {c, dy, sorted_route, expanded_row_idx, expert_cumsum, dc};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if ((probs && !aligned16(probs)) || (dprobs && !aligned16(dprobs)) || !half_type(type))
        return MEGAMOE_EINVAL;
    HalfSwigluParams p{};
    p.c = c;
    p.dy = dy;
    p.route = sorted_route;
    p.row_of = expanded_row_idx;
    p.cumsum = expert_cumsum;
    p.probs = probs;
    p.dc = dc;
    p.dprobs = dprobs;
    p.R = d->M * d->top_k;
    p.E = d->E;
    p.I = d->I;
    return hip_status(launch_half_swiglu(p, type, true, (hipStream_t)stream));
}

int megamoe_norm(const megamoe_dims *d, const void *x, int x_type, const void *rows, int rows_type,
                 const int32_t *expanded_row_idx, const float *w_after, const void *gate,
                 int gate_type, int64_t gate_rows, int64_t gate_cols, float alpha,
                 const float *w_before, float eps, void *s, void *r, void *h, int h_type,
                 void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *nullable[] = {x, rows, expanded_row_idx, w_after, gate, w_before, s, r, h};
    for (const void *p : nullable)
        if (p && !aligned16(p)) return MEGAMOE_EINVAL;
    if ((!x && !rows) || (!s && !r && !h)) return MEGAMOE_EINVAL;
    if (!rows && (expanded_row_idx || w_after || gate || s)) return MEGAMOE_EINVAL;
    if ((h == nullptr) != (w_before == nullptr)) return MEGAMOE_EINVAL;
    if (!type_ok(x_type) || !type_ok(rows_type) || !type_ok(h_type)) return MEGAMOE_EINVAL;
    if (gate && (!type_ok(gate_type) || !gate_ok(*d, gate_rows, gate_cols))) return MEGAMOE_EINVAL;
    if (!(eps > 0.0f) || !std::isfinite(eps) || !std::isfinite(alpha)) return MEGAMOE_EINVAL;
    NormParams p{};
    p.x = x;
    p.rows = rows;
    p.row_of = expanded_row_idx;
    p.w_after = w_after;
    p.w_before = w_before;
    p.gate = gate;
    p.s = s;
    p.r = r;
    p.h = h;
    p.M = d->M;
    p.K = d->K;
    p.top_k = d->top_k;
    p.R = d->M * d->top_k;
    p.gate_type = gate_type;
    p.gate_rows = (int)gate_rows;
    p.gate_cols = (int)gate_cols;
    p.h_type = h_type;
    p.alpha = alpha;
    p.eps = eps;
    return hip_status(launch_norm(p, x_type, rows_type, false, (hipStream_t)stream));
}

int megamoe_norm_grad_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = (size_t)3 * norm_grad_groups(d->M, d->K) * d->K * sizeof(float);
    return MEGAMOE_OK;
}

int megamoe_norm_grad(const megamoe_dims *d, const void *dr, const void *r, int x_type,
                      const void *dh, int h_type, const int32_t *expanded_row_idx, const void *s,
                      int rows_type, const float *w_after, const void *gate, int gate_type,
                      int64_t gate_rows, int64_t gate_cols, float alpha, const float *w_before,
                      float eps, void *dx, void *ds, float *dw_after, float *dw_before,
                      void *dgate, void *ws, size_t ws_bytes, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!aligned16(dx) || !aligned16(ws) || (dr && !aligned16(dr)) || (!dr && !dh))
        return MEGAMOE_EINVAL;
    if (expanded_row_idx && (!aligned16(expanded_row_idx) || !dh)) return MEGAMOE_EINVAL;
    const bool before = w_before != nullptr, block = s != nullptr;
    if (!given(w_before, before) || !given(r, before) || !given(dh, before) ||
        !given(dw_before, before))
        return MEGAMOE_EINVAL;
    if (!given(s, block) || !given(ds, block)) return MEGAMOE_EINVAL;
    const bool after = w_after != nullptr, gated = gate != nullptr;
    if ((after || gated) && !block) return MEGAMOE_EINVAL;
    if (!given(w_after, after) || !given(dw_after, after) || !given(gate, gated) ||
        !given(dgate, gated))
        return MEGAMOE_EINVAL;
    if (!type_ok(x_type) || !type_ok(rows_type) || !type_ok(h_type)) return MEGAMOE_EINVAL;
    if (gated && (!type_ok(gate_type) || !gate_ok(*d, gate_rows, gate_cols))) return MEGAMOE_EINVAL;
    if (!(eps > 0.0f) || !std::isfinite(eps) || !std::isfinite(alpha)) return MEGAMOE_EINVAL;
    size_t need = 0;
    MEGAMOE_TRY(megamoe_norm_grad_workspace_bytes(d, &need));
    if (ws_bytes < need) return MEGAMOE_EWORKSPACE;
    NormParams p{};
    p.row_of = expanded_row_idx;
    p.w_after = w_after;
    p.w_before = w_before;
    p.gate = gate;
    p.s = const_cast<void *>(s);
    p.r = const_cast<void *>(r);
    p.h = const_cast<void *>(dh);
    p.dr = dr;
    p.dx = dx;
    p.ds = ds;
    p.dgate = dgate;
    p.dw_after = dw_after;
    p.dw_before = dw_before;
    p.part = (float *)ws;
    p.M = d->M;
    p.K = d->K;
    p.top_k = d->top_k;
    p.R = d->M * d->top_k;
    p.gate_type = gate_type;
    p.gate_rows = (int)gate_rows;
    p.gate_cols = (int)gate_cols;
    p.h_type = h_type;
    p.alpha = alpha;
    p.eps = eps;
    return hip_status(launch_norm(p, x_type, rows_type, true, (hipStream_t)stream));
}

int megamoe_route_grad(const megamoe_dims *d, const void *logits, int logits_type,
                       const float *bias, int renormalize, const int32_t *expert_idx,
                       const float *probs, const float *dprobs, void *dlogits, void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {logits, expert_idx, probs, dprobs, dlogits};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if ((bias && !aligned16(bias)) || !type_ok(logits_type)) return MEGAMOE_EINVAL;
    const RouteGradParams p{logits, bias, expert_idx, probs, dprobs, dlogits,
                            d->M, d->E, d->top_k, renormalize != 0};
    return hip_status(launch_route_grad(p, logits_type, (hipStream_t)stream));
}

int megamoe_half_workspace_bytes(const megamoe_dims *d, size_t *bytes) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    if (!bytes) return MEGAMOE_EINVAL;
    *bytes = half_layout(*d).total;
    return MEGAMOE_OK;
}

int megamoe_forward_half(const megamoe_dims *d, const uint16_t *x, int type,
                         const int32_t *expert_idx, const float *probs, const uint16_t *w1,
                         const uint16_t *w2, uint16_t *out, void *ws, size_t ws_bytes,
                         void *stream) {
    MEGAMOE_TRY(megamoe_check_dims(d));
    const void *ptrs[] = {x, expert_idx, probs, w1, w2, out, ws};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MEGAMOE_EINVAL;
    if (!half_type(type)) return MEGAMOE_EINVAL;
    const HalfLayout L = half_layout(*d);
    if (ws_bytes < L.total) return MEGAMOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    char *base = (char *)ws;
    int32_t *eri = (int32_t *)(base + L.eri);
    int32_t *sorted = (int32_t *)(base + L.sorted);
    int32_t *cumsum = (int32_t *)(base + L.cumsum);
    uint16_t *y = (uint16_t *)(base + L.y), *g2 = (uint16_t *)(base + L.g2);
    MEGAMOE_TRY(hip_status(launch_route_sort(expert_idx, d->M * d->top_k, d->E, sorted, eri,
                                             (int32_t *)(base + L.counts), cumsum,
                                             (int32_t *)(base + L.err),
                                             (int32_t *)(base + L.bcnt), s)));
    MEGAMOE_TRY(run_half_gmm(*d, kHalfProduct, true, x, w1, type, sorted, 1, cumsum, probs, true, y,
                             type, false, s));
    MEGAMOE_TRY(run_half_gmm(*d, kHalfProduct, false, y, w2, type, nullptr, 0, cumsum, nullptr,
                             false, g2, type, false, s));
    NormParams p{};  // no norm: the rows' sum alone
    p.rows = g2;
    p.row_of = eri;
    p.r = out;
    p.M = d->M;
    p.K = d->K;
    p.top_k = d->top_k;
    p.R = d->M * d->top_k;
    p.alpha = p.eps = 1.0f;
    return hip_status(launch_norm(p, type, type, false, s));
}

int megamoe_set_overlap(int mode) {
    if (mode < 0 || mode > 2) return MEGAMOE_EINVAL;
    g_overlap.store(mode, std::memory_order_relaxed);
    return MEGAMOE_OK;
}

int megamoe_last_error(const void *ws, void *stream, int32_t *bad_route_count) {
    if (!aligned16(ws) || !bad_route_count) return MEGAMOE_EINVAL;
    hipStream_t s = (hipStream_t)stream;
    int32_t v = 0;
    if (hipMemcpyAsync(&v, ws, sizeof(v), hipMemcpyDeviceToHost, s) != hipSuccess)
        return MEGAMOE_EHIP;
    if (hipStreamSynchronize(s) != hipSuccess) return MEGAMOE_EHIP;
    *bad_route_count = v;
    return v ? MEGAMOE_EDEVICE : MEGAMOE_OK;
}

}  // extern "C"
