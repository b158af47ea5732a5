// C ABI of libmgscan (declared in include/mgscan.h): argument validation,
// the per-device error word, and dispatch to the kernel launchers.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <memory>
#include <mutex>
#include <map>
#include <new>
#include <set>
#include <utility>

#include <cudaTypedefs.h>

#include "../../include/mgscan.h"
#include "mgs_launch.h"
#include "mgs_lm.h"

#define MGS_VERSION_INT 100  // 0.1.0

namespace {

// Error word written by kernels whose bounded waits give up (one per device:
// a __device__ variable exists once in every device context that loads the
// library).  Host code never dereferences its name; it asks the runtime for
// the device address, once per device.
__device__ unsigned g_mgs_error_word = 0;

mgs::SymbolAddressCache g_err_cache;
std::atomic<uint64_t> g_timeout_ns{1000000000ull};

mgs_status current_ctl(mgs::DevCtl *ctl) {
    void *p = nullptr;
    if (mgs::cached_symbol_address(g_err_cache, (const void *)&g_mgs_error_word, &p) != cudaSuccess)
        return MGS_ERR_CUDA;
    ctl->err = static_cast<unsigned *>(p);
    ctl->timeout_ns = g_timeout_ns.load();
    return MGS_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// n = a*b*c*... with overflow detection (all factors >= 0).
bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a == 0 || b == 0) { *out = 0; return true; }
    if (a > INT64_MAX / b) return false;
    *out = a * b;
    return true;
}

struct Range {
    uintptr_t lo, hi;
};
Range rng(const void *p, int64_t count) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + uintptr_t(count) * sizeof(float)};
}
bool overlap(Range x, Range y) { return x.lo < y.hi && y.lo < x.hi; }

// Every output must be disjoint from every input and from the other outputs.
bool disjoint(std::initializer_list<std::pair<const void *, int64_t>> outs,
              std::initializer_list<std::pair<const void *, int64_t>> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (o->first == nullptr || o->second == 0) continue;
        Range ro = rng(o->first, o->second);
        for (auto &i : ins)
            if (i.first != nullptr && i.second != 0 && overlap(ro, rng(i.first, i.second))) return false;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (o2->first != nullptr && o2->second != 0 && overlap(ro, rng(o2->first, o2->second)))
                return false;
    }
    return true;
}

bool k_supported(int k, int64_t H) {
    if (k == 4 || k == 8 || k == 16) return true;
    if (k == 1 || k == 2) return (H * k) % 4 == 0;
    return false;
}

struct BlockSizes {
    int64_t mat, vec, init;  // element counts: [B,T,H,k,k], [B,T,H,k], [B,H,k]
};

// Validates (B, T, H, k) for the matrix ops and computes element counts.
mgs_status block_sizes(int64_t B, int64_t T, int64_t H, int k, BlockSizes *s) {
    if (B < 0 || T < 0 || H < 0 || k <= 0) return MGS_ERR_INVALID_ARG;
    if (!k_supported(k, H)) return MGS_ERR_UNSUPPORTED;
    int64_t bth, bh;
    if (!mul_ok(B, T, &bth) || !mul_ok(bth, H, &bth) || !mul_ok(B, H, &bh)) return MGS_ERR_INVALID_ARG;
    if (!mul_ok(bth, int64_t(k) * k, &s->mat) || !mul_ok(bth, k, &s->vec) || !mul_ok(bh, k, &s->init))
        return MGS_ERR_INVALID_ARG;
    if (s->mat > (INT64_MAX / 8)) return MGS_ERR_INVALID_ARG;
    // tensor-map row coordinates are 32-bit
    if (B * T > INT32_MAX || H > INT32_MAX / 256) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

struct GivensSizes {
    int64_t ang, vec, mat, init;  // element counts: [B,T,H,N], [B,T,H,k], [B,T,H,k,k], [B,H,k]
};

// Validates (B, T, H, k) for the Givens-mesh ops (k = 8 only).
mgs_status givens_sizes(int64_t B, int64_t T, int64_t H, int k, GivensSizes *s) {
    if (B < 0 || T < 0 || H < 0 || k <= 0) return MGS_ERR_INVALID_ARG;
    if (k != 8) return MGS_ERR_UNSUPPORTED;
    int64_t bth, bh;
    if (!mul_ok(B, T, &bth) || !mul_ok(bth, H, &bth) || !mul_ok(B, H, &bh)) return MGS_ERR_INVALID_ARG;
    if (!mul_ok(bth, 64, &s->mat) || !mul_ok(bth, 28, &s->ang) || !mul_ok(bth, 8, &s->vec) ||
        !mul_ok(bh, 8, &s->init))
        return MGS_ERR_INVALID_ARG;
    if (s->mat > (INT64_MAX / 8)) return MGS_ERR_INVALID_ARG;
    if (B * T > INT32_MAX || H > INT32_MAX / 256) return MGS_ERR_UNSUPPORTED;  // 32-bit map coordinates
    return MGS_OK;
}

mgs_status check_ptrs(std::initializer_list<const void *> required,
                      std::initializer_list<const void *> optional) {
    for (const void *p : required)
        if (p == nullptr) return MGS_ERR_INVALID_ARG;
    for (const void *p : required)
        if (!aligned16(p)) return MGS_ERR_UNSUPPORTED;
    for (const void *p : optional)
        if (p != nullptr && !aligned16(p)) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

mgs_status check_ws(size_t need, const void *ws, size_t ws_bytes) {
    if (need == 0) return MGS_OK;
    if (ws == nullptr || ws_bytes < need) return MGS_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MGS_ERR_WORKSPACE;
    return MGS_OK;
}

mgs_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MGS_OK : MGS_ERR_CUDA; }

}  // namespace

namespace mgs {

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    std::call_once(once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return encode;
}

cudaError_t make_tmap(CUtensorMap *map, const float *base, int rank, const uint64_t *dims,
                      const uint64_t *byte_strides, const uint32_t *box, bool swizzle128) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    cuuint64_t gdim[3], gstr[2];
    cuuint32_t bdim[3], estr[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        gdim[i] = dims[i];
        bdim[i] = box[i];
    }
    for (int i = 0; i + 1 < rank; ++i) gstr[i] = byte_strides[i];
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, cuuint32_t(rank), const_cast<float *>(base), gdim,
                        gstr, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_tmap_4d(CUtensorMap *map, const void *base, const uint64_t *dims, const uint64_t *byte_strides,
                         const uint32_t *box, bool f32) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    cuuint64_t gdim[4], gstr[3];
    cuuint32_t bdim[4], estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) gdim[i] = dims[i], bdim[i] = box[i];
    for (int i = 0; i < 3; ++i) gstr[i] = byte_strides[i];
    const CUresult r = encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                              const_cast<void *>(base), gdim, gstr, bdim, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

uint64_t current_context_id() {
    static std::once_flag once;
    static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
    static PFN_cuCtxGetId_v12000 get_id = nullptr;
    std::call_once(once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &fn, 4000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(fn);
        fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(fn);
    });
    if (get_current == nullptr || get_id == nullptr) return 0;
    CUcontext c = nullptr;
    if (get_current(&c) != CUDA_SUCCESS || c == nullptr) return 0;
    unsigned long long id = 0;
    return get_id(c, &id) == CUDA_SUCCESS ? uint64_t(id) : 0;
}

cudaError_t cached_symbol_address(SymbolAddressCache &cache, const void *symbol, void **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= SymbolAddressCache::kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(cache.mu);
    const uint64_t ctx = current_context_id();
    if (ctx != 0 && cache.ctx[dev] == ctx && cache.addr[dev] != nullptr) {
        *out = cache.addr[dev];
        return cudaSuccess;
    }
    // the lookup also creates and binds the device's primary context when no
    // context is current yet, so the id is read again after it
    void *p = nullptr;
    if ((e = cudaGetSymbolAddress(&p, symbol)) != cudaSuccess) return e;
    cache.ctx[dev] = current_context_id();
    cache.addr[dev] = p;
    *out = p;
    return cudaSuccess;
}

cudaError_t ensure_smem_attr(const void *fn, int bytes) {
    // the limit set for each kernel in each device context; raised (to the
    // opt-in maximum) when a launch needs more than the 48 KB default
    static std::mutex mu;
    static std::map<std::pair<const void *, uint64_t>, int> limit;
    const uint64_t ctx = current_context_id();
    const int want = bytes > 48 * 1024 ? 227 * 1024 : 48 * 1024;
    std::lock_guard<std::mutex> lk(mu);
    auto key = std::make_pair(fn, ctx);
    auto itr = limit.find(key);
    if (ctx != 0 && itr != limit.end() && itr->second >= want) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, want);
    if (e == cudaSuccess && ctx != 0) limit[key] = want;
    return e;
}

}  // namespace mgs

extern "C" {

static mgs_status psl_sizes(int64_t B, int64_t T, int64_t D, int64_t *n, int64_t *n0);

size_t mgs_workspace_size(int op, int64_t B, int64_t T, int64_t H_or_D, int k) {
    BlockSizes s;
    switch (op) {
        case MGS_OP_MATRIX_AFFINE_SCAN_FWD:
        case MGS_OP_MATRIX_AFFINE_SCAN_BWD:
            if (block_sizes(B, T, H_or_D, k, &s) != MGS_OK) return 0;
            return mgs::mas_workspace_bytes(B, T, H_or_D, k);
        case MGS_OP_LINEAR_SCAN_FWD:
        case MGS_OP_LINEAR_SCAN_BWD:
            if (block_sizes(B, T, H_or_D, 1, &s) != MGS_OK) return 0;
            return mgs::mas_workspace_bytes(B, T, H_or_D, 1);
        case MGS_OP_MATRIX_AFFINE_SCAN_BWD_RECOMPUTE:
            if (block_sizes(B, T, H_or_D, k, &s) != MGS_OK || s.vec == 0) return 0;
            return mgs::mas_rc_workspace_bytes(B, T, H_or_D, k);
        case MGS_OP_MATRIX_SCAN_FWD:
        case MGS_OP_MATRIX_SCAN_BWD:
            if (block_sizes(B, T, H_or_D, k, &s) != MGS_OK) return 0;
            return mgs::ms_workspace_bytes(B, T, H_or_D, k, op == MGS_OP_MATRIX_SCAN_BWD);
        case MGS_OP_GIVENS_AFFINE_SCAN_FWD:
        case MGS_OP_GIVENS_AFFINE_SCAN_BWD:
        case MGS_OP_GIVENS_MATRIX_SCAN_FWD:
        case MGS_OP_GIVENS_MATRIX_SCAN_BWD: {
            GivensSizes gs;
            if (givens_sizes(B, T, H_or_D, k, &gs) != MGS_OK || gs.vec == 0) return 0;
            return mgs::givens_workspace_bytes(op - MGS_OP_GIVENS_AFFINE_SCAN_FWD, B, T, H_or_D);
        }
        case MGS_OP_DELTA_SCAN_FWD: {
            int64_t ns;
            if (B < 0 || T < 0 || H_or_D < 0 || k != 64 || !mul_ok(B, T, &ns) || !mul_ok(ns, H_or_D, &ns) ||
                !mul_ok(B, H_or_D, &ns) || !mul_ok(ns, (T + 63) / 64, &ns) || ns > INT64_MAX / (3 * 64 * 64 * 4))
                return 0;
            return mgs::delta_workspace_bytes(B, T, H_or_D);
        }
        case MGS_OP_PARALLEL_SCAN_LOG_BWD: {
            int64_t n, n0;
            if (psl_sizes(B, T, H_or_D, &n, &n0) != MGS_OK || n == 0) return 0;
            return mgs::psl_recompute_workspace_bytes(B, T, H_or_D);
        }
        default:
            return 0;
    }
}

mgs_status mgs_matrix_affine_scan_fwd(const float *A, const float *b, const float *h0, float *h,
                                      int64_t B, int64_t T, int64_t H, int k, void *workspace,
                                      size_t workspace_bytes, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.vec == 0) return MGS_OK;
    if ((st = check_ptrs({A, b, h}, {h0})) != MGS_OK) return st;
    if (!disjoint({{h, s.vec}}, {{A, s.mat}, {b, s.vec}, {h0, h0 ? s.init : 0}})) return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::mas_workspace_bytes(B, T, H, k), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    if (k == 1 && mgs::lin_supported(B, T, H))
        return from_cuda(mgs::launch_lin_fwd(A, b, h0, h, B, T, H, reinterpret_cast<cudaStream_t>(stream)));
    return from_cuda(mgs::launch_mas_fwd(k, A, b, h0, h, B, T, H, workspace, workspace_bytes, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_matrix_affine_scan_bwd(const float *A, const float *h0, const float *h,
                                      const float *grad_h, float *dA, float *db, float *dh0,
                                      int64_t B, int64_t T, int64_t H, int k, void *workspace,
                                      size_t workspace_bytes, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.init == 0) return MGS_OK;
    if (s.vec == 0) {
        // T == 0: lambda is empty, the initial-state gradient is zero
        if (dh0 == nullptr) return MGS_OK;
        if ((st = check_ptrs({dh0}, {})) != MGS_OK) return st;
        return from_cuda(cudaMemsetAsync(dh0, 0, size_t(s.init) * sizeof(float),
                                         reinterpret_cast<cudaStream_t>(stream)));
    }
    if ((st = check_ptrs({A, h, grad_h, dA, db}, {h0, dh0})) != MGS_OK) return st;
    if (!disjoint({{dA, s.mat}, {db, s.vec}, {dh0, dh0 ? s.init : 0}},
                  {{A, s.mat}, {h0, h0 ? s.init : 0}, {h, s.vec}, {grad_h, s.vec}}))
        return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::mas_workspace_bytes(B, T, H, k), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    if (k == 1 && mgs::lin_supported(B, T, H))
        return from_cuda(mgs::launch_lin_bwd(A, h0, h, grad_h, dA, db, dh0, B, T, H,
                                             reinterpret_cast<cudaStream_t>(stream)));
    return from_cuda(mgs::launch_mas_bwd(k, A, h0, h, grad_h, dA, db, dh0, B, T, H, workspace, workspace_bytes,
                                         ctl, reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_matrix_affine_scan_bwd_recompute(const float *A, const float *b, const float *h0,
                                                const float *grad_h, float *dA, float *db, float *dh0,
                                                int64_t B, int64_t T, int64_t H, int k, void *workspace,
                                                size_t workspace_bytes, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.init == 0) return MGS_OK;
    if (s.vec == 0) {
        // T == 0: lambda is empty, the initial-state gradient is zero
        if (dh0 == nullptr) return MGS_OK;
        if ((st = check_ptrs({dh0}, {})) != MGS_OK) return st;
        return from_cuda(cudaMemsetAsync(dh0, 0, size_t(s.init) * sizeof(float),
                                         reinterpret_cast<cudaStream_t>(stream)));
    }
    if ((st = check_ptrs({A, b, grad_h, dA, db}, {h0, dh0})) != MGS_OK) return st;
    if (!disjoint({{dA, s.mat}, {db, s.vec}, {dh0, dh0 ? s.init : 0}},
                  {{A, s.mat}, {b, s.vec}, {h0, h0 ? s.init : 0}, {grad_h, s.vec}}))
        return MGS_ERR_INVALID_ARG;
    const size_t need = mgs::mas_rc_workspace_bytes(B, T, H, k);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!disjoint({{static_cast<float *>(workspace), int64_t(need / sizeof(float))}},
                  {{A, s.mat}, {b, s.vec}, {h0, h0 ? s.init : 0}, {grad_h, s.vec}, {dA, s.mat}, {db, s.vec},
                   {dh0, dh0 ? s.init : 0}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_mas_bwd_recompute(k, A, b, h0, grad_h, dA, db, dh0, B, T, H, workspace, ctl,
                                                   reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_matrix_scan_fwd(const float *A, float *P, int64_t B, int64_t T, int64_t H, int k,
                               void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.mat == 0) return MGS_OK;
    if ((st = check_ptrs({A, P}, {})) != MGS_OK) return st;
    if (!disjoint({{P, s.mat}}, {{A, s.mat}})) return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::ms_workspace_bytes(B, T, H, k, false), workspace, workspace_bytes)) != MGS_OK)
        return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_ms_fwd(k, A, P, B, T, H, workspace, workspace_bytes, ctl,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_matrix_scan_fwd_noalloc(const float *A, float *P, int64_t B, int64_t T, int64_t H,
                                       int k, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.mat == 0) return MGS_OK;
    if ((st = check_ptrs({A, P}, {})) != MGS_OK) return st;
    if (!disjoint({{P, s.mat}}, {{A, s.mat}})) return MGS_ERR_INVALID_ARG;
    if (mgs::ms_workspace_bytes(B, T, H, k, false) > mgs::ms_static_scratch_bytes()) return MGS_ERR_WORKSPACE;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_ms_fwd_static_scratch(k, A, P, B, T, H, ctl,
                                                       reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_matrix_scan_bwd(const float *A, const float *P, const float *grad_P, float *dA,
                               int64_t B, int64_t T, int64_t H, int k, void *workspace,
                               size_t workspace_bytes, mgs_stream_t stream) {
    BlockSizes s;
    mgs_status st = block_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.mat == 0) return MGS_OK;
    if ((st = check_ptrs({A, P, grad_P, dA}, {})) != MGS_OK) return st;
    if (!disjoint({{dA, s.mat}}, {{A, s.mat}, {P, s.mat}, {grad_P, s.mat}})) return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::ms_workspace_bytes(B, T, H, k, true), workspace, workspace_bytes)) != MGS_OK)
        return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_ms_bwd(k, A, P, grad_P, dA, B, T, H, workspace, workspace_bytes, ctl,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

static mgs_status psl_sizes(int64_t B, int64_t T, int64_t D, int64_t *n, int64_t *n0) {
    if (B < 0 || T < 0 || D < 0) return MGS_ERR_INVALID_ARG;
    if (D % 4 != 0) return MGS_ERR_UNSUPPORTED;
    int64_t bt;
    if (!mul_ok(B, T, &bt) || !mul_ok(bt, D, n) || !mul_ok(B, D, n0)) return MGS_ERR_INVALID_ARG;
    if (*n > INT64_MAX / 8) return MGS_ERR_INVALID_ARG;
    if (B * T > INT32_MAX || D > INT32_MAX) return MGS_ERR_UNSUPPORTED;  // 32-bit map coordinates
    return MGS_OK;
}

mgs_status mgs_parallel_scan_log_fwd(const float *log_coeffs, const float *log_values,
                                     const float *log_h0, float *h, float *log_h, int64_t B,
                                     int64_t T, int64_t D, void *workspace, size_t workspace_bytes,
                                     mgs_stream_t stream) {
    int64_t n, n0;
    mgs_status st = psl_sizes(B, T, D, &n, &n0);
    if (st != MGS_OK) return st;
    if (n == 0) return MGS_OK;
    if ((st = check_ptrs({log_coeffs, log_values, h}, {log_h0, log_h})) != MGS_OK) return st;
    if (!disjoint({{h, n}, {log_h, log_h ? n : 0}},
                  {{log_coeffs, n}, {log_values, n}, {log_h0, log_h0 ? n0 : 0}}))
        return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(0, workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    if (mgs::psl_cl_supported(B, T, D))
        return from_cuda(mgs::launch_psl_fwd_cl(log_coeffs, log_values, log_h0, h, log_h, B, T, D,
                                                reinterpret_cast<cudaStream_t>(stream)));
    return from_cuda(mgs::launch_psl_fwd(log_coeffs, log_values, log_h0, h, log_h, B, T, D, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_parallel_scan_log_bwd(const float *log_coeffs, const float *log_values,
                                     const float *log_h0, const float *h, const float *grad_h,
                                     float *d_log_coeffs, float *d_log_values, float *d_log_h0,
                                     int64_t B, int64_t T, int64_t D, void *workspace,
                                     size_t workspace_bytes, mgs_stream_t stream) {
    int64_t n, n0;
    mgs_status st = psl_sizes(B, T, D, &n, &n0);
    if (st != MGS_OK) return st;
    if (d_log_h0 != nullptr && log_h0 == nullptr) return MGS_ERR_INVALID_ARG;
    if (n0 == 0) return MGS_OK;
    if (n == 0) {
        if (d_log_h0 == nullptr) return MGS_OK;
        if ((st = check_ptrs({d_log_h0}, {})) != MGS_OK) return st;
        return from_cuda(cudaMemsetAsync(d_log_h0, 0, size_t(n0) * sizeof(float),
                                         reinterpret_cast<cudaStream_t>(stream)));
    }
    if ((st = check_ptrs({log_coeffs, log_values, grad_h, d_log_coeffs, d_log_values},
                         {log_h0, h, d_log_h0})) != MGS_OK)
        return st;
    if (!disjoint({{d_log_coeffs, n}, {d_log_values, n}, {d_log_h0, d_log_h0 ? n0 : 0}},
                  {{log_coeffs, n}, {log_values, n}, {log_h0, log_h0 ? n0 : 0}, {h, h ? n : 0},
                   {grad_h, n}}))
        return MGS_ERR_INVALID_ARG;
    const size_t need = (h == nullptr) ? mgs::psl_recompute_workspace_bytes(B, T, D) : 0;
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    if (h == nullptr && mgs::psl_cl_supported(B, T, D))
        return from_cuda(mgs::launch_psl_bwd_rc_cl(log_coeffs, log_values, log_h0, grad_h, d_log_coeffs,
                                                   d_log_values, d_log_h0, B, T, D,
                                                   reinterpret_cast<cudaStream_t>(stream)));
    if (h == nullptr)
        return from_cuda(mgs::launch_psl_bwd_recompute(log_coeffs, log_values, log_h0, grad_h, d_log_coeffs,
                                                       d_log_values, d_log_h0, workspace, B, T, D, ctl,
                                                       reinterpret_cast<cudaStream_t>(stream)));
    if (mgs::psl_cl_supported(B, T, D))
        return from_cuda(mgs::launch_psl_bwd_cl(log_coeffs, log_values, log_h0, h, grad_h, d_log_coeffs,
                                                d_log_values, d_log_h0, B, T, D,
                                                reinterpret_cast<cudaStream_t>(stream)));
    return from_cuda(mgs::launch_psl_bwd(log_coeffs, log_values, log_h0, h, grad_h, d_log_coeffs,
                                         d_log_values, d_log_h0, B, T, D, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

// linear_scan is matrix_affine_scan with 1 x 1 blocks: [B][T][D] is
// [B][T][H=D][1][1], so it validates and runs exactly as that op with k = 1.
mgs_status mgs_linear_scan_fwd(const float *a, const float *b, const float *h0, float *h, int64_t B,
                               int64_t T, int64_t D, void *workspace, size_t workspace_bytes,
                               mgs_stream_t stream) {
    if (D >= 0 && D % 4 != 0) return MGS_ERR_UNSUPPORTED;
    return mgs_matrix_affine_scan_fwd(a, b, h0, h, B, T, D, 1, workspace, workspace_bytes, stream);
}

mgs_status mgs_linear_scan_bwd(const float *a, const float *h0, const float *h, const float *grad_h,
                               float *da, float *db, float *dh0, int64_t B, int64_t T, int64_t D,
                               void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    if (D >= 0 && D % 4 != 0) return MGS_ERR_UNSUPPORTED;
    return mgs_matrix_affine_scan_bwd(a, h0, h, grad_h, da, db, dh0, B, T, D, 1, workspace, workspace_bytes,
                                      stream);
}

mgs_status mgs_givens_affine_scan_fwd(const float *theta, const float *a, const float *b,
                                      const float *h0, float *h, int64_t B, int64_t T, int64_t H,
                                      int k, void *workspace, size_t workspace_bytes,
                                      mgs_stream_t stream) {
    GivensSizes s;
    mgs_status st = givens_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.vec == 0) return MGS_OK;
    if ((st = check_ptrs({theta, b, h}, {a, h0})) != MGS_OK) return st;
    if (!disjoint({{h, s.vec}}, {{theta, s.ang}, {a, a ? s.vec : 0}, {b, s.vec}, {h0, h0 ? s.init : 0}}))
        return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::givens_workspace_bytes(0, B, T, H), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gas_fwd(theta, a, b, h0, h, B, T, H, workspace, workspace_bytes, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_givens_affine_scan_bwd(const float *theta, const float *a, const float *h0,
                                      const float *h, const float *grad_h, float *d_theta, float *da,
                                      float *db, float *dh0, int64_t B, int64_t T, int64_t H, int k,
                                      void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    GivensSizes s;
    mgs_status st = givens_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (da != nullptr && a == nullptr) return MGS_ERR_INVALID_ARG;
    if (s.init == 0) return MGS_OK;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (s.vec == 0) {  // T = 0: dh0 = 0
        if (dh0 == nullptr) return MGS_OK;
        if ((st = check_ptrs({dh0}, {})) != MGS_OK) return st;
        return from_cuda(cudaMemsetAsync(dh0, 0, size_t(s.init) * sizeof(float), cs));
    }
    if ((st = check_ptrs({theta, h, grad_h, d_theta, db}, {a, h0, da, dh0})) != MGS_OK) return st;
    if (!disjoint({{d_theta, s.ang}, {da, da ? s.vec : 0}, {db, s.vec}, {dh0, dh0 ? s.init : 0}},
                  {{theta, s.ang}, {a, a ? s.vec : 0}, {h0, h0 ? s.init : 0}, {h, s.vec}, {grad_h, s.vec}}))
        return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::givens_workspace_bytes(1, B, T, H), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gas_bwd(theta, a, h0, h, grad_h, d_theta, da, db, dh0, B, T, H, workspace,
                                         workspace_bytes, ctl, cs));
}

mgs_status mgs_givens_matrix_scan_fwd(const float *theta, float *P, int64_t B, int64_t T, int64_t H,
                                      int k, void *workspace, size_t workspace_bytes,
                                      mgs_stream_t stream) {
    GivensSizes s;
    mgs_status st = givens_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.mat == 0) return MGS_OK;
    if ((st = check_ptrs({theta, P}, {})) != MGS_OK) return st;
    if (!disjoint({{P, s.mat}}, {{theta, s.ang}})) return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::givens_workspace_bytes(2, B, T, H), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gms_fwd(theta, P, B, T, H, workspace, workspace_bytes, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_givens_matrix_scan_bwd(const float *theta, const float *P, const float *grad_P,
                                      float *d_theta, int64_t B, int64_t T, int64_t H, int k,
                                      void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    GivensSizes s;
    mgs_status st = givens_sizes(B, T, H, k, &s);
    if (st != MGS_OK) return st;
    if (s.mat == 0) return MGS_OK;
    if ((st = check_ptrs({theta, P, grad_P, d_theta}, {})) != MGS_OK) return st;
    if (!disjoint({{d_theta, s.ang}}, {{theta, s.ang}, {P, s.mat}, {grad_P, s.mat}})) return MGS_ERR_INVALID_ARG;
    if ((st = check_ws(mgs::givens_workspace_bytes(3, B, T, H), workspace, workspace_bytes)) != MGS_OK) return st;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gms_bwd(theta, P, grad_P, d_theta, B, T, H, workspace, workspace_bytes, ctl,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_delta_scan_fwd(const float *q, const float *k, const float *v, const float *beta,
                              const float *S0, float *o, float *S_T, int64_t B, int64_t T, int64_t H,
                              int D, void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    if (B < 0 || T < 0 || H < 0 || D <= 0) return MGS_ERR_INVALID_ARG;
    if (D != 64) return MGS_ERR_UNSUPPORTED;
    int64_t nb, n, ns;
    if (!mul_ok(B, T, &nb) || !mul_ok(nb, H, &nb) || !mul_ok(nb, D, &n) || !mul_ok(B, H, &ns) ||
        !mul_ok(ns, int64_t(D) * D, &ns))
        return MGS_ERR_INVALID_ARG;
    if (n > INT64_MAX / 8 || ns > INT64_MAX / 8) return MGS_ERR_INVALID_ARG;
    if (B * T > INT32_MAX || H > INT32_MAX) return MGS_ERR_UNSUPPORTED;  // 32-bit map coordinates
    if (ns == 0) return MGS_OK;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    mgs_status st;
    if (n == 0) {  // T = 0: the final state is the initial one
        if (S_T == nullptr) return MGS_OK;
        if ((st = check_ptrs({S_T}, {S0})) != MGS_OK) return st;
        if (!disjoint({{S_T, ns}}, {{S0, S0 ? ns : 0}})) return MGS_ERR_INVALID_ARG;
        return from_cuda(S0 ? cudaMemcpyAsync(S_T, S0, size_t(ns) * sizeof(float), cudaMemcpyDeviceToDevice, cs)
                            : cudaMemsetAsync(S_T, 0, size_t(ns) * sizeof(float), cs));
    }
    if ((st = check_ptrs({q, k, v, o}, {S0, S_T})) != MGS_OK) return st;
    if (beta == nullptr) return MGS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(beta) & 3u) != 0) return MGS_ERR_UNSUPPORTED;
    if (!disjoint({{o, n}, {S_T, S_T ? ns : 0}},
                  {{q, n}, {k, n}, {v, n}, {beta, nb}, {S0, S0 ? ns : 0}}))
        return MGS_ERR_INVALID_ARG;
    int64_t chunks;
    if (!mul_ok(B * H, (T + 63) / 64, &chunks) || chunks > INT32_MAX / (3 * 64)) return MGS_ERR_UNSUPPORTED;
    const size_t need = mgs::delta_workspace_bytes(B, T, H);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!disjoint({{static_cast<float *>(workspace), int64_t(need / sizeof(float))}},
                  {{q, n}, {k, n}, {v, n}, {beta, nb}, {S0, S0 ? ns : 0}, {o, n}, {S_T, S_T ? ns : 0}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_delta_fwd(q, k, v, beta, S0, o, S_T, B, T, H, workspace, ctl, cs));
}

mgs_status mgs_check(mgs_stream_t stream) {
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MGS_ERR_CUDA;
    mgs::DevCtl ctl;
    mgs_status st = current_ctl(&ctl);
    if (st != MGS_OK) return st;
    unsigned word = 0;
    if (cudaMemcpy(&word, ctl.err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return MGS_ERR_CUDA;
    if (word != 0) {
        if (cudaMemset(ctl.err, 0, sizeof(unsigned)) != cudaSuccess) return MGS_ERR_CUDA;
        return MGS_ERR_TIMEOUT;
    }
    return MGS_OK;
}

void mgs_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns < 1000 ? 1000 : ns); }

const char *mgs_status_string(mgs_status status) {
    switch (status) {
        case MGS_OK: return "MGS_OK";
        case MGS_ERR_INVALID_ARG: return "MGS_ERR_INVALID_ARG";
        case MGS_ERR_UNSUPPORTED: return "MGS_ERR_UNSUPPORTED";
        case MGS_ERR_WORKSPACE: return "MGS_ERR_WORKSPACE";
        case MGS_ERR_CUDA: return "MGS_ERR_CUDA";
        case MGS_ERR_TIMEOUT: return "MGS_ERR_TIMEOUT";
        default: return "MGS_ERR_UNKNOWN";
    }
}

int mgs_version(void) { return MGS_VERSION_INT; }

}  // extern "C"

// ---------------------------------------------------------------- diagnostic wait
namespace {
__global__ void debug_wait_flag_kernel(const int *flag, mgs::DevCtl ctl) {
    if (threadIdx.x != 0) return;
    const uint64_t t0 = mgs::global_ns();
    while (true) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v != 0) return;
        if (mgs::global_ns() - t0 > ctl.timeout_ns) {
            mgs::record_error(ctl, mgs::ERR_FLAG_TIMEOUT);
            return;
        }
        __nanosleep(1000);
    }
}
}  // namespace

extern "C" mgs_status mgs_debug_wait_flag(const int *flag, mgs_stream_t stream) {
    if (flag == nullptr) return MGS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(flag) & 3u) != 0) return MGS_ERR_UNSUPPORTED;
    mgs::DevCtl ctl;
    mgs_status st = current_ctl(&ctl);
    if (st != MGS_OK) return st;
    debug_wait_flag_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(flag, ctl);
    return from_cuda(cudaGetLastError());
}

// ---------------------------------------------------------------- language-model operators
namespace {

// Byte ranges of arguments, for the overlap checks of operators whose
// arguments differ in type.
struct Bytes {
    const void *p;
    int64_t n;
};
bool apart(std::initializer_list<Bytes> outs, std::initializer_list<Bytes> ins) {
    auto hit = [](const Bytes &a, const Bytes &b) {
        if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return x < y + uintptr_t(b.n) && y < x + uintptr_t(a.n);
    };
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto &i : ins)
            if (hit(*o, i)) return false;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (hit(*o, *o2)) return false;
    }
    return true;
}

int esize(int dtype) { return dtype == MGS_F32 ? 4 : dtype == MGS_BF16 ? 2 : 0; }

struct AttnSizes {
    int64_t qk, v, q_span, k_span, v_span, do_span;  // bytes: dense [B,T,Hk,D], [B,T,H,D]; spans of the strided inputs
    int64_t g, state;                                // bytes
};

// Bytes from the first to the last element of [B][T][h][D] with these
// strides; false when a stride is negative, no multiple of 16 bytes, or too large.
bool span_of(const int64_t (&st)[3], int64_t B, int64_t T, int64_t h, int64_t inner, int es, int mult, int64_t *out) {
    int64_t n = inner - 1, x;
    const int64_t dims[3] = {B, T, h};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || (dims[i] > 1 && (st[i] * es) % mult != 0)) return false;
        if (!mul_ok(dims[i] - 1, st[i], &x) || x > INT64_MAX / 64 - n) return false;
        n += x;
    }
    *out = (n + 1) * es;
    return true;
}

mgs_status attn_sizes(const mgs_attention_shape *sh, bool with_do, AttnSizes *z) {
    if (sh == nullptr || sh->B < 0 || sh->T < 0 || sh->H < 0 || sh->Hk < 0) return MGS_ERR_INVALID_ARG;
    const int es = esize(sh->dtype);
    if (es == 0 || (sh->D != 64 && sh->D != 128)) return MGS_ERR_UNSUPPORTED;
    if (sh->H > 0 && (sh->Hk == 0 || sh->H % sh->Hk != 0)) return MGS_ERR_INVALID_ARG;
    int64_t bt, n, ns;
    if (!mul_ok(sh->B, sh->T, &bt) || !mul_ok(bt, sh->H > 0 ? sh->H : sh->Hk, &n) || !mul_ok(n, int64_t(sh->D) * 8, &n) ||
        !mul_ok(sh->B, sh->H, &ns) || !mul_ok(ns, int64_t(sh->D) * sh->D * 4, &ns))
        return MGS_ERR_INVALID_ARG;
    if (n > INT64_MAX / 64 || ns > INT64_MAX / 64) return MGS_ERR_INVALID_ARG;
    // 32-bit grid and tensor-map coordinates
    if (sh->T > INT32_MAX / 2 || sh->B * sh->H > 65535 * 16 || (sh->T / 128 + 1) * sh->B * sh->H > INT32_MAX / 4)
        return MGS_ERR_UNSUPPORTED;
    z->qk = bt * sh->Hk * sh->D * es;
    z->v = bt * sh->H * sh->D * es;
    z->state = ns;
    z->q_span = z->k_span = z->v_span = z->do_span = z->g = 0;
    if (bt == 0 || sh->H == 0) return MGS_OK;
    if (!span_of(sh->q_stride, sh->B, sh->T, sh->Hk, sh->D, es, 16, &z->q_span) ||
        !span_of(sh->k_stride, sh->B, sh->T, sh->Hk, sh->D, es, 16, &z->k_span) ||
        !span_of(sh->v_stride, sh->B, sh->T, sh->H, sh->D, es, 16, &z->v_span) ||
        (with_do && !span_of(sh->do_stride, sh->B, sh->T, sh->H, sh->D, es, 16, &z->do_span)))
        return MGS_ERR_UNSUPPORTED;
    if (sh->fixed_decay)
        z->g = sh->H * 4;
    else if (!span_of(sh->g_stride, sh->B, sh->T, sh->H, 1, 4, 4, &z->g))
        return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

size_t mgs_linear_attention_workspace_size(const mgs_attention_shape *shape, int backward) {
    AttnSizes z;
    if (attn_sizes(shape, false, &z) != MGS_OK || z.v == 0) return 0;
    return mgs::attn_workspace_bytes(*shape, backward != 0);
}

mgs_status mgs_linear_attention_fwd(const mgs_attention_shape *shape, const void *q, const void *k, const void *v,
                                    const float *g, const float *S0, void *o, float *S_T, void *workspace,
                                    size_t workspace_bytes, mgs_stream_t stream) {
    AttnSizes z;
    mgs_status st = attn_sizes(shape, false, &z);
    if (st != MGS_OK) return st;
    if (z.state == 0) return MGS_OK;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (z.v == 0) {  // T = 0: the final state is the initial one
        if (S_T == nullptr) return MGS_OK;
        if ((st = check_ptrs({S_T}, {S0})) != MGS_OK) return st;
        if (!apart({{S_T, z.state}}, {{S0, z.state}})) return MGS_ERR_INVALID_ARG;
        return from_cuda(S0 ? cudaMemcpyAsync(S_T, S0, size_t(z.state), cudaMemcpyDeviceToDevice, cs)
                            : cudaMemsetAsync(S_T, 0, size_t(z.state), cs));
    }
    if ((st = check_ptrs({q, k, v, o}, {S0, S_T})) != MGS_OK) return st;
    if (g == nullptr) return MGS_ERR_INVALID_ARG;
    if (!aligned4(g)) return MGS_ERR_UNSUPPORTED;
    const size_t need = mgs::attn_workspace_bytes(*shape, false);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!apart({{o, z.v}, {S_T, z.state}, {workspace, int64_t(need)}},
               {{q, z.q_span}, {k, z.k_span}, {v, z.v_span}, {g, z.g}, {S0, z.state}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_attn_fwd(*shape, q, k, v, g, S0, o, S_T, workspace, ctl, cs));
}

mgs_status mgs_linear_attention_bwd(const mgs_attention_shape *shape, const void *q, const void *k, const void *v,
                                    const float *g, const float *S0, const void *grad_o, const float *grad_S_T,
                                    void *dq, void *dk, void *dv, float *dg, float *dS0, void *workspace,
                                    size_t workspace_bytes, mgs_stream_t stream) {
    AttnSizes z;
    mgs_status st = attn_sizes(shape, true, &z);
    if (st != MGS_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (z.v == 0) {  // T = 0: dS0 is the final state's gradient; a fixed decay has none
        if (z.qk > 0) {  // H = 0: no value head reads the queries and keys
            if ((st = check_ptrs({dq, dk}, {})) != MGS_OK) return st;
            if (!apart({{dq, z.qk}, {dk, z.qk}}, {})) return MGS_ERR_INVALID_ARG;
            if (cudaMemsetAsync(dq, 0, size_t(z.qk), cs) != cudaSuccess || cudaMemsetAsync(dk, 0, size_t(z.qk), cs) != cudaSuccess)
                return MGS_ERR_CUDA;
        }
        if (shape->fixed_decay && dg != nullptr && shape->H > 0) {
            if (!aligned4(dg)) return MGS_ERR_UNSUPPORTED;
            if (cudaMemsetAsync(dg, 0, size_t(shape->H) * 4, cs) != cudaSuccess) return MGS_ERR_CUDA;
        }
        if (z.state == 0 || dS0 == nullptr) return MGS_OK;
        if ((st = check_ptrs({dS0}, {grad_S_T})) != MGS_OK) return st;
        if (!apart({{dS0, z.state}}, {{grad_S_T, z.state}})) return MGS_ERR_INVALID_ARG;
        return from_cuda(grad_S_T
                             ? cudaMemcpyAsync(dS0, grad_S_T, size_t(z.state), cudaMemcpyDeviceToDevice, cs)
                             : cudaMemsetAsync(dS0, 0, size_t(z.state), cs));
    }
    if ((st = check_ptrs({q, k, v, grad_o, dq, dk, dv}, {S0, grad_S_T, dS0})) != MGS_OK) return st;
    if (g == nullptr || dg == nullptr) return MGS_ERR_INVALID_ARG;
    if (!aligned4(g) || !aligned4(dg)) return MGS_ERR_UNSUPPORTED;
    const size_t need = mgs::attn_workspace_bytes(*shape, true);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    const int64_t ndg = (shape->fixed_decay ? shape->H : shape->B * shape->T * shape->H) * 4;
    if (!apart({{dq, z.qk}, {dk, z.qk}, {dv, z.v}, {dg, ndg}, {dS0, z.state}, {workspace, int64_t(need)}},
               {{q, z.q_span}, {k, z.k_span}, {v, z.v_span}, {g, z.g}, {S0, z.state}, {grad_o, z.do_span},
                {grad_S_T, z.state}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_attn_bwd(*shape, q, k, v, g, S0, grad_o, grad_S_T, dq, dk, dv, dg, dS0, workspace,
                                          ctl, cs));
}

mgs_status mgs_linear_attention_step(const mgs_attention_shape *shape, const void *q, const void *k, const void *v,
                                     const float *g, float *S, const int32_t *slots, int64_t n_slots, void *o,
                                     mgs_stream_t stream) {
    AttnSizes z;
    if (shape == nullptr || shape->T != 1 || n_slots < 0) return MGS_ERR_INVALID_ARG;
    mgs_status st = attn_sizes(shape, false, &z);
    if (st != MGS_OK) return st;
    if (z.state == 0) return MGS_OK;
    if ((st = check_ptrs({q, k, v, o, S}, {})) != MGS_OK) return st;
    if (g == nullptr || (slots == nullptr && n_slots < shape->B)) return MGS_ERR_INVALID_ARG;
    if (!aligned4(g) || !aligned4(slots)) return MGS_ERR_UNSUPPORTED;
    int64_t ns;
    if (!mul_ok(n_slots, shape->H * shape->D * int64_t(shape->D) * 4, &ns)) return MGS_ERR_INVALID_ARG;
    if (!apart({{o, z.v}, {S, ns}},
               {{q, z.q_span}, {k, z.k_span}, {v, z.v_span}, {g, z.g}, {slots, slots ? shape->B * 4 : 0}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_attn_step(*shape, q, k, v, g, S, slots, n_slots, o,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

// rows x N elements of the type, as bytes
static mgs_status norm_sizes(int dtype, int64_t rows, int64_t N, int64_t *bytes) {
    if (rows < 0 || N < 0) return MGS_ERR_INVALID_ARG;
    if (esize(dtype) == 0 || N > INT32_MAX / 2) return MGS_ERR_UNSUPPORTED;
    if (!mul_ok(rows, N, bytes) || *bytes > INT64_MAX / 64) return MGS_ERR_INVALID_ARG;
    if (rows > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    *bytes *= esize(dtype);
    return MGS_OK;
}
static mgs_status typed_ptrs(int es, std::initializer_list<const void *> required,
                             std::initializer_list<const void *> optional) {
    for (const void *p : required) {
        if (p == nullptr) return MGS_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(p) % unsigned(es)) return MGS_ERR_UNSUPPORTED;
    }
    for (const void *p : optional)
        if (reinterpret_cast<uintptr_t>(p) % unsigned(es)) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

mgs_status mgs_rms_norm_fwd(const void *x, const void *residual, const void *weight, float eps, void *r, void *y,
                            float *rstd, int64_t rows, int64_t N, int dtype, mgs_stream_t stream) {
    int64_t n;
    mgs_status st = norm_sizes(dtype, rows, N, &n);
    if (st != MGS_OK) return st;
    if (n == 0) {  // rows of nothing: their mean is none
        if (rows == 0 || rstd == nullptr) return MGS_OK;
        if (!aligned4(rstd)) return MGS_ERR_UNSUPPORTED;
        return from_cuda(cudaMemsetAsync(rstd, 0xff, size_t(rows) * 4, reinterpret_cast<cudaStream_t>(stream)));  // NaN
    }
    const int es = esize(dtype);
    if ((st = typed_ptrs(es, {x, weight, y}, {residual, r})) != MGS_OK) return st;
    if ((residual == nullptr) != (r == nullptr)) return MGS_ERR_INVALID_ARG;
    if (!aligned4(rstd)) return MGS_ERR_UNSUPPORTED;
    if (!apart({{r, n}, {y, n}, {rstd, rows * 4}}, {{x, n}, {residual, n}, {weight, N * es}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_rms_norm_fwd(dtype, x, residual, weight, eps, r, y, rstd, rows, N,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

mgs_status mgs_rms_norm_fp8_fwd(const void *x, const void *residual, const void *weight, float eps, void *r, void *q,
                                float *scales, int64_t rows, int64_t N, int group, int dtype, mgs_stream_t stream) {
    int64_t n;
    mgs_status st = norm_sizes(dtype, rows, N, &n);
    if (st != MGS_OK) return st;
    if (group != 0 && (group != 128 || N % 128 != 0)) return MGS_ERR_UNSUPPORTED;
    if (n == 0) {  // rows of nothing: no value has a magnitude
        if (rows == 0 || group != 0) return MGS_OK;
        if (scales == nullptr) return MGS_ERR_INVALID_ARG;
        if (!aligned4(scales)) return MGS_ERR_UNSUPPORTED;
        return from_cuda(cudaMemsetAsync(scales, 0, size_t(rows) * 4, reinterpret_cast<cudaStream_t>(stream)));
    }
    const int es = esize(dtype);
    if ((st = typed_ptrs(es, {x, weight, q}, {residual, r})) != MGS_OK) return st;
    if (scales == nullptr || (residual == nullptr) != (r == nullptr)) return MGS_ERR_INVALID_ARG;
    if (!aligned4(scales)) return MGS_ERR_UNSUPPORTED;
    const int64_t nsc = rows * (group ? N / group : 1) * 4;
    if (!apart({{r, n}, {q, n / es}, {scales, nsc}}, {{x, n}, {residual, n}, {weight, N * es}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_rms_norm_fp8(dtype, x, residual, weight, eps, r, q, scales, rows, N, group,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

size_t mgs_rms_norm_bwd_workspace_size(int64_t rows, int64_t N) {
    int64_t n;
    if (norm_sizes(MGS_F32, rows, N, &n) != MGS_OK || n == 0) return 0;
    return mgs::rms_norm_bwd_workspace_bytes(rows, N);
}

mgs_status mgs_rms_norm_bwd(const void *r, const void *weight, const float *rstd, const void *grad_y,
                            const void *grad_r, void *dx, void *dweight, int64_t rows, int64_t N, int dtype,
                            void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    int64_t n;
    mgs_status st = norm_sizes(dtype, rows, N, &n);
    if (st != MGS_OK) return st;
    const int es = esize(dtype);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {  // no rows: the weight's gradient is zero
        if (N == 0) return MGS_OK;
        if ((st = typed_ptrs(es, {dweight}, {})) != MGS_OK) return st;
        return from_cuda(cudaMemsetAsync(dweight, 0, size_t(N) * es, cs));
    }
    if ((st = typed_ptrs(es, {r, weight, grad_y, dx, dweight}, {grad_r})) != MGS_OK) return st;
    if (rstd == nullptr) return MGS_ERR_INVALID_ARG;
    if (!aligned4(rstd)) return MGS_ERR_UNSUPPORTED;
    const size_t need = mgs::rms_norm_bwd_workspace_bytes(rows, N);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!apart({{dx, n}, {dweight, N * es}, {workspace, int64_t(need)}},
               {{r, n}, {weight, N * es}, {rstd, rows * 4}, {grad_y, n}, {grad_r, n}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_rms_norm_bwd(dtype, r, weight, rstd, grad_y, grad_r, dx, dweight, rows, N, workspace,
                                              cs));
}

// The byte ranges that a call on many tensors reads (of those that it does not
// write in place) and writes.
struct Span {
    uintptr_t lo, hi;
};
static void by_address(Span *s, int64_t n) {
    auto before = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);  // gradients mostly lie in their order
}
// Whether no written range meets another one, read or written: in the order of
// their addresses, none of a pair that meets begins behind the other's end.
static bool written_apart(Span *in, int64_t nin, Span *out, int64_t nout) {
    by_address(in, nin), by_address(out, nout);
    uintptr_t read = 0, written = 0;  // the furthest ends so far
    for (int64_t i = 0, j = 0; i < nin || j < nout;) {
        if (j == nout || (i < nin && in[i].lo < out[j].lo)) {
            if (in[i].lo < written) return false;
            read = std::max(read, in[i++].hi);
        } else {
            if (out[j].lo < std::max(read, written)) return false;
            written = out[j++].hi;
        }
    }
    return true;
}

size_t mgs_clip_grad_norm_workspace_size(int64_t count) { return count < 0 ? 0 : mgs::clip_workspace_bytes(count); }

mgs_status mgs_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numels,
                              const int32_t *dtypes, int64_t count, float max_norm, float *norm, void *workspace,
                              size_t workspace_bytes, mgs_stream_t stream) {
    if (count < 0 || norm == nullptr || !(max_norm >= 0.f)) return MGS_ERR_INVALID_ARG;
    if (!aligned4(norm)) return MGS_ERR_UNSUPPORTED;
    if (count > 0 && (grads == nullptr || outs == nullptr || numels == nullptr || dtypes == nullptr))
        return MGS_ERR_INVALID_ARG;
    const size_t need = mgs::clip_workspace_bytes(count);
    if (count > (int64_t(1) << 32)) return MGS_ERR_UNSUPPORTED;
    Span few[512];
    std::unique_ptr<Span[]> many(2 * count > 512 ? new (std::nothrow) Span[2 * count] : nullptr);
    if (2 * count > 512 && many == nullptr) return MGS_ERR_UNSUPPORTED;  // more tensors than the host has memory for
    Span *const reads = many ? many.get() : few, *const writes = reads + count;
    int64_t nreads = 0, nwrites = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int es = esize(dtypes[i]);
        if (es == 0) return MGS_ERR_UNSUPPORTED;
        if (numels[i] < 0 || numels[i] > INT64_MAX / 64) return MGS_ERR_INVALID_ARG;
        if (numels[i] == 0) continue;
        mgs_status st = typed_ptrs(es, {grads[i], outs[i]}, {});
        if (st != MGS_OK) return st;
        const Bytes in{grads[i], numels[i] * es}, out{outs[i], numels[i] * es};
        const uintptr_t a = reinterpret_cast<uintptr_t>(in.p), b = reinterpret_cast<uintptr_t>(out.p);
        if (a != b) reads[nreads++] = {a, a + uintptr_t(in.n)};
        writes[nwrites++] = {b, b + uintptr_t(out.n)};
        if (!apart({{norm, 4}, {workspace, int64_t(need)}}, {in, out})) return MGS_ERR_INVALID_ARG;
    }
    if (!written_apart(reads, nreads, writes, nwrites)) return MGS_ERR_INVALID_ARG;
    const mgs_status st = check_ws(need, workspace, workspace_bytes);
    if (st != MGS_OK) return st;
    return from_cuda(mgs::launch_clip(grads, outs, numels, dtypes, count, max_norm, norm, workspace,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

static cudaStream_t cs_of(mgs_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// ---------------------------------------------------------------- gated linear recurrence
struct GatedSizes {
    int64_t n, gate, value, gh, state, carries;  // bytes: dense, spans of the strided inputs, [B,D] and the carries in fp32
};

static mgs_status gated_sizes(const mgs_gated_shape *sh, bool with_gh, GatedSizes *z) {
    if (sh == nullptr || sh->B < 0 || sh->T < 0 || sh->D < 0) return MGS_ERR_INVALID_ARG;
    const int es = esize(sh->dtype);
    if (es == 0) return MGS_ERR_UNSUPPORTED;
    int64_t bt, n, bd;
    if (!mul_ok(sh->B, sh->T, &bt) || !mul_ok(bt, sh->D, &n) || !mul_ok(sh->B, sh->D, &bd) || n > INT64_MAX / 64 ||
        bd > INT64_MAX / 64)
        return MGS_ERR_INVALID_ARG;
    // 32-bit grids and steps
    if (sh->T > INT32_MAX / 2 || sh->D > INT32_MAX / 2 || sh->B > INT32_MAX || bd > (int64_t(1) << 34))
        return MGS_ERR_UNSUPPORTED;
    *z = {n * es, 0, 0, 0, bd * 4, sh->B * ((sh->T + MGS_GATED_SPAN - 1) / MGS_GATED_SPAN) * sh->D * 4};
    if (n == 0) return MGS_OK;
    auto span = [&](const int64_t (&st)[2], int64_t *out) {
        const int64_t s3[3] = {st[0], st[1], 0};
        return span_of(s3, sh->B, sh->T, 1, sh->D, es, es, out);
    };
    if (!span(sh->gate_stride, &z->gate) || !span(sh->value_stride, &z->value) ||
        (with_gh && !span(sh->gh_stride, &z->gh)))
        return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}
// T = 0: one [B,D] in fp32 is another, or zeros
static mgs_status pass_state(float *out, const float *in, int64_t bytes, cudaStream_t cs) {
    if (out == nullptr || bytes == 0) return MGS_OK;
    if (!aligned4(out) || !aligned4(in)) return MGS_ERR_UNSUPPORTED;
    if (!apart({{out, bytes}}, {{in, bytes}})) return MGS_ERR_INVALID_ARG;
    return from_cuda(in ? cudaMemcpyAsync(out, in, size_t(bytes), cudaMemcpyDeviceToDevice, cs)
                        : cudaMemsetAsync(out, 0, size_t(bytes), cs));
}

mgs_status mgs_gated_scan_fwd(const mgs_gated_shape *shape, const void *gate, const void *value, const float *h0,
                              void *h, float *h_T, float *carries, mgs_stream_t stream) {
    GatedSizes z;
    mgs_status st = gated_sizes(shape, false, &z);
    if (st != MGS_OK) return st;
    const cudaStream_t cs = cs_of(stream);
    if (z.n == 0) return pass_state(h_T, h0, z.state, cs);
    if ((st = typed_ptrs(esize(shape->dtype), {gate, value, h}, {})) != MGS_OK) return st;
    if ((st = typed_ptrs(4, {}, {h0, h_T, carries})) != MGS_OK) return st;
    if (!apart({{h, z.n}, {h_T, z.state}, {carries, z.carries}}, {{gate, z.gate}, {value, z.value}, {h0, z.state}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gated_fwd(*shape, gate, value, h0, h, h_T, carries, ctl, cs));
}

mgs_status mgs_gated_scan_bwd(const mgs_gated_shape *shape, const void *gate, const void *value, const float *carries,
                              const void *grad_h, const float *grad_h_T, void *d_gate, void *d_value, float *d_h0,
                              mgs_stream_t stream) {
    GatedSizes z;
    mgs_status st = gated_sizes(shape, true, &z);
    if (st != MGS_OK) return st;
    const cudaStream_t cs = cs_of(stream);
    if (z.n == 0) return pass_state(d_h0, grad_h_T, z.state, cs);
    if ((st = typed_ptrs(esize(shape->dtype), {gate, value, grad_h, d_gate, d_value}, {})) != MGS_OK) return st;
    if ((st = typed_ptrs(4, {carries}, {grad_h_T, d_h0})) != MGS_OK) return st;
    if (!apart({{d_gate, z.n}, {d_value, z.n}, {d_h0, z.state}},
               {{gate, z.gate}, {value, z.value}, {carries, z.carries}, {grad_h, z.gh}, {grad_h_T, z.state}}))
        return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    if ((st = current_ctl(&ctl)) != MGS_OK) return st;
    return from_cuda(mgs::launch_gated_bwd(*shape, gate, value, carries, grad_h, grad_h_T, d_gate, d_value, d_h0, ctl, cs));
}

mgs_status mgs_gated_scan_step(const mgs_gated_shape *shape, const void *gate, const void *value, float *state,
                               const int32_t *slots, int64_t n_slots, void *h, mgs_stream_t stream) {
    GatedSizes z;
    if (shape == nullptr || shape->T != 1 || n_slots < 0) return MGS_ERR_INVALID_ARG;
    mgs_status st = gated_sizes(shape, false, &z);
    if (st != MGS_OK) return st;
    if (z.n == 0) return MGS_OK;
    if ((st = typed_ptrs(esize(shape->dtype), {gate, value, h}, {})) != MGS_OK) return st;
    if ((st = typed_ptrs(4, {state}, {slots})) != MGS_OK) return st;
    if (slots == nullptr && n_slots < shape->B) return MGS_ERR_INVALID_ARG;
    int64_t ns;
    if (!mul_ok(n_slots, shape->D * 4, &ns) || ns > INT64_MAX / 64) return MGS_ERR_INVALID_ARG;
    if (!apart({{h, z.n}, {state, ns}}, {{gate, z.gate}, {value, z.value}, {slots, slots ? shape->B * 4 : 0}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_gated_step(*shape, gate, value, state, slots, n_slots, h, cs_of(stream)));
}

mgs_status mgs_debug_exchange(int32_t late_block, int32_t late_round, uint64_t late_ns, int32_t *rounds, int32_t *wrong,
                              mgs_stream_t stream) {
    if (rounds == nullptr || wrong == nullptr || late_ns > 1000000000ull) return MGS_ERR_INVALID_ARG;
    if (!aligned4(rounds) || !aligned4(wrong)) return MGS_ERR_UNSUPPORTED;
    constexpr int64_t n = MGS_EXCHANGE_BLOCKS * 4;
    if (!apart({{rounds, n}, {wrong, n}}, {})) return MGS_ERR_INVALID_ARG;
    mgs::DevCtl ctl;
    const mgs_status st = current_ctl(&ctl);
    if (st != MGS_OK) return st;
    return from_cuda(mgs::launch_exchange_check(late_block, late_round, late_ns, rounds, wrong, ctl, cs_of(stream)));
}

// ---------------------------------------------------------------- norm of queries and keys
struct QkSizes {
    int64_t q, k, q_span, k_span, gq_span, gk_span, table, pos;  // bytes
};

static mgs_status qk_sizes(const mgs_qk_norm_shape *sh, bool bwd, bool positions, QkSizes *z) {
    if (sh == nullptr || sh->B < 0 || sh->T < 0 || sh->Hq < 0 || sh->Hk < 0 || sh->positions < 0)
        return MGS_ERR_INVALID_ARG;
    const int es = esize(sh->dtype);
    if (es == 0 || sh->D <= 0 || sh->D > 256 || sh->D % 8 != 0 || sh->rotary < 0 || sh->rotary > sh->D ||
        sh->rotary % 8 != 0)
        return MGS_ERR_UNSUPPORTED;
    int64_t bt, nq, nk;
    if (!mul_ok(sh->B, sh->T, &bt) || !mul_ok(bt, sh->Hq, &nq) || !mul_ok(bt, sh->Hk, &nk) ||
        nq > INT64_MAX / (64 * 256 * 4) || nk > INT64_MAX / (64 * 256 * 4) || sh->positions > INT64_MAX / (64 * 256 * 4))
        return MGS_ERR_INVALID_ARG;
    // 32-bit counts of tokens and of a warp's heads
    if (sh->Hq > (1 << 20) || sh->Hk > (1 << 20) || bt > INT32_MAX / 2) return MGS_ERR_UNSUPPORTED;
    *z = {nq * sh->D * es, nk * sh->D * es, 0, 0, 0, 0, sh->positions * sh->rotary * 4, 0};
    if (nq + nk == 0) return MGS_OK;
    auto span = [&](const int64_t (&st)[3], int64_t H, int64_t *out) {
        return H == 0 || span_of(st, sh->B, sh->T, H, sh->D, es, es, out);
    };
    if (!span(sh->q_stride, sh->Hq, &z->q_span) || !span(sh->k_stride, sh->Hk, &z->k_span) ||
        (bwd && (!span(sh->gq_stride, sh->Hq, &z->gq_span) || !span(sh->gk_stride, sh->Hk, &z->gk_span))))
        return MGS_ERR_UNSUPPORTED;
    if (sh->rotary > 0 && positions) {
        const int64_t st[3] = {sh->pos_stride[0], sh->pos_stride[1], 0};
        if (!span_of(st, sh->B, sh->T, 1, 1, 4, 4, &z->pos)) return MGS_ERR_UNSUPPORTED;
    }
    return MGS_OK;
}
// the arguments that both passes read
static mgs_status qk_inputs(const mgs_qk_norm_shape *sh, const void *q, const void *k, const void *qw, const void *kw,
                            const float *table, const int32_t *pos) {
    const int es = esize(sh->dtype);
    mgs_status st = typed_ptrs(es, {}, {q, k, qw, kw});
    if (st != MGS_OK) return st;
    if ((sh->Hq > 0 && q == nullptr) || (sh->Hk > 0 && k == nullptr)) return MGS_ERR_INVALID_ARG;
    if ((sh->rotary > 0) != (table != nullptr) || (pos != nullptr && table == nullptr)) return MGS_ERR_INVALID_ARG;
    if (sh->rotary > 0 && pos == nullptr && sh->positions < sh->T) return MGS_ERR_INVALID_ARG;
    return aligned16(table) && aligned4(pos) ? MGS_OK : MGS_ERR_UNSUPPORTED;
}

mgs_status mgs_qk_norm_fwd(const mgs_qk_norm_shape *shape, const void *q, const void *k, const void *q_weight,
                           const void *k_weight, const float *table, const int32_t *token_positions, void *yq,
                           void *yk, mgs_stream_t stream) {
    QkSizes z;
    mgs_status st = qk_sizes(shape, false, token_positions != nullptr, &z);
    if (st != MGS_OK) return st;
    if (z.q + z.k == 0) return MGS_OK;
    if ((st = qk_inputs(shape, q, k, q_weight, k_weight, table, token_positions)) != MGS_OK) return st;
    const int es = esize(shape->dtype);
    if ((st = typed_ptrs(es, {}, {yq, yk})) != MGS_OK) return st;
    if ((z.q > 0 && yq == nullptr) || (z.k > 0 && yk == nullptr)) return MGS_ERR_INVALID_ARG;
    const int64_t nw = shape->D * es;
    if (!apart({{yq, z.q}, {yk, z.k}},
               {{q, z.q_span}, {k, z.k_span}, {q_weight, nw}, {k_weight, nw}, {table, z.table}, {token_positions, z.pos}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_qk_norm_fwd(*shape, q, k, q_weight, k_weight, table, token_positions, yq, yk,
                                             cs_of(stream)));
}

size_t mgs_qk_norm_bwd_workspace_size(const mgs_qk_norm_shape *shape) {
    QkSizes z;
    if (qk_sizes(shape, true, false, &z) != MGS_OK || z.q + z.k == 0) return 0;
    return mgs::qk_norm_bwd_workspace_bytes(*shape);
}

mgs_status mgs_qk_norm_bwd(const mgs_qk_norm_shape *shape, const void *q, const void *k, const void *q_weight,
                           const void *k_weight, const void *grad_yq, const void *grad_yk, const float *table,
                           const int32_t *token_positions, void *dq, void *dk, void *dq_weight, void *dk_weight,
                           void *workspace, size_t workspace_bytes, mgs_stream_t stream) {
    QkSizes z;
    mgs_status st = qk_sizes(shape, true, token_positions != nullptr, &z);
    if (st != MGS_OK) return st;
    const int es = esize(shape->dtype);
    const int64_t nw = shape->D * es;
    if ((st = typed_ptrs(es, {}, {dq_weight, dk_weight})) != MGS_OK) return st;
    if (z.q + z.k == 0) {  // no heads: the weights' gradients are zero
        if (!apart({{dq_weight, nw}, {dk_weight, nw}}, {})) return MGS_ERR_INVALID_ARG;
        for (void *dw : {dq_weight, dk_weight})
            if (dw != nullptr && cudaMemsetAsync(dw, 0, size_t(nw), cs_of(stream)) != cudaSuccess) return MGS_ERR_CUDA;
        return MGS_OK;
    }
    if ((st = qk_inputs(shape, q, k, q_weight, k_weight, table, token_positions)) != MGS_OK) return st;
    if ((st = typed_ptrs(es, {}, {grad_yq, grad_yk, dq, dk})) != MGS_OK) return st;
    if ((z.q > 0 && (grad_yq == nullptr || dq == nullptr)) || (z.k > 0 && (grad_yk == nullptr || dk == nullptr)))
        return MGS_ERR_INVALID_ARG;
    const size_t need = mgs::qk_norm_bwd_workspace_bytes(*shape);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!apart({{dq, z.q}, {dk, z.k}, {dq_weight, nw}, {dk_weight, nw}, {workspace, int64_t(need)}},
               {{q, z.q_span}, {k, z.k_span}, {q_weight, nw}, {k_weight, nw}, {grad_yq, z.gq_span},
                {grad_yk, z.gk_span}, {table, z.table}, {token_positions, z.pos}}))
        return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_qk_norm_bwd(*shape, q, k, q_weight, k_weight, grad_yq, grad_yk, table,
                                             token_positions, dq, dk, dq_weight, dk_weight, workspace, cs_of(stream)));
}

// ---------------------------------------------------------------- embedding
static mgs_status embed_sizes(int token_type, int64_t N, int64_t V, int64_t D, int dtype, int64_t *tokens, int64_t *rows,
                              int64_t *table) {
    if (N < 0 || V < 0 || D < 0) return MGS_ERR_INVALID_ARG;
    const int es = esize(dtype);
    if (es == 0 || (token_type != MGS_I32 && token_type != MGS_I64)) return MGS_ERR_UNSUPPORTED;
    if (!mul_ok(N, D, rows) || !mul_ok(V, D, table) || *rows > INT64_MAX / 64 || *table > INT64_MAX / 64)
        return MGS_ERR_INVALID_ARG;
    // 32-bit places in the sorted order, 16-bit grids over the columns
    if (N > INT32_MAX / 2 || V > INT32_MAX / 2 || D > (1 << 22)) return MGS_ERR_UNSUPPORTED;
    *tokens = N * (token_type == MGS_I64 ? 8 : 4), *rows *= es, *table *= es;
    return MGS_OK;
}
static bool aligned_tokens(int token_type, const void *p) {
    return reinterpret_cast<uintptr_t>(p) % (token_type == MGS_I64 ? 8 : 4) == 0;
}

mgs_status mgs_embedding_fwd(const void *tokens, int token_type, const void *weight, float scale, void *out,
                             int64_t N, int64_t V, int64_t D, int dtype, mgs_stream_t stream) {
    int64_t nt, nr, nw;
    mgs_status st = embed_sizes(token_type, N, V, D, dtype, &nt, &nr, &nw);
    if (st != MGS_OK) return st;
    if (nr == 0) return MGS_OK;
    if (tokens == nullptr || (weight == nullptr && nw > 0)) return MGS_ERR_INVALID_ARG;
    if ((st = typed_ptrs(esize(dtype), {out}, {weight})) != MGS_OK) return st;
    if (!aligned_tokens(token_type, tokens)) return MGS_ERR_UNSUPPORTED;
    if (!apart({{out, nr}}, {{tokens, nt}, {weight, nw}})) return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_embed_fwd(token_type, dtype, tokens, weight, scale, out, N, V, D, cs_of(stream)));
}

size_t mgs_embedding_bwd_workspace_size(int64_t N, int64_t V, int64_t D) {
    int64_t nt, nr, nw;
    if (embed_sizes(MGS_I64, N, V, D, MGS_F32, &nt, &nr, &nw) != MGS_OK || nr == 0 || nw == 0) return 0;
    return mgs::embed_bwd_workspace_bytes(N, V, D);
}

mgs_status mgs_embedding_bwd(const void *tokens, int token_type, const void *grad, int64_t grad_stride, float scale,
                             void *dweight, int64_t N, int64_t V, int64_t D, int dtype, void *workspace,
                             size_t workspace_bytes, mgs_stream_t stream) {
    int64_t nt, nr, nw;
    mgs_status st = embed_sizes(token_type, N, V, D, dtype, &nt, &nr, &nw);
    if (st != MGS_OK) return st;
    if (nw == 0) return MGS_OK;
    const int es = esize(dtype);
    if ((st = typed_ptrs(es, {dweight}, {grad})) != MGS_OK) return st;
    if (N == 0) return from_cuda(cudaMemsetAsync(dweight, 0, size_t(nw), cs_of(stream)));
    if (tokens == nullptr || grad == nullptr) return MGS_ERR_INVALID_ARG;
    if (!aligned_tokens(token_type, tokens)) return MGS_ERR_UNSUPPORTED;
    int64_t span;
    const int64_t gs[3] = {grad_stride, 0, 0};
    if (!span_of(gs, N, 1, 1, D, es, es, &span)) return MGS_ERR_UNSUPPORTED;
    const size_t need = mgs::embed_bwd_workspace_bytes(N, V, D);
    if ((st = check_ws(need, workspace, workspace_bytes)) != MGS_OK) return st;
    if (!apart({{dweight, nw}, {workspace, int64_t(need)}}, {{tokens, nt}, {grad, span}})) return MGS_ERR_INVALID_ARG;
    return from_cuda(mgs::launch_embed_bwd(token_type, dtype, tokens, grad, grad_stride, scale, dweight, N, V, D,
                                           workspace, cs_of(stream)));
}

}  // extern "C"
