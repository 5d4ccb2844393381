// The C ABI of the library (declared in include/fa.h): argument checks, TMA
// descriptor encoding, the per-device error word and the kernel launches.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_paged.h"
#include "fa_score.h"
#include "fa_window.h"
#include "ptx.cuh"

// Two error words per device, of timeouts and of pages (each device holds its own copy of
// this variable; host code must look its address up per device).
__device__ unsigned int g_fa_error_word[2];

namespace fa {
namespace {

constexpr unsigned long long kDefaultWaitLimitNs = 2000000000ull;
std::atomic<unsigned long long> g_wait_limit_ns{kDefaultWaitLimitNs};
thread_local cudaEvent_t t_ev_start = nullptr;  // fa_set_timing_events
thread_local cudaEvent_t t_ev_stop = nullptr;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

typedef CUresult (*CtxGetCurrentFn)(CUcontext*);

// A function of the driver as of a CUDA version, or null.
void* driver_fn(const char* name, unsigned version) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &p, version, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
        return nullptr;
    return p;
}
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(driver_fn("cuTensorMapEncodeTiled", 12000));
    return fn;
}
CtxGetCurrentFn get_current_fn() {
    static const CtxGetCurrentFn fn = reinterpret_cast<CtxGetCurrentFn>(driver_fn("cuCtxGetCurrent", 4000));
    return fn;
}

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    std::once_flag once;
    bool supported = false;
    unsigned int* err_word = nullptr;  // device address of g_fa_error_word[0]
};
DeviceInfo g_dev[kMaxDevices];

// Checks the current device once: it must be sm_103 and the error word's
// device address must resolve.  Returns nullptr if the device is unusable.
DeviceInfo* current_device(fa_status* why) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        *why = FA_ERR_CUDA;
        return nullptr;
    }
    // A thread that has made no call of the runtime that needs one (autograd's workers are such) has no current
    // context, without which descriptors cannot be encoded: it gets the device's primary one.  A context that the
    // caller has made current stays.
    CUcontext now = nullptr;
    const CtxGetCurrentFn get_current = get_current_fn();
    if (get_current == nullptr || get_current(&now) != CUDA_SUCCESS || (now == nullptr && cudaSetDevice(dev) != cudaSuccess)) {
        cudaGetLastError();
        *why = FA_ERR_CUDA;
        return nullptr;
    }
    DeviceInfo& di = g_dev[dev];
    std::call_once(di.once, [&di, dev] {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        if (major != 10 || minor != 3) return;
        void* addr = nullptr;
        if (cudaGetSymbolAddress(&addr, g_fa_error_word) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        di.err_word = static_cast<unsigned int*>(addr);
        di.supported = true;
    });
    if (!di.supported) {
        *why = FA_ERR_UNSUPPORTED;
        return nullptr;
    }
    return &di;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Shape checks common to every call.  Returns FA_OK and sets *empty when the
// problem has no rows.
fa_status check_shape(int B, int H, int N, int d, float tau, int causal, bool* empty) {
    if (B < 0 || H < 0 || N < 0 || d < 0) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(tau) && tau > 0.f)) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    *empty = (B == 0 || H == 0 || N == 0);
    if (d != 64 && d != 128) return *empty ? FA_OK : FA_ERR_UNSUPPORTED;
    if (*empty) return FA_OK;
    const long long bh = static_cast<long long>(B) * H;
    if (bh > INT_MAX) return FA_ERR_UNSUPPORTED;
    // grid.y holds 256-row query-tile pairs (forward) and 128-row key tiles (backward)
    if ((static_cast<long long>(N) + 127) / 128 > 65535) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

fa_status map_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Block-mask checks: mask_heads is 1 or B*H and the mask fits the kernels'
// per-tile bit sets.  Sets *bytes (the mask's size) and *head_stride.
fa_status check_blocks(const uint8_t* blocks, int mask_heads, int B, int H, int N, size_t* bytes,
                       long long* head_stride) {
    if (blocks == nullptr) return FA_ERR_INVALID_ARG;
    const long long bh = static_cast<long long>(B) * H;
    if (mask_heads != 1 && mask_heads != bh) return FA_ERR_INVALID_ARG;
    const long long nb = (static_cast<long long>(N) + kMaskBlockEdge - 1) / kMaskBlockEdge;
    if (nb > kMaxMaskBlocks) return FA_ERR_UNSUPPORTED;
    *bytes = static_cast<size_t>(mask_heads) * static_cast<size_t>(nb * nb);
    *head_stride = mask_heads == 1 ? 0 : nb * nb;
    return FA_OK;
}

fa_status fwd_common(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                     int N, int d, float tau, int causal, void* stream, bool o32, int window = 0,
                     const uint8_t* blocks = nullptr, int mask_heads = 0, int sinks = 0) {
    bool empty = false;
    fa_status s = check_shape(B, H, N, d, tau, causal, &empty);
    if (s != FA_OK || empty) return s;
    size_t mask_bytes = 0;
    long long mask_stride = 0;
    if (mask_heads != 0) {
        s = check_blocks(blocks, mask_heads, B, H, N, &mask_bytes, &mask_stride);
        if (s != FA_OK) return s;
    }
    const void* ptrs[] = {Q, K, V, O, LSE};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(B) * H * N;
    const size_t in_bytes = rows * d * 2, o_bytes = rows * d * (o32 ? 4 : 2), l_bytes = rows * 4;
    const void* ins[] = {Q, K, V};
    for (const void* in : ins)
        if (overlaps(O, o_bytes, in, in_bytes) || overlaps(LSE, l_bytes, in, in_bytes))
            return FA_ERR_INVALID_ARG;
    if (overlaps(O, o_bytes, LSE, l_bytes)) return FA_ERR_INVALID_ARG;
    if (blocks && (overlaps(O, o_bytes, blocks, mask_bytes) || overlaps(LSE, l_bytes, blocks, mask_bytes)))
        return FA_ERR_INVALID_ARG;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    FwdArgs a;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.LSE = LSE;
    a.BH = B * H;
    a.N = N;
    a.d = d;
    a.tau = tau;
    a.causal = causal != 0;
    // (where the window hides nothing the kernels without one run)
    const bool hides = window_hides(N, window, sinks);
    a.window = hides ? window : 0;
    a.sinks = hides ? sinks : 0;
    a.blocks = blocks;
    a.blocks_head_stride = mask_stride;
    a.o32 = o32;
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    return map_cuda(launch_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

__global__ void watchdog_selftest_kernel(unsigned int* err, unsigned long long limit_ns) {
    __shared__ uint64_t never;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_addr(&never), 1);
        mbar_init_fence();
    }
    __syncthreads();
    const Watchdog wd{err, &abort_flag, limit_ns};
    // Nothing ever arrives on `never`: the wait must give up after limit_ns.
    mbar_wait(smem_addr(&never), 0, wd, 0xEE);
    __syncthreads();
}

}  // namespace

namespace {
// Encoded maps, keyed by every argument of the encode: a map only describes an
// address, a shape and a box, so a hit is the same 128 bytes the driver would
// produce again.  Bounded: cleared when full.
struct MapKey {
    uintptr_t base;
    int dtype, esize, cols, rows, planes, box_cols, box_rows;
    bool operator==(const MapKey& o) const {
        return base == o.base && dtype == o.dtype && esize == o.esize && cols == o.cols &&
               rows == o.rows && planes == o.planes && box_cols == o.box_cols && box_rows == o.box_rows;
    }
};
struct MapKeyHash {
    size_t operator()(const MapKey& k) const {
        uint64_t h = k.base * 0x9E3779B97F4A7C15ull;
        const int f[] = {k.dtype, k.esize, k.cols, k.rows, k.planes, k.box_cols, k.box_rows};
        for (int x : f) h = (h ^ static_cast<uint64_t>(x)) * 0x100000001B3ull;
        return static_cast<size_t>(h);
    }
};
constexpr size_t kMapCacheMax = 4096;
std::mutex g_map_mutex;
std::unordered_map<MapKey, CUtensorMap, MapKeyHash>& map_cache() {
    static std::unordered_map<MapKey, CUtensorMap, MapKeyHash> cache;
    return cache;
}
}  // namespace

bool make_tile_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                   int cols, int rows, int planes, int box_cols, int box_rows) {
    const MapKey key{reinterpret_cast<uintptr_t>(base), static_cast<int>(dtype), esize, cols, rows,
                     planes, box_cols, box_rows};
    {
        std::lock_guard<std::mutex> lock(g_map_mutex);
        auto it = map_cache().find(key);
        if (it != map_cache().end()) {
            *map = it->second;
            return true;
        }
    }
    if (!encode_tile_map(map, base, dtype, esize, cols, rows, planes, box_cols, box_rows)) return false;
    std::lock_guard<std::mutex> lock(g_map_mutex);
    if (map_cache().size() >= kMapCacheMax) map_cache().clear();
    map_cache().emplace(key, *map);
    return true;
}

bool encode_tile_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                     int cols, int rows, int planes, int box_cols, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * esize,
                                   static_cast<cuuint64_t>(cols) * rows * esize};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    return fn(map, dtype, 3, const_cast<void*>(base), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_watchdog_selftest(unsigned int* err, unsigned long long limit_ns,
                                     cudaStream_t stream) {
    watchdog_selftest_kernel<<<1, 32, 0, stream>>>(err, limit_ns);
    return cudaGetLastError();
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                 int N, int d, float tau, int causal, void* stream) {
    return fwd_common(Q, K, V, O, LSE, B, H, N, d, tau, causal, stream, false);
}

fa_status fa_fwd_o32(const void* Q, const void* K, const void* V, float* O, float* LSE, int B,
                     int H, int N, int d, float tau, int causal, void* stream) {
    return fwd_common(Q, K, V, O, LSE, B, H, N, d, tau, causal, stream, true);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
    if (B <= 0 || H <= 0 || N <= 0 || (d != 64 && d != 128)) return 0;
    const size_t rows = static_cast<size_t>(B) * H * N;
    return round256(rows * sizeof(float)) + round256(rows * d * sizeof(float));
}

static fa_status bwd_common(const void* Q, const void* K, const void* V, const void* O,
                            const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                            void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                            float tau, int causal, int window, void* stream,
                            const uint8_t* blocks = nullptr, int mask_heads = 0, int sinks = 0) {
    bool empty = false;
    fa_status s = check_shape(B, H, N, d, tau, causal, &empty);
    if (s != FA_OK || empty) return s;
    size_t mask_bytes = 0;
    long long mask_stride = 0;
    if (mask_heads != 0) {
        s = check_blocks(blocks, mask_heads, B, H, N, &mask_bytes, &mask_stride);
        if (s != FA_OK) return s;
    }
    const void* ptrs[] = {Q, K, V, O, dO, LSE, dQ, dK, dV};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(B) * H * N;
    const size_t tb = rows * d * 2;
    const void* ins[] = {Q, K, V, O, dO};
    void* outs[] = {dQ, dK, dV};
    for (void* o : outs) {
        for (const void* in : ins)
            if (overlaps(o, tb, in, tb)) return FA_ERR_INVALID_ARG;
        if (overlaps(o, tb, LSE, rows * 4)) return FA_ERR_INVALID_ARG;
    }
    if (overlaps(dQ, tb, dK, tb) || overlaps(dQ, tb, dV, tb) || overlaps(dK, tb, dV, tb))
        return FA_ERR_INVALID_ARG;
    if (blocks)
        for (void* o : outs)
            if (overlaps(o, tb, blocks, mask_bytes)) return FA_ERR_INVALID_ARG;
    const size_t need = fa_bwd_workspace_size(B, H, N, d);
    if (workspace != nullptr) {
        if (workspace_bytes < need) return FA_ERR_WORKSPACE;
        const void* all[] = {Q, K, V, O, dO, dQ, dK, dV};
        for (const void* p : all)
            if (overlaps(workspace, need, p, tb)) return FA_ERR_INVALID_ARG;
        if (overlaps(workspace, need, LSE, rows * 4)) return FA_ERR_INVALID_ARG;
        if (blocks && overlaps(workspace, need, blocks, mask_bytes)) return FA_ERR_INVALID_ARG;
    }
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = workspace;
    if (ws == nullptr && cudaMallocAsync(&ws, need, st) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    BwdArgs a;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.dO = dO;
    a.LSE = LSE;
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    a.D = static_cast<float*>(ws);
    a.dQacc = reinterpret_cast<float*>(static_cast<char*>(ws) + round256(rows * sizeof(float)));
    a.BH = B * H;
    a.N = N;
    a.d = d;
    a.tau = tau;
    a.causal = causal != 0;
    const WindowCut cut = cut_window(N, window, sinks);
    a.window = cut.window;
    a.sinks = cut.sinks;
    a.blocks = blocks;
    a.blocks_head_stride = mask_stride;
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    const cudaError_t e = launch_bwd(a, st);
    if (workspace == nullptr) cudaFreeAsync(ws, st);
    return map_cuda(e);
}

fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                 size_t workspace_bytes, int B, int H, int N, int d, float tau, int causal,
                 void* stream) {
    return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, workspace_bytes, B, H, N, d, tau,
                      causal, 0, stream);
}

fa_status fa_fwd_window(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                        int H, int N, int d, float tau, int window, void* stream) {
    if (window < 1) return FA_ERR_INVALID_ARG;
    return fwd_common(Q, K, V, O, LSE, B, H, N, d, tau, 1, stream, false, window);
}

fa_status fa_bwd_window(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                        const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                        size_t workspace_bytes, int B, int H, int N, int d, float tau, int window,
                        void* stream) {
    if (window < 1) return FA_ERR_INVALID_ARG;
    return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, workspace_bytes, B, H, N, d, tau,
                      1, window, stream);
}

fa_status fa_fwd_sinks(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                       int N, int d, float tau, int window, int sinks, void* stream) {
    if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
    return fwd_common(Q, K, V, O, LSE, B, H, N, d, tau, 1, stream, false, window, nullptr, 0, sinks);
}

fa_status fa_bwd_sinks(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                       const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                       size_t workspace_bytes, int B, int H, int N, int d, float tau, int window,
                       int sinks, void* stream) {
    if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
    return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, workspace_bytes, B, H, N, d, tau,
                      1, window, stream, nullptr, 0, sinks);
}

fa_status fa_fwd_blocks(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                        int H, int N, int d, float tau, int causal, const unsigned char* block_mask,
                        int mask_heads, void* stream) {
    if (mask_heads == 0) return FA_ERR_INVALID_ARG;
    return fwd_common(Q, K, V, O, LSE, B, H, N, d, tau, causal, stream, false, 0, block_mask,
                      mask_heads);
}

fa_status fa_bwd_blocks(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                        const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                        size_t workspace_bytes, int B, int H, int N, int d, float tau, int causal,
                        const unsigned char* block_mask, int mask_heads, void* stream) {
    if (mask_heads == 0) return FA_ERR_INVALID_ARG;
    return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, workspace_bytes, B, H, N, d, tau,
                      causal, 0, stream, block_mask, mask_heads);
}

size_t fa_decode_workspace_size(int B, int H, int Nq, int Nk, int d) {
    if (B <= 0 || H <= 0 || Nq <= 0 || Nq > 8 || Nk <= 0 || (d != 64 && d != 128)) return 0;
    const long long bh = static_cast<long long>(B) * H;
    if (bh > INT_MAX) return 0;
    int splits = 1, chunk = 0;
    decode_plan(static_cast<int>(bh), Nk, &splits, &chunk);
    if (splits <= 1) return 0;
    const size_t rows = static_cast<size_t>(bh) * Nq;
    return round256(static_cast<size_t>(splits) * rows * (d + 2) * sizeof(float));
}

fa_status fa_fwd_decode(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                        int H, int Nq, int Nk, int d, float tau, int causal, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (B < 0 || H < 0 || Nq < 0 || Nk < 0 || d < 0) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(tau) && tau > 0.f)) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || Nq == 0) return FA_OK;
    if (Nk == 0 || (causal && Nq > Nk)) return FA_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || Nq > 8) return FA_ERR_UNSUPPORTED;
    const long long bh = static_cast<long long>(B) * H;
    if (bh > INT_MAX) return FA_ERR_UNSUPPORTED;
    int splits = 1, chunk = 0;
    decode_plan(static_cast<int>(bh), Nk, &splits, &chunk);
    if (splits > 65535) return FA_ERR_UNSUPPORTED;
    const void* ptrs[] = {Q, K, V, O, LSE};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    const size_t qb = static_cast<size_t>(bh) * Nq * d * 2, kb = static_cast<size_t>(bh) * Nk * d * 2;
    const size_t lb = static_cast<size_t>(bh) * Nq * 4;
    const void* ins[] = {Q, K, V};
    const size_t in_bytes[] = {qb, kb, kb};
    for (int i = 0; i < 3; ++i)
        if (overlaps(O, qb, ins[i], in_bytes[i]) || overlaps(LSE, lb, ins[i], in_bytes[i]))
            return FA_ERR_INVALID_ARG;
    if (overlaps(O, qb, LSE, lb)) return FA_ERR_INVALID_ARG;
    const size_t need = fa_decode_workspace_size(B, H, Nq, Nk, d);
    if (workspace != nullptr && need > 0) {
        if (workspace_bytes < need) return FA_ERR_WORKSPACE;
        const void* all[] = {Q, K, V, O, LSE};
        const size_t all_bytes[] = {qb, kb, kb, qb, lb};
        for (int i = 0; i < 5; ++i)
            if (overlaps(workspace, need, all[i], all_bytes[i])) return FA_ERR_INVALID_ARG;
    }
    fa_status s = FA_OK;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = need > 0 ? workspace : nullptr;
    const bool own = need > 0 && workspace == nullptr;
    if (own && cudaMallocAsync(&ws, need, st) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    DecArgs a;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.LSE = LSE;
    a.workspace = static_cast<float*>(ws);
    a.BH = static_cast<int>(bh);
    a.Nq = Nq;
    a.Nk = Nk;
    a.d = d;
    a.tau = tau;
    a.causal = causal != 0;
    a.splits = splits;
    a.chunk = chunk;
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    const cudaError_t e = launch_decode(a, st);
    if (own) cudaFreeAsync(ws, st);
    return map_cuda(e);
}

fa_status fa_fwd_fp8(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                     int N, int d, float tau, int causal, float q_scale, float k_scale,
                     float v_scale, void* stream) {
    bool empty = false;
    fa_status s = check_shape(B, H, N, d, tau, causal, &empty);
    if (s != FA_OK || empty) return s;
    if (d != 128) return FA_ERR_UNSUPPORTED;
    const float scales[] = {q_scale, k_scale, v_scale};
    for (float sc : scales)
        if (!(std::isfinite(sc) && sc > 0.f)) return FA_ERR_INVALID_ARG;
    const void* ptrs[] = {Q, K, V, O, LSE};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(B) * H * N;
    const size_t in_bytes = rows * d, o_bytes = rows * d * 2, l_bytes = rows * 4;
    const void* ins[] = {Q, K, V};
    for (const void* in : ins)
        if (overlaps(O, o_bytes, in, in_bytes) || overlaps(LSE, l_bytes, in, in_bytes))
            return FA_ERR_INVALID_ARG;
    if (overlaps(O, o_bytes, LSE, l_bytes)) return FA_ERR_INVALID_ARG;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    Fp8Args a;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.LSE = LSE;
    a.BH = B * H;
    a.N = N;
    a.tau = tau;
    a.q_scale = q_scale;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.causal = causal != 0;
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    return map_cuda(launch_fwd_fp8(a, static_cast<cudaStream_t>(stream)));
}

// --- paged key/value cache ---
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Elements from the first to one past the last of a strided [n0][n1][n2][d] tensor, or
// -1 for strides that the kernels do not take: negative ones, and any that is no multiple
// of 8 elements (16 bytes) where its dimension has more than one entry.
static long long strided_span(const long long n[3], const long long st[3], int d) {
    long long span = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < 0 || (st[i] & 7) != 0 || st[i] > (1ll << 60) / n[i]) return -1;
        span += (n[i] - 1) * st[i];
    }
    return span;
}
// Whether no two entries of such a tensor share memory (sorted by stride, each dimension
// steps over all that the smaller ones span).
static bool strided_distinct(const long long n[3], const long long st[3], int d) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[order[j]] < st[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    long long inner = d;
    for (int i : order) {
        if (n[i] <= 1) continue;
        if (st[i] < inner) return false;
        inner = st[i] * (n[i] - 1) + inner;
    }
    return true;
}

// log2 of a page size that the kernels take.
static bool page_shift(int page_size, int* shift) {
    *shift = 0;
    while ((1 << *shift) < page_size && *shift < 30) ++*shift;
    return page_size == 1 << *shift && page_size >= kPagedMinPage && page_size <= kPagedMaxPage;
}

// Checks a cache's description and fills the internal form.  fp8 says what the entry
// point takes.  Sets *bytes (of K, and of V).
static fa_status check_cache(const fa_paged_cache* c, bool fp8, PagedCache* out, size_t* bytes) {
    if (c == nullptr) return FA_ERR_INVALID_ARG;
    if (c->B < 0 || c->H_kv < 0 || c->d < 0 || c->num_pages < 0 || c->page_size < 0 || c->max_pages < 0)
        return FA_ERR_INVALID_ARG;
    out->B = c->B;
    out->H_kv = c->H_kv;
    out->d = c->d;
    out->num_pages = c->num_pages;
    out->max_pages = c->max_pages;
    if (c->B == 0 || c->H_kv == 0) return FA_OK;  // empty: the caller returns
    if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
    if (!page_shift(c->page_size, &out->shift)) return FA_ERR_UNSUPPORTED;
    if (c->num_pages == 0 || c->max_pages == 0) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(c->max_pages) * c->page_size > kPagedMaxKeys) return FA_ERR_UNSUPPORTED;
    if (c->K == nullptr || c->V == nullptr || c->page_table == nullptr || c->lens == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned16(c->K) || !aligned16(c->V) || !aligned4(c->page_table) || !aligned4(c->lens)) return FA_ERR_INVALID_ARG;
    if ((c->k_scale != nullptr) != fp8 || (c->v_scale != nullptr) != fp8) return FA_ERR_INVALID_ARG;
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return FA_ERR_INVALID_ARG;
    const double elems = static_cast<double>(c->num_pages) * c->H_kv * c->page_size * c->d;
    if (elems > 1e15) return FA_ERR_UNSUPPORTED;
    *bytes = static_cast<size_t>(c->num_pages) * c->H_kv * c->page_size * c->d * (fp8 ? 1 : 2);
    if (overlaps(c->K, *bytes, c->V, *bytes)) return FA_ERR_INVALID_ARG;
    out->K = c->K;
    out->V = c->V;
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->page_table = c->page_table;
    out->lens = c->lens;
    return FA_OK;
}

static fa_status append_common(const fa_paged_cache* c, bool fp8, const void* k, long long k_st,
                               long long k_sh, const void* v, long long v_st, long long v_sh, int T,
                               const int* cu_new, const void* q, long long q_st, long long q_sh,
                               void* q_out, long long qo_st, long long qo_sh, int H,
                               const double* inv_freq, int rot, int interleaved, void* stream) {
    AppendArgs a;
    size_t cache_bytes = 0;
    fa_status s = check_cache(c, fp8, &a.cache, &cache_bytes);
    if (s != FA_OK) return s;
    if (T < 0 || H < 0 || rot < 0 || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
    if (c->H_kv == 0 && H > 0) return FA_ERR_INVALID_ARG;
    if (c->B == 0 || c->H_kv == 0 || T == 0) return FA_OK;
    if (rot > c->d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
    if ((rot > 0) != (inv_freq != nullptr) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0) return FA_ERR_INVALID_ARG;
    if (cu_new == nullptr ? T % c->B != 0 : !aligned4(cu_new)) return FA_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
    const bool has_q = q != nullptr;
    if (has_q != (q_out != nullptr) || has_q != (H > 0)) return FA_ERR_INVALID_ARG;
    if (has_q && (rot == 0 || !aligned16(q) || !aligned16(q_out))) return FA_ERR_INVALID_ARG;
    // (token, head) as a [T][heads][1][d] tensor
    const long long nk[3] = {T, c->H_kv, 1}, nq[3] = {T, H, 1};
    const auto span = [&](const long long* n, long long st, long long sh) {
        const long long s3[3] = {st, sh, 0};
        return strided_span(n, s3, c->d);
    };
    const long long ks = span(nk, k_st, k_sh), vs = span(nk, v_st, v_sh);
    if (ks < 0 || vs < 0) return FA_ERR_INVALID_ARG;
    size_t q_bytes = 0;  // of q_out
    long long q_span = 0;
    const void* caches[] = {c->K, c->V};
    for (const void* x : caches)
        if (overlaps(x, cache_bytes, k, ks * 2) || overlaps(x, cache_bytes, v, vs * 2)) return FA_ERR_INVALID_ARG;
    if (has_q) {
        const long long qs = span(nq, q_st, q_sh), os = span(nq, qo_st, qo_sh);
        if (qs < 0 || os < 0) return FA_ERR_INVALID_ARG;
        q_span = qs;
        const long long o3[3] = {qo_st, qo_sh, 0};
        if (!strided_distinct(nq, o3, c->d)) return FA_ERR_INVALID_ARG;
        // in place (the same rows) or apart from everything else
        const bool in_place = q == q_out && (T == 1 || q_st == qo_st) && (H == 1 || q_sh == qo_sh);
        for (const void* x : caches)
            if (overlaps(x, cache_bytes, q, qs * 2) || overlaps(x, cache_bytes, q_out, os * 2)) return FA_ERR_INVALID_ARG;
        if (!in_place && (overlaps(q_out, os * 2, q, qs * 2) || overlaps(q_out, os * 2, k, ks * 2) ||
                          overlaps(q_out, os * 2, v, vs * 2)))
            return FA_ERR_INVALID_ARG;
        if (in_place) {
            // (rows: q, k and v may be slices of one tensor, but no key is a query's place)
            const auto at = [](const void* x) { return static_cast<long long>(reinterpret_cast<uintptr_t>(x) / 2); };
            const RowSet rows{at(q_out), qo_st, qo_sh, T, H};
            if (rows_meet(rows, {at(k), k_st, k_sh, T, c->H_kv}, c->d) || rows_meet(rows, {at(v), v_st, v_sh, T, c->H_kv}, c->d))
                return FA_ERR_INVALID_ARG;
        }
        q_bytes = static_cast<size_t>(os) * 2;
        a.q_st = q_st;
        a.q_sh = q_sh;
        a.o_st = qo_st;
        a.o_sh = qo_sh;
    } else {
        a.q_st = a.q_sh = a.o_st = a.o_sh = 0;
    }
    // what the kernels read as indices and angles lies apart from all that they write, the new
    // rows apart from the scales
    const size_t sb = fp8 ? static_cast<size_t>(c->num_pages) * c->H_kv * 4 : 0;
    const void* scales[] = {c->k_scale, c->v_scale};
    for (const void* x : scales)
        if (fp8 && (overlaps(x, sb, k, ks * 2) || overlaps(x, sb, v, vs * 2) || (has_q && overlaps(x, sb, q, q_span * 2))))
            return FA_ERR_INVALID_ARG;
    const void* ins[] = {c->page_table, c->lens, cu_new, inv_freq};
    const size_t in_bytes[] = {static_cast<size_t>(c->B) * c->max_pages * 4, static_cast<size_t>(c->B) * 4,
                               cu_new ? (static_cast<size_t>(c->B) + 1) * 4 : 0, static_cast<size_t>(rot) * 4};
    const void* outs[] = {c->K, c->V, q_out, c->k_scale, c->v_scale};
    const size_t out_bytes[] = {cache_bytes, cache_bytes, q_bytes, sb, sb};
    for (int o = 0; o < 5; ++o) {
        if (out_bytes[o] == 0) continue;
        for (int i = 0; i < 4; ++i)
            if (in_bytes[i] > 0 && overlaps(outs[o], out_bytes[o], ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
        for (int o2 = 3; o2 < 5; ++o2)
            if (sb > 0 && o2 != o && overlaps(outs[o], out_bytes[o], outs[o2], sb)) return FA_ERR_INVALID_ARG;
    }
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.cu_new = cu_new;
    a.inv_freq = inv_freq;
    a.k_st = k_st;
    a.k_sh = k_sh;
    a.v_st = v_st;
    a.v_sh = v_sh;
    a.T = T;
    a.H = H;
    a.rot = rot;
    a.interleaved = interleaved;
    a.err = di->err_word;
    return map_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_append(const fa_paged_cache* cache, const void* k, long long k_st, long long k_sh,
                       const void* v, long long v_st, long long v_sh, int T, const int* cu_new,
                       const void* q, long long q_st, long long q_sh, void* q_out, long long qo_st,
                       long long qo_sh, int H, const double* inv_freq, int rot, int interleaved,
                       void* stream) {
    return append_common(cache, false, k, k_st, k_sh, v, v_st, v_sh, T, cu_new, q, q_st, q_sh, q_out,
                         qo_st, qo_sh, H, inv_freq, rot, interleaved, stream);
}

fa_status fa_kv_append_fp8(const fa_paged_cache* cache, const void* k, long long k_st, long long k_sh,
                       const void* v, long long v_st, long long v_sh, int T, const int* cu_new,
                       const void* q, long long q_st, long long q_sh, void* q_out, long long qo_st,
                       long long qo_sh, int H, const double* inv_freq, int rot, int interleaved,
                       void* stream) {
    return append_common(cache, true, k, k_st, k_sh, v, v_st, v_sh, T, cu_new, q, q_st, q_sh, q_out,
                         qo_st, qo_sh, H, inv_freq, rot, interleaved, stream);
}

// A window or a number of sinks beyond any length, cut to what the kernels' integers hold
// (the same keys are visible).
static int cut_keys(int x) { return x < (1 << 30) ? x : (1 << 30); }

size_t fa_paged_workspace_size(const fa_paged_cache* cache, int H, int Nq, int window, int sinks) {
    if (cache == nullptr || H <= 0 || Nq <= 0 || Nq > 8 || window < 0 || sinks < 0) return 0;
    if (cache->B <= 0 || cache->H_kv <= 0 || H % cache->H_kv != 0 || H / cache->H_kv > (1 << 20)) return 0;
    if ((cache->d != 64 && cache->d != 128) || cache->max_pages <= 0) return 0;
    PagedCache c;
    if (!page_shift(cache->page_size, &c.shift)) return 0;
    c.B = cache->B;
    c.H_kv = cache->H_kv;
    c.d = cache->d;
    c.max_pages = cache->max_pages;
    return paged_workspace(c, H, Nq, cut_keys(window), cut_keys(sinks), cache->k_scale != nullptr);
}

// Bytes of what a fa_score names.
struct ScoreBytes {
    size_t slopes, table, buckets, docs, prefix;
};
// Checks a fa_score for B sequences of N tokens (of a cache: without documents or prefix)
// and H query heads, and fills the internal form (its window aside).
static fa_status check_score(const fa_score* f, int B, int H, int N, bool cache, ScoreMod* m, ScoreBytes* bytes) {
    if (!(f->softcap == 0.f || (f->softcap >= 0x1p-20f && f->softcap <= 0x1p60f))) return FA_ERR_INVALID_ARG;
    if (f->bias_f32 != 0 && f->bias_f32 != 1) return FA_ERR_INVALID_ARG;
    if (f->window < 0) return FA_ERR_INVALID_ARG;
    if ((f->bias != nullptr) != (f->buckets != nullptr) || (f->bias != nullptr && f->slopes != nullptr)) return FA_ERR_INVALID_ARG;
    if (f->bias != nullptr) {
        if (f->num_buckets < 1 || f->max_distance < 1) return FA_ERR_INVALID_ARG;
        if (f->num_buckets > kScoreMaxBuckets || f->max_distance > kScoreMaxFar) return FA_ERR_UNSUPPORTED;
        if ((reinterpret_cast<uintptr_t>(f->bias) & (f->bias_f32 ? 3u : 1u)) != 0) return FA_ERR_INVALID_ARG;
        m->num_buckets = f->num_buckets;
        m->far = f->max_distance;
        m->table_f32 = f->bias_f32 != 0;
    }
    if (!aligned4(f->slopes) || !aligned4(f->buckets) || !aligned4(f->docs) || !aligned4(f->prefix)) return FA_ERR_INVALID_ARG;
    if (cache && (f->docs != nullptr || f->prefix != nullptr)) return FA_ERR_INVALID_ARG;
    m->softcap = f->softcap;
    m->slopes = f->slopes;
    m->table = f->bias;
    m->buckets = f->buckets;
    m->docs = f->docs;
    m->prefix = f->prefix;
    bytes->slopes = f->slopes ? static_cast<size_t>(H) * 4 : 0;
    bytes->table = f->bias ? static_cast<size_t>(f->num_buckets) * H * (f->bias_f32 ? 4 : 2) : 0;
    bytes->buckets = f->bias ? (2 * static_cast<size_t>(f->max_distance) + 1) * 4 : 0;
    bytes->docs = f->docs ? static_cast<size_t>(B) * N * 4 : 0;
    bytes->prefix = f->prefix ? static_cast<size_t>(B) * 4 : 0;
    return FA_OK;
}

static fa_status paged_common(const fa_paged_cache* c, bool fp8, const void* Q, long long q_sb,
                              long long q_sh, long long q_sn, void* O, long long o_sb, long long o_sh,
                              long long o_sn, float* LSE, int H, int Nq, float tau, int window, int sinks,
                              void* workspace, size_t workspace_bytes, void* stream,
                              const fa_score* score = nullptr) {
    PagedArgs a;
    size_t cache_bytes = 0;
    fa_status s = check_cache(c, fp8, &a.cache, &cache_bytes);
    if (s != FA_OK) return s;
    if (H < 0 || Nq < 0 || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(tau) && tau > 0.f)) return FA_ERR_INVALID_ARG;
    if (c->B == 0 || H == 0 || Nq == 0) return FA_OK;
    if (c->H_kv == 0 || H % c->H_kv != 0) return FA_ERR_INVALID_ARG;
    if (Nq > 8 || H / c->H_kv > (1 << 20)) return FA_ERR_UNSUPPORTED;
    if (paged_max_tiles(c->B, H, c->H_kv, Nq, c->max_pages, a.cache.shift) > INT_MAX) return FA_ERR_UNSUPPORTED;
    if (Q == nullptr || O == nullptr || LSE == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(O) || !aligned16(LSE)) return FA_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    const long long n[3] = {c->B, H, Nq}, q_strides[3] = {q_sb, q_sh, q_sn}, o_strides[3] = {o_sb, o_sh, o_sn};
    const long long qs = strided_span(n, q_strides, c->d), os = strided_span(n, o_strides, c->d);
    if (qs < 0 || os < 0 || !strided_distinct(n, o_strides, c->d)) return FA_ERR_INVALID_ARG;
    const size_t need = fa_paged_workspace_size(c, H, Nq, window, sinks);
    if (workspace != nullptr && workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t lb = static_cast<size_t>(c->B) * H * Nq * 4, tb = static_cast<size_t>(c->B) * c->max_pages * 4;
    const size_t sb = fp8 ? static_cast<size_t>(c->num_pages) * c->H_kv * 4 : 0;
    ScoreBytes mod{};
    if (score != nullptr) {
        s = check_score(score, 0, H, 0, true, &a.mod, &mod);
        if (s != FA_OK) return s;
    }
    const void* ins[] = {Q, c->K, c->V, c->page_table, c->lens, a.mod.slopes, a.mod.table, a.mod.buckets, c->k_scale,
                         c->v_scale};
    const size_t in_bytes[] = {static_cast<size_t>(qs) * 2, cache_bytes, cache_bytes, tb, static_cast<size_t>(c->B) * 4,
                               mod.slopes, mod.table, mod.buckets, sb, sb};
    const void* outs[] = {O, LSE, workspace};
    const size_t out_bytes[] = {static_cast<size_t>(os) * 2, lb, need};
    for (int o = 0; o < (workspace && need > 0 ? 3 : 2); ++o) {
        for (int i = 0; i < 10; ++i)
            if (ins[i] != nullptr && overlaps(outs[o], out_bytes[o], ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
        for (int o2 = 0; o2 < o; ++o2)
            if (overlaps(outs[o], out_bytes[o], outs[o2], out_bytes[o2])) return FA_ERR_INVALID_ARG;
    }
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = need > 0 ? workspace : nullptr;
    const bool own = need > 0 && workspace == nullptr;
    if (own && cudaMallocAsync(&ws, need, st) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    a.Q = Q;
    a.O = O;
    a.LSE = LSE;
    a.workspace = ws;
    a.q_sb = q_sb;
    a.q_sh = q_sh;
    a.q_sn = q_sn;
    a.o_sb = o_sb;
    a.o_sh = o_sh;
    a.o_sn = o_sn;
    a.H = H;
    a.Nq = Nq;
    a.window = cut_keys(window);
    a.sinks = cut_keys(sinks);
    a.tau = tau;
    a.err = di->err_word;
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    const cudaError_t e = score != nullptr ? launch_fwd_paged_score(a, st) : launch_fwd_paged(a, st);
    if (own) cudaFreeAsync(ws, st);
    return map_cuda(e);
}

fa_status fa_fwd_paged(const fa_paged_cache* cache, const void* Q, long long q_sb, long long q_sh,
                       long long q_sn, void* O, long long o_sb, long long o_sh, long long o_sn,
                       float* LSE, int H, int Nq, float tau, int window, int sinks, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return paged_common(cache, false, Q, q_sb, q_sh, q_sn, O, o_sb, o_sh, o_sn, LSE, H, Nq, tau, window,
                        sinks, workspace, workspace_bytes, stream);
}

fa_status fa_fwd_paged_fp8(const fa_paged_cache* cache, const void* Q, long long q_sb, long long q_sh,
                       long long q_sn, void* O, long long o_sb, long long o_sh, long long o_sn,
                       float* LSE, int H, int Nq, float tau, int window, int sinks, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return paged_common(cache, true, Q, q_sb, q_sh, q_sn, O, o_sb, o_sh, o_sn, LSE, H, Nq, tau, window,
                        sinks, workspace, workspace_bytes, stream);
}

fa_status fa_fwd_paged_score(const fa_paged_cache* cache, const void* Q, long long q_sb, long long q_sh,
                             long long q_sn, void* O, long long o_sb, long long o_sh, long long o_sn,
                             float* LSE, int H, int Nq, float tau, int window, int sinks,
                             const fa_score* score, void* workspace, size_t workspace_bytes, void* stream) {
    if (score == nullptr || score->window != 0) return FA_ERR_INVALID_ARG;
    return paged_common(cache, false, Q, q_sb, q_sh, q_sn, O, o_sb, o_sh, o_sn, LSE, H, Nq, tau, window,
                        sinks, workspace, workspace_bytes, stream, score);
}

fa_status fa_fwd_paged_score_fp8(const fa_paged_cache* cache, const void* Q, long long q_sb,
                                 long long q_sh, long long q_sn, void* O, long long o_sb, long long o_sh,
                                 long long o_sn, float* LSE, int H, int Nq, float tau, int window,
                                 int sinks, const fa_score* score, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (score == nullptr || score->window != 0) return FA_ERR_INVALID_ARG;
    return paged_common(cache, true, Q, q_sb, q_sh, q_sn, O, o_sb, o_sh, o_sn, LSE, H, Nq, tau, window,
                        sinks, workspace, workspace_bytes, stream, score);
}

// A list of device buffers, for the checks that what a call writes lies apart from all else.
struct Buffer {
    const void* p;
    size_t n;
};
// Whether every one of the first n_out buffers lies apart from all others (null: none).
static bool apart(const Buffer* bs, int n_out, int n) {
    for (int o = 0; o < n_out; ++o)
        for (int i = o + 1; i < n; ++i)
            if (bs[o].p != nullptr && bs[i].p != nullptr && overlaps(bs[o].p, bs[o].n, bs[i].p, bs[i].n)) return false;
    return true;
}

// Checks that the forward and the backward share; *empty: no rows.  Fills the arguments'
// sizes and scores.
static fa_status score_shape(int B, int H, int H_kv, int N, int d, float tau, int causal, const fa_score* score,
                             ScoreArgs* a, ScoreBytes* mod, bool* empty) {
    if (score == nullptr || H_kv < 0) return FA_ERR_INVALID_ARG;
    fa_status s = check_shape(B, H, N, d, tau, causal, empty);
    if (s != FA_OK) return s;
    if (H_kv == 0 ? H > 0 : H % H_kv != 0) return FA_ERR_INVALID_ARG;
    s = check_score(score, B, H, N, false, &a->mod, mod);
    if (s != FA_OK) return s;
    if ((score->prefix != nullptr || score->window != 0) && !causal) return FA_ERR_INVALID_ARG;
    if (*empty) return FA_OK;
    // (the backward's grid, one block per key tile; window: cut to the N keys that there are)
    if (static_cast<long long>(B) * H * ((static_cast<long long>(N) + 127) / 128) > INT_MAX) return FA_ERR_UNSUPPORTED;
    a->mod.window = score->window < N ? score->window : 0;
    a->B = B;
    a->H = H;
    a->H_kv = H_kv;
    a->N = N;
    a->d = d;
    a->tau = tau;
    a->causal = causal != 0;
    return FA_OK;
}

size_t fa_fwd_score_workspace_size(int B, int N, const fa_score* score) {
    if (score == nullptr || B <= 0 || N <= 0) return 0;
    return score_fwd_workspace(B, N, score->docs != nullptr);
}

static size_t score_bwd_bytes(int B, int H, int N, int d, int causal, const fa_score* score, bool grad) {
    ScoreArgs a;
    ScoreBytes mod;
    bool empty = false;
    if (score_shape(B, H, H, N, d, 1.f, causal, score, &a, &mod, &empty) != FA_OK || empty) return 0;
    return score_bwd_workspace(a, grad);
}

size_t fa_bwd_score_workspace_size(int B, int H, int N, int d, int causal, const fa_score* score) {
    return score_bwd_bytes(B, H, N, d, causal, score, true);
}

size_t fa_bwd_score_frozen_workspace_size(int B, int H, int N, int d, int causal, const fa_score* score) {
    return score_bwd_bytes(B, H, N, d, causal, score, false);
}

fa_status fa_fwd_score(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                       int H_kv, int N, int d, float tau, int causal, const fa_score* score,
                       void* workspace, size_t workspace_bytes, void* stream) {
    ScoreArgs a;
    ScoreBytes mod;
    bool empty = false;
    fa_status s = score_shape(B, H, H_kv, N, d, tau, causal, score, &a, &mod, &empty);
    if (s != FA_OK || empty) return s;
    const void* ptrs[] = {Q, K, V, O, LSE};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    const size_t need = fa_fwd_score_workspace_size(B, N, score);
    if (workspace != nullptr && workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(B) * H * N, tb = rows * d * 2, kb = tb / H * H_kv;
    const Buffer bs[] = {{O, tb}, {LSE, rows * 4}, {need > 0 ? workspace : nullptr, need}, {Q, tb}, {K, kb}, {V, kb},
                         {a.mod.slopes, mod.slopes}, {a.mod.table, mod.table}, {a.mod.buckets, mod.buckets},
                         {a.mod.docs, mod.docs}, {a.mod.prefix, mod.prefix}};
    if (!apart(bs, 3, 11)) return FA_ERR_INVALID_ARG;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = need > 0 ? workspace : nullptr;
    const bool own = need > 0 && workspace == nullptr;
    if (own && cudaMallocAsync(&ws, need, st) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.LSE = LSE;
    a.workspace = static_cast<uint8_t*>(ws);
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    const cudaError_t e = launch_score_fwd(a, st);
    if (own) cudaFreeAsync(ws, st);
    return map_cuda(e);
}

fa_status fa_bwd_score(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                       const float* LSE, void* dQ, void* dK, void* dV, void* dBias, int B, int H, int H_kv,
                       int N, int d, float tau, int causal, const fa_score* score, void* workspace,
                       size_t workspace_bytes, void* stream) {
    ScoreArgs a;
    ScoreBytes mod;
    bool empty = false;
    fa_status s = score_shape(B, H, H_kv, N, d, tau, causal, score, &a, &mod, &empty);
    if (s != FA_OK) return s;
    if (dBias != nullptr && a.mod.table == nullptr) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dBias) & (a.mod.table_f32 ? 3u : 1u)) != 0) return FA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) {  // (no pair: gradients of zeros, of a bias, or of keys that no query head reads)
        bool none = false;
        s = check_shape(B, H_kv, N, d, tau, causal, &none);
        if (s != FA_OK) return s;
        const size_t kb = none ? 0 : static_cast<size_t>(B) * H_kv * N * d * 2, tb = dBias ? mod.table : 0;
        if (kb > 0 && (dK == nullptr || dV == nullptr || !aligned16(dK) || !aligned16(dV))) return FA_ERR_INVALID_ARG;
        const auto of = [](const void* p, size_t n) { return Buffer{n > 0 ? p : nullptr, n}; };
        const Buffer bs[] = {of(dK, kb), of(dV, kb), of(dBias, tb), of(K, kb), of(V, kb), of(a.mod.table, mod.table),
                             of(a.mod.buckets, mod.buckets), of(a.mod.docs, mod.docs), of(a.mod.prefix, mod.prefix)};
        if (!apart(bs, 3, 9)) return FA_ERR_INVALID_ARG;
        if (kb == 0 && tb == 0) return FA_OK;
        if (!current_device(&s)) return s;
        for (int i = 0; i < 3; ++i)
            if (bs[i].p != nullptr && cudaMemsetAsync(const_cast<void*>(bs[i].p), 0, bs[i].n, st) != cudaSuccess) return FA_ERR_CUDA;
        return FA_OK;
    }
    const void* ptrs[] = {Q, K, V, O, dO, LSE, dQ, dK, dV};
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return FA_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    const size_t need = score_bwd_workspace(a, dBias != nullptr);
    if (workspace != nullptr && workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(B) * H * N, tb = rows * d * 2, kb = tb / H * H_kv;
    const Buffer bs[] = {{dQ, tb}, {dK, kb}, {dV, kb}, {dBias, mod.table}, {workspace, need}, {Q, tb}, {K, kb}, {V, kb},
                         {O, tb}, {dO, tb}, {LSE, rows * 4}, {a.mod.slopes, mod.slopes}, {a.mod.table, mod.table},
                         {a.mod.buckets, mod.buckets}, {a.mod.docs, mod.docs}, {a.mod.prefix, mod.prefix}};
    if (!apart(bs, 5, 16)) return FA_ERR_INVALID_ARG;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    void* ws = workspace;
    if (workspace == nullptr && cudaMallocAsync(&ws, need, st) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = const_cast<void*>(O);
    a.dO = dO;
    a.LSE = const_cast<float*>(LSE);
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    a.dTable = dBias;
    a.workspace = static_cast<uint8_t*>(ws);
    a.err = di->err_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.ev_start = t_ev_start;
    a.ev_stop = t_ev_stop;
    const cudaError_t e = launch_score_bwd(a, st);
    if (workspace == nullptr) cudaFreeAsync(ws, st);
    return map_cuda(e);
}

const char* fa_status_string(fa_status s) {
    switch (s) {
        case FA_OK: return "FA_OK";
        case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG: invalid argument";
        case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: unsupported head dim, size or device";
        case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE: workspace too small";
        case FA_ERR_CUDA: return "FA_ERR_CUDA: CUDA runtime or launch error";
        case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a kernel pipeline wait timed out";
        case FA_ERR_PAGE: return "FA_ERR_PAGE: a cache length, token count or page number out of bounds";
    }
    return "unknown fa_status";
}

fa_status fa_last_device_error(void* stream) {
    fa_status s;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    unsigned int words[2] = {0, 0};
    if (cudaMemcpy(words, di->err_word, sizeof(words), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    for (int i = 0; i < 2; ++i) {
        if (words[i] == 0) continue;
        const unsigned int zero = 0;
        if (cudaMemcpy(di->err_word + i, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_CUDA;
        }
        return i == 0 ? FA_ERR_TIMEOUT : FA_ERR_PAGE;
    }
    return FA_OK;
}

fa_status fa_set_wait_limit_ns(unsigned long long ns) {
    g_wait_limit_ns.store(ns == 0 ? kDefaultWaitLimitNs : ns);
    return FA_OK;
}

fa_status fa_set_timing_events(void* start, void* stop) {
    if ((start == nullptr) != (stop == nullptr)) return FA_ERR_INVALID_ARG;
    t_ev_start = static_cast<cudaEvent_t>(start);
    t_ev_stop = static_cast<cudaEvent_t>(stop);
    return FA_OK;
}

fa_status fa_watchdog_selftest(unsigned long long limit_ns, void* stream) {
    if (limit_ns == 0 || limit_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
    fa_status s;
    DeviceInfo* di = current_device(&s);
    if (!di) return s;
    return map_cuda(launch_watchdog_selftest(di->err_word, limit_ns,
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free backward (fa_bwd_noalloc).  The scratch is a fixed array in
// the device image.  In host code `g_fa_noalloc_scratch` only names a host-side
// stand-in, so its device address is looked up per device with
// cudaGetSymbolAddress before it is handed to the kernels.
static __device__ __align__(256) unsigned char g_fa_noalloc_scratch[FA_NOALLOC_SCRATCH_BYTES];

namespace {
// The scratch array's device address, per device; null until a lookup succeeds.
// A failed lookup (for instance a first call made while the stream is being
// captured) is not remembered: the next call tries again.
std::atomic<void*> g_noalloc_ptr[fa::kMaxDevices];

// Looks the array's address up on the current device (the caller's).
void* noalloc_scratch_for_current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= fa::kMaxDevices) {
        cudaGetLastError();
        return nullptr;
    }
    void* p = g_noalloc_ptr[dev].load(std::memory_order_acquire);
    if (p != nullptr) return p;
    if (cudaGetSymbolAddress(&p, g_fa_noalloc_scratch) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    g_noalloc_ptr[dev].store(p, std::memory_order_release);
    return p;
}
}  // namespace

extern "C" fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                                    const void* dO, const float* LSE, void* dQ, void* dK,
                                    void* dV, int B, int H, int N, int d, float tau, int causal,
                                    void* stream) {
    bool empty = false;
    const fa_status s = fa::check_shape(B, H, N, d, tau, causal, &empty);
    if (s != FA_OK || empty) return s;
    // the one limit of this entry point: the problem's scratch must fit the array
    if (fa_bwd_workspace_size(B, H, N, d) > FA_NOALLOC_SCRATCH_BYTES) return FA_ERR_WORKSPACE;
    // an unsupported device gets the same answer as from every other entry point
    fa_status why = FA_OK;
    if (fa::current_device(&why) == nullptr) return why;
    void* scratch = noalloc_scratch_for_current_device();
    if (scratch == nullptr) return FA_ERR_CUDA;
    // fa_bwd with a caller-provided workspace allocates nothing
    return fa_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, scratch, FA_NOALLOC_SCRATCH_BYTES, B, H, N, d,
                  tau, causal, stream);
}

