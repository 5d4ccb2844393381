// Host-side declarations shared by the library's translation units.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <utility>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// Block masks (block-sparse attention): one byte per [128 query x 128 key] block,
// at most kMaxMaskBlocks blocks per row (so N <= 131072).
constexpr int kMaskBlockEdge = 128;
constexpr int kMaxMaskBlocks = 1024;

// Arguments of one forward launch (device pointers, validated by the caller).
struct FwdArgs {
    const void* Q;
    const void* K;
    const void* V;
    void* O;          // bf16 or fp32 (o32)
    float* LSE;
    int BH, N, d;
    float tau;
    bool causal;
    int window;       // causal sliding window in keys (0: none, or it hides nothing)
    int sinks = 0;    // keys [0, sinks) that stay visible behind the window (0 without one)
    const uint8_t* blocks = nullptr;  // block mask [heads][nb][nb] (device) or null
    long long blocks_head_stride = 0;  // bytes between heads' masks (0: one mask)
    bool o32;
    unsigned int* err;
    unsigned long long wait_limit_ns;
    cudaEvent_t ev_start;  // optional: recorded around the kernel
    cudaEvent_t ev_stop;
};

// Arguments of one backward launch sequence.
struct BwdArgs {
    const void* Q;
    const void* K;
    const void* V;
    const void* O;
    const void* dO;
    const float* LSE;
    void* dQ;
    void* dK;
    void* dV;
    float* D;       // workspace: fp32 [BH*N]
    float* dQacc;   // workspace: fp32 [BH*N*d]
    int BH, N, d;
    float tau;
    bool causal;
    int window;     // causal sliding window in keys, at most N (0 = none)
    int sinks = 0;  // keys [0, sinks), at most N, that stay visible behind the window
    const uint8_t* blocks = nullptr;  // block mask [heads][nb][nb] (device) or null
    long long blocks_head_stride = 0;  // bytes between heads' masks (0: one mask)
    unsigned int* err;
    unsigned long long wait_limit_ns;
    cudaEvent_t ev_start;  // optional: recorded around the main kernel
    cudaEvent_t ev_stop;
};

// Arguments of one FP8 (e4m3) forward: Q, K, V are e4m3 bytes [BH][N][128]
// with one scale per tensor (value = byte * scale); O bf16, LSE fp32.
struct Fp8Args {
    const void* Q;
    const void* K;
    const void* V;
    void* O;
    float* LSE;
    int BH, N;
    float tau, q_scale, k_scale, v_scale;
    bool causal;
    unsigned int* err;
    unsigned long long wait_limit_ns;
    cudaEvent_t ev_start;  // optional: recorded around the kernel
    cudaEvent_t ev_stop;
};

// Arguments of one decode forward (split kernel + combine kernel).
struct DecArgs {
    const void* Q;    // bf16 [BH][Nq][d]
    const void* K;    // bf16 [BH][Nk][d]
    const void* V;
    void* O;          // bf16 [BH][Nq][d]
    float* LSE;       // fp32 [BH][Nq]
    float* workspace; // splits > 1: partials (decode_workspace_bytes)
    int BH, Nq, Nk, d;
    float tau;
    bool causal;
    int splits, chunk;  // from decode_plan
    unsigned int* err;
    unsigned long long wait_limit_ns;
    cudaEvent_t ev_start;  // optional: recorded around the two kernels
    cudaEvent_t ev_stop;
};

// A paged key/value cache: K, V [num_pages][H_kv][1 << shift][d], bf16, or e4m3 with
// scales [num_pages][H_kv] (null for bf16); page_table [B][max_pages], lens [B].
struct PagedCache {
    void* K;
    void* V;
    float* k_scale;
    float* v_scale;
    const int* page_table;
    const int* lens;
    int B, H_kv, d, num_pages, max_pages, shift;
};

// Records a length, token count or page number out of bounds: in the second error word, so
// that it never stands before a timeout (the first: 1 | site << 8 of the first wait that ran
// out).
__device__ __forceinline__ void page_error(unsigned int* err) { *reinterpret_cast<volatile unsigned int*>(err + 1) = 1u; }

// Arguments of one append.  Strides in elements: token, head.
struct AppendArgs {
    PagedCache cache;
    const void* q;       // bf16 [T][H][d], or null
    const void* k;       // bf16 [T][H_kv][d]
    const void* v;
    void* q_out;
    const int* cu_new;   // [B + 1], or null: T / B tokens each
    const double* inv_freq;  // [rot / 2]
    long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;
    int T, H, rot, interleaved;
    unsigned int* err;
};

// What changes the scores of an attention call, and which are hidden (fa_score in
// include/fa.h; device pointers, validated by the caller).
struct ScoreMod {
    float softcap = 0.f;            // 0: none
    const float* slopes = nullptr;  // [H]
    const void* table = nullptr;    // [num_buckets][H], bf16 or fp32 (table_f32)
    const int* buckets = nullptr;   // [2 far + 1]
    bool table_f32 = false;
    int num_buckets = 0, far = 0;
    const int* docs = nullptr;      // [B][N]
    const int* prefix = nullptr;    // [B]
    int window = 0;                 // causal sliding window, at most N (0: none)
};

// Arguments of one attention step over a paged cache.  Strides in elements: sequence,
// head, row.
struct PagedArgs {
    PagedCache cache;
    const void* Q;     // bf16 [B][H][Nq][d]
    void* O;
    float* LSE;        // fp32 [B][H][Nq]
    void* workspace;
    long long q_sb, q_sh, q_sn, o_sb, o_sh, o_sn;
    int H, Nq, window, sinks;
    float tau;
    ScoreMod mod;      // (launch_fwd_paged_score; no documents, prefix or window of its own)
    unsigned int* err;
    cudaEvent_t ev_start;  // optional: recorded around the two kernels
    cudaEvent_t ev_stop;
};
// Bytes of workspace one such step takes, whatever the sequences' lengths (only the
// cache's sizes are looked at).
size_t paged_workspace(const PagedCache& c, int H, int Nq, int window, int sinks, bool fp8);
// 16-key tiles that full tables hold, which 32-bit counts must not pass.
long long paged_max_tiles(int B, int H, int H_kv, int Nq, int max_pages, int shift);

// Arguments of attention with such scores, forward and backward.
struct ScoreArgs {
    const void* Q;   // bf16 [B][H][N][d]; K, V [B][H_kv][N][d]
    const void* K;
    const void* V;
    void* O;         // (the backward does not need it)
    float* LSE;      // (backward: read)
    const void* dO = nullptr;
    void* dQ = nullptr;
    void* dK = nullptr;
    void* dV = nullptr;
    void* dTable = nullptr;  // [num_buckets][H], of the table's type
    uint8_t* workspace;
    int B, H, H_kv, N, d;
    float tau;
    bool causal;
    ScoreMod mod;
    unsigned int* err;
    unsigned long long wait_limit_ns;
    cudaEvent_t ev_start;  // optional: recorded around the main kernel
    cudaEvent_t ev_stop;
};
// Orders in which tiles are taken, each [B][tiles], or null: of 128 queries, of 256, of 128 keys.
struct ScoreOrder {
    int* queries = nullptr;
    int* pairs = nullptr;
    int* keys = nullptr;
};
size_t score_fwd_workspace(int B, int N, bool docs);
size_t score_bwd_workspace(const ScoreArgs& a, bool grad);  // grad: with the table's

// How the decode forward cuts the KV cache: `splits` chunks of `chunk` keys
// (a multiple of 64).  Depends only on its arguments.
void decode_plan(int BH, int Nk, int* splits, int* chunk);

// Encodes a 3-D tiled tensor map over a contiguous [BH][N][cols] tensor with
// a {box_cols, box_rows, 1} box and the 128-byte swizzle (box_cols * esize
// must be 128).  Returns false if the driver rejects it.  make_tile_map keeps
// the maps it has encoded and returns a kept one for the same arguments.
bool make_tile_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                   int cols, int rows, int planes, int box_cols, int box_rows);
bool encode_tile_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                     int cols, int rows, int planes, int box_cols, int box_rows);

// Raises a kernel's dynamic shared-memory limit to `bytes`, once per device
// (the attribute stays set; later calls only check a flag).
template <auto Kern>
cudaError_t set_max_dyn_smem_once(int bytes) {
    static std::atomic<int> done[64] = {};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
    const bool cacheable = dev >= 0 && dev < 64;
    if (cacheable && done[dev].load(std::memory_order_acquire) == bytes) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && cacheable) done[dev].store(bytes, std::memory_order_release);
    return e;
}

// Launches `kern` as a programmatic dependent of the previous kernel on the
// stream: it may be scheduled before that kernel has finished, and must call
// griddepcontrol.wait before touching anything that kernel writes.
// (clusters: in clusters of that many blocks along x.)
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_clusters(void (*kern)(KArgs...), unsigned cluster, dim3 grid, dim3 block, size_t smem,
                                      cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
    return launch_dependent_clusters(kern, 1u, grid, block, smem, stream, std::forward<Args>(args)...);
}

cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t stream);
// d = 64, bf16 O, no block mask: the persistent forward for N <= 2048 without a window,
// and for causal windows with sinks (sinks > 0)
cudaError_t launch_fwd_short(const FwdArgs& a, cudaStream_t stream);
// d = 128 with a block mask, bf16 O: the persistent block-sparse forward
cudaError_t launch_fwd_sparse(const FwdArgs& a, cudaStream_t stream);
cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t stream);
cudaError_t launch_score_fwd(const ScoreArgs& a, cudaStream_t stream);
cudaError_t launch_score_bwd(const ScoreArgs& a, cudaStream_t stream);
// D_i = sum_j P_ij dP_ij and a zeroed dQ accumulator (spans, order of pairs and bias2: of the workspace, or null)
cudaError_t launch_score_rows(const ScoreArgs& a, float* dvec, float* acc, unsigned* next, const void* spans, const int* order,
                              const float* bias2, cudaStream_t stream);
// documents' ids -> each token's document as [first, end) (int2 [B][N]), and tiles' orders
cudaError_t launch_score_spans(const ScoreArgs& a, void* spans, const ScoreOrder& order, cudaStream_t stream);
size_t score_spans_bytes(int B, int N);
cudaError_t launch_decode(const DecArgs& a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_paged_score(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_fp8(const Fp8Args& a, cudaStream_t stream);
cudaError_t launch_watchdog_selftest(unsigned int* err, unsigned long long limit_ns,
                                     cudaStream_t stream);

}  // namespace fa
