// internal.cuh -- shared declarations of the CUDA library (not part of the ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "gdn_layer.h"
#include "gdn_tree.h"

namespace gdn {

constexpr int kMaxNodes = 256;
constexpr int kMaxWords = kMaxNodes / 32;

__device__ __forceinline__ float load_f(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const __nv_bfloat16 *p, int64_t i) {
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ void store_f(float *p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16 *p, int64_t i, float x) {
    p[i] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ void flag(int32_t *status, int bits) {
    if (status) atomicOr(status, bits);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// the message behind gdn_last_error(): cleared at an entry, set with the code returned
void clear_error();
int fail(int code, const char *fmt, ...);

// ---------------------------------------------------------------------------
// launchers (one per translation unit); each returns a cudaError_t
// ---------------------------------------------------------------------------
cudaError_t launch_build_desc(const int32_t *parent, const int32_t *node_offsets, int batch,
                              int max_nodes, uint32_t *anc_mask, int mask_words,
                              int32_t *depth, int32_t *dev_status, cudaStream_t stream);

cudaError_t launch_verify_simt(const gdn_verify_args &a, cudaStream_t stream);
cudaError_t launch_relabel(const int32_t *parent_in, const int32_t *node_offsets, int batch, int total,
                           int max_nodes, int32_t *order, int32_t *rank, int32_t *parent_out,
                           int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_grow(const int32_t *node_offsets, int batch, int total, int width, int max_depth, int max_children,
                        const int32_t *n_children, const float *draws, int32_t *parent, float *score, int32_t *n_nodes,
                        int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_gather_rows(const void *src, void *dst, const int32_t *index, const int32_t *node_offsets,
                               int batch, int total, int64_t row_bytes, int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_verify_branches(const gdn_verify_args &a, cudaStream_t stream);
cudaError_t launch_commit_simt(const gdn_commit_args &a, cudaStream_t stream);

// TMA-staged commit for d_k = d_v = 128 and accepted paths of at most 16 nodes
bool commit_fast_supported(const gdn_commit_args &a);
cudaError_t launch_commit_fast(const gdn_commit_args &a, cudaStream_t stream);

// tensor-core commit for bf16 k/v, d_k = d_v = 128 and paths of at most 16 nodes
bool commit_tc_supported(const gdn_commit_args &a);
cudaError_t launch_commit_tc(const gdn_commit_args &a, cudaStream_t stream);

// the same kernel writing the states at selected nodes
bool states_tc_supported(const gdn_states_args &a);
cudaError_t launch_states_tc(const gdn_states_args &a, cudaStream_t stream);

// the layer around the tree (gdn_layer.h)
cudaError_t launch_prefill_simt(const gdn_prefill_args &a, cudaStream_t stream);
// chunked tensor-core prompts for bf16, d_k = d_v = 128
bool prefill_tc_supported(const gdn_prefill_args &a);
int64_t prefill_tc_workspace(const gdn_prefill_args &a);  // bytes, 256-byte aligned
cudaError_t launch_prefill_tc(const gdn_prefill_args &a, cudaStream_t stream);
cudaError_t launch_decode(const gdn_decode_args &a, cudaStream_t stream);
cudaError_t launch_qk_gates(const gdn_qk_gates_args &a, cudaStream_t stream);
cudaError_t launch_norm_gate(const gdn_norm_gate_args &a, cudaStream_t stream);
cudaError_t launch_residual_norm(const gdn_residual_norm_args &a, cudaStream_t stream);

// driver entry point for TMA descriptors (nullptr when the driver lacks it)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// A launch whose blocks may take their places while the kernel before it in the stream ends: the kernel calls
// after_previous() before it reads or writes global memory, which waits for that kernel to be done and lets the next
// one do the same.  The kernel before may write in this one's lifetime, so what it may have written is read with
// ordinary loads: __ldg and the like are for memory that nobody writes while the kernel lives, and the compiler may
// move them up past the wait.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// 16 bytes that are not needed again soon, for kernels launched like that: in order with the wait, and coherent.
__device__ __forceinline__ uint4 load_streaming(const void *p) {
    uint4 r;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

// Prompts longest first, so that none begins when the others are nearly done: the length of prompt b (-1 where its
// offsets are not a prompt's), and the place of number i among n lengths.
__device__ __forceinline__ int prompt_length(const int32_t *offsets, int b) {
    const int lo = __ldg(offsets + b), hi = __ldg(offsets + b + 1);
    return lo >= 0 && hi >= lo ? hi - lo : -1;
}
__device__ __forceinline__ int length_rank(const int *len, int n, int i) {
    const int mine = len[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += len[j] > mine || (len[j] == mine && j < i);
    return r;
}

// streaming multiprocessors on the current device (1 if the query fails)
int sm_count();

// Poll limit of the wait probe (0 = off), set by gdn_test_set_wait_probe.
int wait_probe_polls();

// Raise a kernel's dynamic shared-memory limit to `bytes` on the current device,
// once per (kernel, device, size): `have` remembers the largest size set so far
// per device.  Launches after the first make no attribute call, so they can be
// captured into a CUDA graph.
template <typename Kernel>
cudaError_t ensure_smem(Kernel kern, int bytes, int (&have)[16]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 16 && bytes <= have[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 16) have[dev] = bytes;
    return e;
}

// tcgen05/TMA fast path; after_commit launches it as the programmatic dependent
// of the commit launched just before it in the stream
bool verify_tc_supported(const gdn_verify_args &a);
cudaError_t launch_verify_tc(const gdn_verify_args &a, cudaStream_t stream, bool after_commit);

// the same for trees of 129 to 256 nodes (two node tiles per request)
bool verify_wide_supported(const gdn_verify_args &a);
cudaError_t launch_verify_wide(const gdn_verify_args &a, cudaStream_t stream, bool after_commit);

}  // namespace gdn
