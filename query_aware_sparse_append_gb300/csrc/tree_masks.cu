// tree_masks.cu -- mask rows and depths of trees of drafted tokens from their parents.
//
//   M_t = M_parent(t) | 1 << t,   depth_t = depth_parent(t) + 1  (0 without a parent)
//
// One thread per token walks up to the top, as many steps as its token is deep, over the
// sequence's parents in shared memory; its mask row lies there too and goes out in
// whole words.  A step's masks serve all layers of a model: what it takes is its launch
// (8 tokens: 3.4 us cold).
#include "qasa_device.cuh"
#include "qasa_launch.h"

namespace qasa {

namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) tree_masks_kernel(TreeMaskParams p) {
    extern __shared__ int smem[];
    int *up = smem;                               // parents of all tokens
    uint32_t *rows = reinterpret_cast<uint32_t *>(smem + p.T);
    const int b = blockIdx.y, t0 = blockIdx.x * kThreads, t = t0 + threadIdx.x;
    int n = p.lens ? p.lens[b] : p.T;
    if (n < 0 || n > p.T) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, QASA_DEVERR_APPEND);
        n = n < 0 ? 0 : p.T;
    }
    if (t0 >= n) return;
    const int last = min(n, t0 + kThreads);       // parents come before their children
    for (int i = threadIdx.x; i < last; i += kThreads) {
        int parent = p.parents[(size_t)b * p.T + i];
        if (parent < -1 || parent >= i) {
            if (i >= t0 && p.status) atomicOr(p.status, QASA_DEVERR_PARENT);
            parent = -1;
        }
        up[i] = parent;
    }
    for (int i = threadIdx.x; i < kThreads * p.words; i += kThreads) rows[i] = 0;
    __syncthreads();
    if (t < last) {
        int depth = -1;
        for (int at = t; at >= 0; at = up[at]) {
            rows[threadIdx.x * p.words + (at >> 5)] |= 1u << (at & 31);
            ++depth;
        }
        if (p.depths) p.depths[(size_t)b * p.T + t] = depth;
    }
    __syncthreads();
    int32_t *out = p.mask + ((size_t)b * p.T + t0) * p.words;
    for (int i = threadIdx.x; i < (last - t0) * p.words; i += kThreads) out[i] = (int32_t)rows[i];
}

}  // namespace

cudaError_t launch_tree_masks(const TreeMaskParams &p, int batch, cudaStream_t stream) {
    const size_t smem = 4u * ((size_t)p.T + kThreads * p.words);      // 20 KB for 1024 tokens
    tree_masks_kernel<<<dim3((p.T + kThreads - 1) / kThreads, batch), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace qasa
