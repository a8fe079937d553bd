// Attention for a tree of drafted tokens over the paged cache (sm_103a).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb_device.cuh"
#include "tb_kv.h"

namespace tb {
namespace {

using namespace dev;

constexpr int kThreads = 128;
constexpr int kRows = 16;     // query rows of a CTA, kRows / 4 per warp
constexpr int kTile = 32;     // positions of a tile, one per lane
constexpr int kMaxDim = 128;

template <class T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__half x)
{
    return __half2float(x);
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float(float x)
{
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x)
{
    return __float2bfloat16_rn(x);
}

// One CTA: kRows rows of one sequence and cache head; rows are (draft, head of
// the group) pairs.  One pass over the positions in tiles with the running
// maximum and sum of the softmax; a lane holds one position's score, then a
// stripe of the output.
template <class T>
__global__ void __launch_bounds__(kThreads) k_tree_plain(const TreePlan p)
{
    __shared__ float q[kRows][kMaxDim], key[kTile][kMaxDim + 1], value[kTile][kMaxDim];
    __shared__ int s_seq, s_block;
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const KvView &c = p.c;
    if (threadIdx.x == 0) {
        int left = blockIdx.x, b = 0;
        for (; b < p.seqs; ++b) {
            const int t = min(p.q_start[b + 1], p.rows) - max(p.q_start[b], 0);
            const int blocks = max((t * p.group + kRows - 1) / kRows, 0);
            if (left < blocks)
                break;
            left -= blocks;
        }
        s_seq = b;
        s_block = left;
    }
    __syncthreads();
    const int b = s_seq;
    if (b >= p.seqs)
        return;
    const int slot = p.seq_slots ? p.seq_slots[b] : b;
    const int row0 = max(p.q_start[b], 0), drafts = min(p.q_start[b + 1], p.rows) - row0;
    const bool known = slot >= 0 && slot < c.slots;
    const int n = known ? max(c.lens[slot], 0) : 0, end = known ? n + drafts : 0;
    const int head = blockIdx.y, D = p.head_dim;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
        const int r = s_block * kRows + i / D, d = i % D;
        float x = 0.0f;
        if (r < drafts * p.group)
            x = to_float(reinterpret_cast<const T *>(p.q + (row0 + r / p.group) * p.q_row +
                                                     (head * p.group + r % p.group) * p.q_head)[d]);
        q[i / D][d] = x;
    }
    float top[kRows / 4], sum[kRows / 4], acc[kRows / 4][kMaxDim / 32];
#pragma unroll
    for (int r = 0; r < kRows / 4; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.0f;
        for (int i = 0; i < kMaxDim / 32; ++i)
            acc[r][i] = 0.0f;
    }
    for (int base = 0; base < end; base += kTile) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * D; i += kThreads) {
            const int j = base + i / D, d = i % D;
            float kx = 0.0f, vx = 0.0f;
            if (j < end && j / c.page_tokens < c.width) {
                const int page = c.table[(int64_t)slot * c.width + j / c.page_tokens];
                if (page >= 0 && page < c.pages) {
                    const int64_t at = page * c.page_stride + j % c.page_tokens * c.token_stride +
                                       head * c.head_stride;
                    kx = to_float(reinterpret_cast<const T *>(c.pool[0] + at)[d]);
                    vx = to_float(reinterpret_cast<const T *>(c.pool[1] + at)[d]);
                }
            }
            key[i / D][d] = kx;
            value[i / D][d] = vx;
        }
        __syncthreads();
        const int j = base + lane, draft = j - n;
#pragma unroll
        for (int r = 0; r < kRows / 4; ++r) {
            const int row = s_block * kRows + warp * (kRows / 4) + r;
            if (row >= drafts * p.group)
                break;
            bool seen = j < n;
            if (draft >= 0 && draft < drafts && draft / 32 < p.mask_words)
                seen = p.mask[(int64_t)(row0 + row / p.group) * p.mask_words + draft / 32] >>
                           (draft % 32) & 1u;
            float s = -INFINITY;
            if (seen) {
                s = 0.0f;
                for (int d = 0; d < D; ++d)
                    s = fmaf(q[warp * (kRows / 4) + r][d], key[lane][d], s);
                s *= p.scale;
            }
            float m = s;
            for (int o = 16; o; o /= 2)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, top[r]);
            const float shift = m == -INFINITY ? 0.0f : m;
            const float w = expf(s - shift), old = expf(top[r] - shift);
            float total = w;
            for (int o = 16; o; o /= 2)
                total += __shfl_xor_sync(0xffffffffu, total, o);
            sum[r] = sum[r] * old + total;
            top[r] = m;
            const uint32_t visible = __ballot_sync(0xffffffffu, seen);
#pragma unroll
            for (int i = 0; i < kMaxDim / 32; ++i)
                acc[r][i] *= old;
            for (int k = 0; k < kTile; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (visible >> k & 1u)  // a hidden value never enters, even times 0
#pragma unroll
                    for (int i = 0; i < kMaxDim / 32; ++i)
                        if (lane + 32 * i < D)
                            acc[r][i] = fmaf(wk, value[k][lane + 32 * i], acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows / 4; ++r) {
        const int row = s_block * kRows + warp * (kRows / 4) + r;
        if (row >= drafts * p.group)
            break;
        const int64_t t = row0 + row / p.group;
        const int h = head * p.group + row % p.group;
        const float inv = sum[r] > 0.0f ? 1.0f / sum[r] : sum[r] == 0.0f ? 0.0f : NAN;
        T *out = reinterpret_cast<T *>(p.out + t * p.o_row + h * p.o_head);
#pragma unroll
        for (int i = 0; i < kMaxDim / 32; ++i)
            if (lane + 32 * i < D)
                out[lane + 32 * i] = from_float<T>(acc[r][i] * inv);
        if (p.lse && lane == 0)
            p.lse[t * p.q_heads + h] = top[r] + logf(sum[r]);
    }
}

}  // namespace

uint64_t tree_workspace_bytes(int num_sms, int head_dim)
{
    (void)num_sms;
    (void)head_dim;
    return 16;
}

cudaError_t launch_tree(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream)
{
    (void)num_sms;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int64_t blocks = (int64_t)p.rows * p.group / kRows + p.seqs;
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)p.c.heads);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return p.bf16 ? cudaLaunchKernelEx(&cfg, k_tree_plain<__nv_bfloat16>, p)
                  : cudaLaunchKernelEx(&cfg, k_tree_plain<__half>, p);
}

}  // namespace tb
