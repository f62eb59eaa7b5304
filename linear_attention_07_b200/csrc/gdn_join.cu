// Gated delta rule, one decay per head: the start states of segments that ran
// at the same time (gdn_chunk.cuh).
#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

// start_{p+1} = M_p start_p + N_p in fp32 for 32 columns of one head, a step
// after the other; M_{p+1} is on its way in registers meanwhile.  Thread: rows
// tid / 8 + 32 r, columns 4 (tid % 8) .. + 3.
// 9 us for one step of 32 heads, 4 us for each further one (64 KB of M from L2
// and 4,100 cycles of FMAs a CTA).
constexpr int JOIN_NT = 256, JOIN_COLS = 32, JOIN_LD = D + 4;
constexpr uint32_t JOIN_SMEM = (D * JOIN_LD + D * JOIN_COLS) * 4;

__global__ void __launch_bounds__(JOIN_NT)
join_kernel(const __grid_constant__ JoinArgs p)
{
    const JoinSet& a = p.set[blockIdx.z];
    extern __shared__ __align__(16) float jsm[];
    float* m = jsm;                                  // [D][JOIN_LD]
    float* st = jsm + D * JOIN_LD;                   // [D][JOIN_COLS]
    const int tid = threadIdx.x, l = blockIdx.y / p.HV, hv = blockIdx.y % p.HV, between = p.between;
    if (long_sequence(p.seqs, p.min_chunks, l) < 0) return;
    const int row = tid / 8, cs = 4 * (tid % 8), col = blockIdx.x * JOIN_COLS + cs;
    const int64_t head = ((int64_t)l * p.HV + hv) * D * D;
    auto mid = [&](int k) { return (((int64_t)l * between + k) * p.HV + hv) * D * D; };
    float4 next[D * D / 4 / JOIN_NT], cur[4];
    auto load = [&](int k) {
        const float4* src = reinterpret_cast<const float4*>(a.M + mid(k));
#pragma unroll
        for (int u = 0; u < D * D / 4 / JOIN_NT; ++u) next[u] = src[u * JOIN_NT + tid];
    };
    load(0);
#pragma unroll
    for (int r = 0; r < 4; ++r) cur[r] = *reinterpret_cast<const float4*>(a.first + head + (row + 32 * r) * D + col);
#pragma unroll 1
    for (int k = 0; k < between; ++k) {
        float4 acc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t at = mid(k) + (row + 32 * r) * D + col;
            acc[r] = *reinterpret_cast<const float4*>(a.N + at);
            *reinterpret_cast<float4*>(a.start + at) = cur[r];
        }
        __syncthreads();                             // the last step has read m and st
#pragma unroll
        for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(st + (row + 32 * r) * JOIN_COLS + cs) = cur[r];
#pragma unroll
        for (int u = 0; u < D * D / 4 / JOIN_NT; ++u) {
            const int e = 4 * (u * JOIN_NT + tid);
            *reinterpret_cast<float4*>(m + e / D * JOIN_LD + e % D) = next[u];
        }
        __syncthreads();
        if (k + 1 < between) load(k + 1);
#pragma unroll 4
        for (int i = 0; i < D; i += 4) {
            float4 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float4*>(st + (i + e) * JOIN_COLS + cs);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 y = *reinterpret_cast<const float4*>(m + (row + 32 * r) * JOIN_LD + i);
                const float f[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[r].x = fmaf(f[e], x[e].x, acc[r].x); acc[r].y = fmaf(f[e], x[e].y, acc[r].y);
                    acc[r].z = fmaf(f[e], x[e].z, acc[r].z); acc[r].w = fmaf(f[e], x[e].w, acc[r].w);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) cur[r] = acc[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(a.before_last + head + (row + 32 * r) * D + col) = cur[r];
}

static DeviceFlags g_join_attr_done;

cudaError_t join_launch(const JoinArgs& a, int sets, int64_t heads, cudaStream_t stream)
{
    const cudaError_t e = once_per_device(g_join_attr_done, [](int) {
        return cudaFuncSetAttribute(join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)JOIN_SMEM);
    });
    if (e != cudaSuccess) return e;
    join_kernel<<<dim3(D / JOIN_COLS, (unsigned)heads, (unsigned)sets), JOIN_NT, JOIN_SMEM, stream>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace gdn
}  // namespace kda
