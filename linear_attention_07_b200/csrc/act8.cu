// Activation checkpoints in 8 bits: bf16 rows into e4m3 with one power-of-two
// scale (E8M0: the biased exponent) per 32 channels, and back.
//
// The scale 2^e of a block is the smallest with max|x| <= 448 * 2^e, read off
// the bits of the largest magnitude: with max|x| = (1 + m / 128) 2^x it is
// e = x - 8 for m <= 96 (448 = 1.75 * 2^8) and x - 7 above, at least -127.
// Every step is exact but the one rounding to e4m3 (to nearest, ties to even),
// and a power-of-two scale makes every value of the 8-bit form exact in bf16
// again (down to bf16's own smallest numbers).  Nothing saturates, but for
// numbers that would round up to 2^128, which bf16 does not have: they become
// 240 * 2^120.  A block with an infinity or a NaN gets the scale 255 and reads
// as NaN.
//
// Bound by HBM: 2 bytes read and 1 + 1/32 written per value.  A thread takes
// UNITS times 8 channels, all loads first, so that a warp's accesses are whole
// lines on both sides (16 bytes a lane of bf16, 8 of e4m3) and four lanes share
// a block; one launch takes up to four tensors, whose rows may be slices of
// wider rows.  134 M values (16384 tokens of 64 x 128): packed in 73 us, 5.6
// TB/s, where issuing the conversions is as long as the loads; unpacked in 57 us
// (67 in a run of calls), 7.1 TB/s, part of it from L2.  With 16 channels a
// thread, 32 bytes apart, it was 81 and 82 us.
#include "kda_common.cuh"

namespace kda {
namespace act8 {

constexpr int NT = 256, UNITS = 4;
constexpr int MAX_TENSORS = 4;

struct Job {
    const void* src;       // pack: bf16 rows; unpack: e4m3
    void* dst;             // pack: e4m3; unpack: bf16
    uint8_t* scales;
    int64_t stride;        // elements between the bf16 rows
    int64_t n;             // 8-channel units
    int per_row;           // units per row, at least 4
    uint64_t recip;        // 2^64 / per_row, rounded up
};
struct Jobs {
    Job job[MAX_TENSORS];
};

// Unit i of the bf16 rows: i / per_row as a product, exact while i * per_row < 2^64 (a division is a hundred
// instructions, and these are what the kernel would wait for).
__device__ __forceinline__ const uint4* unit_of(const Job& j, int64_t i)
{
    const int64_t row = (int64_t)__umul64hi((uint64_t)i, j.recip);
    return reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(j.src) + row * j.stride) + (i - row * j.per_row);
}

__global__ void __launch_bounds__(NT) pack_kernel(const __grid_constant__ Jobs jobs)
{
    const Job& j = jobs.job[blockIdx.y];
    const int64_t i0 = (int64_t)blockIdx.x * (NT * UNITS) + threadIdx.x;
    uint4 in[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        if (i0 + u * NT < j.n) in[u] = __ldcs(unit_of(j, i0 + u * NT));
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const int64_t i = i0 + u * NT;
        if (i >= j.n) return;                        // n is a multiple of 4: the lanes of a block leave together
        const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
        // the largest magnitude as bits: NaN > infinity > every number
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
        const uint32_t block = 15u << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(block, m, 1));
        m = max(m, __shfl_xor_sync(block, m, 2));
        const int x_exp = (int)(m >> 7);
        int s = x_exp - ((m & 0x7fu) <= 96u ? 8 : 7);
        s = x_exp == 255 ? 255 : s < 0 ? 0 : s;
        const float inv = __uint_as_float((uint32_t)(254 - (s == 255 ? 0 : s)) << 23);     // 2^-e
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16) * inv;
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * inv;
        }
        if (s == 247) {                              // the scale 2^120, of magnitudes above 1.75 * 2^127
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -240.f), 240.f);
        }
        uint32_t out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * e], x[4 * e + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * e + 2], x[4 * e + 3]), __NV_SATFINITE, __NV_E4M3);
            out[e] = lo | (hi << 16);
        }
        reinterpret_cast<uint2*>(j.dst)[i] = make_uint2(out[0], out[1]);
        if ((i & 3) == 0) j.scales[i >> 2] = (uint8_t)s;
    }
}

__global__ void __launch_bounds__(NT) unpack_kernel(const __grid_constant__ Jobs jobs)
{
    const Job& j = jobs.job[blockIdx.y];
    const int64_t i0 = (int64_t)blockIdx.x * (NT * UNITS) + threadIdx.x;
    uint2 in[UNITS];
    uint32_t s[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        if (i0 + u * NT < j.n) {
            in[u] = __ldcs(reinterpret_cast<const uint2*>(j.src) + i0 + u * NT);
            s[u] = j.scales[(i0 + u * NT) >> 2];
        }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        if (i0 + u * NT >= j.n) return;
        uint32_t out[4];
        act8_expand(in[u], act8_scale(s[u]), out);
        reinterpret_cast<uint4*>(j.dst)[i0 + u * NT] = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

}  // namespace act8

cudaError_t act8_launch(int count, const void* const* src, void* const* dst, void* const* scales, const int64_t* rows,
                        const int64_t* cols, const int64_t* strides, bool pack, cudaStream_t stream)
{
    using namespace act8;
    Jobs jobs = {};
    int64_t most = 0;
    for (int t = 0; t < count; ++t) {
        Job& j = jobs.job[t];
        j.src = src[t];
        j.dst = dst[t];
        j.scales = (uint8_t*)scales[t];
        j.per_row = (int)(cols[t] / 8);
        j.n = rows[t] * j.per_row;
        j.recip = j.per_row ? ~(uint64_t)0 / j.per_row + 1 : 0;
        j.stride = strides ? strides[t] : cols[t];
        if (j.n > most) most = j.n;
    }
    if (most == 0) return cudaSuccess;
    const dim3 grid((unsigned)((most + NT * UNITS - 1) / (NT * UNITS)), (unsigned)count);
    if (pack) pack_kernel<<<grid, NT, 0, stream>>>(jobs);
    else unpack_kernel<<<grid, NT, 0, stream>>>(jobs);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
