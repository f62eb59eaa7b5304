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
// 16 channels (two 16-byte loads, one 16-byte store), two lanes share a block;
// one launch takes up to four tensors, whose rows may be slices of wider rows.
#include "kda_common.cuh"

namespace kda {
namespace act8 {

constexpr int NT = 256;
constexpr int MAX_TENSORS = 4;

struct Job {
    const void* src;       // pack: bf16 rows; unpack: e4m3
    void* dst;             // pack: e4m3; unpack: bf16
    uint8_t* scales;
    int64_t stride;        // elements between the bf16 rows
    int64_t n;             // 16-channel pieces
    int per_row;           // pieces per row
};
struct Jobs {
    Job job[MAX_TENSORS];
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

__global__ void __launch_bounds__(NT) pack_kernel(const __grid_constant__ Jobs jobs)
{
    const Job& j = jobs.job[blockIdx.y];
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= j.n) return;                            // n is even: the two lanes of a block leave together
    const int64_t row = i / j.per_row;
    const int c = (int)(i - row * j.per_row);
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(j.src) + row * j.stride) + 2 * c;
    const uint4 x[2] = {__ldcs(p), __ldcs(p + 1)};
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    // the largest magnitude as bits: NaN > infinity > every number
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_u16x2(m, w[e] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    const uint32_t pair = 3u << (threadIdx.x & 30);
    m = max(m, __shfl_xor_sync(pair, m, 1));
    const int x_exp = (int)(m >> 7);
    int s = x_exp - ((m & 0x7fu) <= 96u ? 8 : 7);
    s = x_exp == 255 ? 255 : s < 0 ? 0 : s;
    const float inv = __uint_as_float((uint32_t)(254 - (s == 255 ? 0 : s)) << 23);     // 2^-e
    const float most = s == 247 ? 240.f : 448.f;     // 247: the scale 2^120, of magnitudes above 1.75 * 2^127
    auto q = [&](float x) { return fminf(fmaxf(x * inv, -most), most); };
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * e]));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * e + 1]));
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q(a.x), q(a.y)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q(b.x), q(b.y)), __NV_SATFINITE, __NV_E4M3);
        out[e] = lo | (hi << 16);
    }
    reinterpret_cast<uint4*>(j.dst)[i] = make_uint4(out[0], out[1], out[2], out[3]);
    if ((i & 1) == 0) j.scales[i >> 1] = (uint8_t)s;
}

__global__ void __launch_bounds__(NT) unpack_kernel(const __grid_constant__ Jobs jobs)
{
    const Job& j = jobs.job[blockIdx.y];
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= j.n) return;
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(j.src) + i);
    const float sc = act8_scale(j.scales[i >> 1]);
    uint32_t out[8];
    act8_expand(x, sc, out);
    uint4* p = reinterpret_cast<uint4*>(j.dst) + 2 * i;
    p[0] = make_uint4(out[0], out[1], out[2], out[3]);
    p[1] = make_uint4(out[4], out[5], out[6], out[7]);
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
        j.per_row = (int)(cols[t] / 16);
        j.n = rows[t] * j.per_row;
        j.stride = strides ? strides[t] : cols[t];
        if (j.n > most) most = j.n;
    }
    if (most == 0) return cudaSuccess;
    const dim3 grid((unsigned)((most + NT - 1) / NT), (unsigned)count);
    if (pack) pack_kernel<<<grid, NT, 0, stream>>>(jobs);
    else unpack_kernel<<<grid, NT, 0, stream>>>(jobs);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
