// Gated delta rule, one decay per head: one token for each of N requests,
// state updated in place.  Per (request, value head), with a = exp(g):
//   p = a S^T k,  r = a S^T q,  u = beta (v - p),
//   o = scale (r + (q . k) u)  (= scale S_new^T q),   S_new = a S + k u^T.
//
// Bound by HBM: the fp32 state is read once and written once (128 KB per
// request and head at d_k = d_v = 128), everything else is 1 % of that.  The
// state's columns are independent, but a CTA of 256 threads takes all of them:
// thread (rg, cg) owns columns 4 cg .. 4 cg + 3 of rows rg, rg + RSTEP, ... ,
// every access a 16-byte vector of a full 128-byte line, all loads of the
// state issued before any arithmetic: more bytes in flight per thread.  Four
// CTAs of 32 columns each took as long at 32 states of 128 x 128 (5.6 us) and
// longer at all other counts (8.0 against 5.9 us at 128, 41 against 25 us at
// 1184).  176 us for 256 requests x 32 heads: 6.1 TB/s.  The two column sums over d_k go through
// shuffles where lanes of a warp share a column group and one shared-memory
// pass.
#include "gdn_common.cuh"

namespace kda {
namespace gdn {

constexpr int STEP_NT = 256;

template <int DK, int DV>
struct StepMap {
    static constexpr int CG = DV / 4;                // float4 column groups
    static constexpr int RSTEP = STEP_NT / CG;       // rows covered per pass
    static constexpr int ROWS = (DK + RSTEP - 1) / RSTEP;
    static_assert(DK % RSTEP == 0, "rows per thread");
};

template <int DK, int DV>
__global__ void __launch_bounds__(STEP_NT)
step_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
            const __nv_bfloat16* __restrict__ v, const void* __restrict__ g, const void* __restrict__ beta,
            float* __restrict__ state, __nv_bfloat16* __restrict__ o, const int* __restrict__ slots, int n_slots,
            float scale, int HK, int HV, int64_t q_stride, int64_t k_stride, int64_t v_stride, int f32_gates)
{
    using M = StepMap<DK, DV>;
    constexpr int CG = M::CG, RSTEP = M::RSTEP, ROWS = M::ROWS;
    __shared__ float sh_k[DK], sh_q[DK], sh_qk;
    __shared__ float4 red[2][RSTEP][CG];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    const int hv = blockIdx.y;
    const int64_t n = blockIdx.x;
    const int64_t row = slots ? slots[n] : n;
    __nv_bfloat16* on = o + (n * HV + hv) * DV + 4 * cg;
    if (row < 0 || row >= n_slots) {                 // a padded row of the batch: no state, o = 0
        if (rg == 0) *reinterpret_cast<uint2*>(on) = make_uint2(0u, 0u);
        return;
    }
    float* S = state + (row * HV + hv) * (int64_t)(DK * DV) + 4 * cg;
    float4 s[ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
        s[m] = __ldcs(reinterpret_cast<const float4*>(S + (rg + m * RSTEP) * DV));
    const int hk = hv / (HV / HK);
    if (tid < DK) {
        sh_k[tid] = to_f32(k[n * k_stride + hk * DK + tid]);
        sh_q[tid] = to_f32(q[n * q_stride + hk * DK + tid]);
    }
    const __nv_bfloat162* v2 = reinterpret_cast<const __nv_bfloat162*>(v + n * v_stride + (int64_t)hv * DV + 4 * cg);
    const float2 v01 = __bfloat1622float2(v2[0]), v23 = __bfloat1622float2(v2[1]);
    // one branch per pair of types, so that both loads go out together
    const int64_t at = n * HV + hv;
    float a, b;
    if (f32_gates == 0) a = gate(g, at, false), b = gate(beta, at, false);
    else if (f32_gates == G_F32) a = gate(g, at, true), b = gate(beta, at, false);
    else a = gate(g, at, true), b = gate(beta, at, true);
    a = expf(a);
    __syncthreads();
    if (tid < 32) {
        float acc = 0.f;
        for (int i = tid; i < DK; i += 32) acc = fmaf(sh_q[i], sh_k[i], acc);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (tid == 0) sh_qk = acc;
    }
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f), r = p;
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
        const float ki = sh_k[rg + m * RSTEP], qi = sh_q[rg + m * RSTEP];
        p.x = fmaf(s[m].x, ki, p.x); p.y = fmaf(s[m].y, ki, p.y); p.z = fmaf(s[m].z, ki, p.z); p.w = fmaf(s[m].w, ki, p.w);
        r.x = fmaf(s[m].x, qi, r.x); r.y = fmaf(s[m].y, qi, r.y); r.z = fmaf(s[m].z, qi, r.z); r.w = fmaf(s[m].w, qi, r.w);
    }
    red[0][rg][cg] = p;
    red[1][rg][cg] = r;
    __syncthreads();
    float4 P = make_float4(0.f, 0.f, 0.f, 0.f), R = P;
#pragma unroll
    for (int w = 0; w < RSTEP; ++w) {
        const float4 x = red[0][w][cg];
        P.x += x.x; P.y += x.y; P.z += x.z; P.w += x.w;
    }
    float4 u;
    u.x = b * (v01.x - a * P.x); u.y = b * (v01.y - a * P.y);
    u.z = b * (v23.x - a * P.z); u.w = b * (v23.y - a * P.w);
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
        const float ki = sh_k[rg + m * RSTEP];
        float4 x;
        x.x = fmaf(ki, u.x, a * s[m].x); x.y = fmaf(ki, u.y, a * s[m].y);
        x.z = fmaf(ki, u.z, a * s[m].z); x.w = fmaf(ki, u.w, a * s[m].w);
        __stcs(reinterpret_cast<float4*>(S + (rg + m * RSTEP) * DV), x);
    }
    if (rg == 0) {
        for (int w = 0; w < RSTEP; ++w) {
            const float4 x = red[1][w][cg];
            R.x += x.x; R.y += x.y; R.z += x.z; R.w += x.w;
        }
        const float qk = sh_qk;
        const __nv_bfloat162 o01 = __floats2bfloat162_rn(scale * fmaf(qk, u.x, a * R.x), scale * fmaf(qk, u.y, a * R.y));
        const __nv_bfloat162 o23 = __floats2bfloat162_rn(scale * fmaf(qk, u.z, a * R.z), scale * fmaf(qk, u.w, a * R.w));
        reinterpret_cast<__nv_bfloat162*>(on)[0] = o01;
        reinterpret_cast<__nv_bfloat162*>(on)[1] = o23;
    }
}

}  // namespace gdn

cudaError_t gdn_step_launch(const void* q, const void* k, const void* v, const void* g, const void* beta, float* state,
                            void* o, const int* slots, int n_slots, float scale, int N, int HK, int HV, int dk, int dv,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride, int f32_gates, cudaStream_t stream)
{
    using namespace gdn;
    using bf = __nv_bfloat16;
#define GDN_STEP(DK_, DV_)                                                                                      \
    step_kernel<DK_, DV_><<<dim3((unsigned)N, (unsigned)HV), STEP_NT, 0, stream>>>(                              \
        (const bf*)q, (const bf*)k, (const bf*)v, g, beta, state, (bf*)o, slots, n_slots, scale, HK, HV,         \
        q_stride, k_stride, v_stride, f32_gates)
#define GDN_STEP_DV(DK_) \
    if (dv == 128) GDN_STEP(DK_, 128); else if (dv == 64) GDN_STEP(DK_, 64); else GDN_STEP(DK_, 32)
    if (dk == 128) { GDN_STEP_DV(128); }
    else if (dk == 64) { GDN_STEP_DV(64); }
    else { GDN_STEP_DV(32); }
#undef GDN_STEP_DV
#undef GDN_STEP
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
