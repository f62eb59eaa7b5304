// Gated delta rule, one decay per head: chunked forward, after the prep kernel
// (gdn_prep.cu).  One CTA per sequence and value head carries the state
// through the chunks; per chunk (gdn_chunk.cuh)
//     X_K = K S,  X_Q = Q S,  R = beta (V - gam X_K),  U = X R,
//     O = scale gam X_Q + P U,  S <- gam_last S + K^T (eta U).
// Every product is computed transposed, with d_v as the M = 128 of the MMA:
//     X^T = S^T K^T,  U^T = R^T X^T,  O^T = U^T P^T,  S^T += (eta U)^T K,
// so the left operands (S, R, U: fp32 values as two bf16) go from registers
// to tensor memory, the right ones (K, Q, X, P: bf16 in memory) stay as TMA
// left them, and thread j owns column j of S, R, U and O throughout: nothing
// the chain computes passes through shared memory.  Sums are fp32; the state
// is updated in fp32 registers (never accumulated in tensor memory, whose
// additions need not round to nearest).
//
// Roles (14 warps):
//   warps 0-7   chain: thread (j, half) holds S[dk][j] for 32 + 32 values of
//               dk; R, U, the state update, and their split into bf16 pairs
//   warps 8-11  output: thread j takes O^T's row j, 64 tokens, through
//               shared memory to 16-byte stores, off the chain's path
//   warp 12     issues every MMA
//   warp 13     loads: K, Q (128-byte swizzle), V, the chunk's record, two
//               stages
// The chain is what bounds it (per chunk three products that wait for one
// another, with the conversions between them).  To shorten it the state is
// updated in two halves of d_k: while the second half of K^T U is computed
// the first half is updated and split, and X_K starts on it.
#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

__device__ int g_fwd_status;

namespace fw {

constexpr int N_CHAIN = 8, N_OUT = 4;                // warps
constexpr int W_MMA = N_CHAIN + N_OUT, W_LOAD = W_MMA + 1;
constexpr int NT = 32 * (W_LOAD + 1);

// a stage: K0 Q0 K1 Q1 (boxes of 64 tokens x 64 channels), V rows, record
constexpr uint32_t S_V = 4 * 8192;
constexpr uint32_t S_REC = S_V + C * D * 2;
constexpr uint32_t STAGE = S_REC + REC_BYTES;
static_assert(STAGE % 1024 == 0, "swizzled tiles are 1024-byte aligned");
constexpr uint32_t OST = 2 * STAGE;                  // o staging [64][128] bf16
constexpr uint32_t SMEM = OST + C * D * 2 + 1024;

// barriers
enum { B_FULL = 0, B_READY = 2, B_EMPTY = 4, B_MX = 6, B_MU, B_MD0, B_MD1, B_MO, B_S0, B_S1, B_R, B_U, B_OFREE, B_DRAIN, N_BAR };

// tensor memory columns
constexpr uint32_t T_SH = 0, T_SL = 64;              // S^T, upper and lower half: two d_k per column
constexpr uint32_t T_XK = 128, T_U = 192;            // X_K^T, U^T
constexpr uint32_t T_D = 128;                        // (K^T U)^T, when X_K and U are done with
constexpr uint32_t T_XQ = 256;
constexpr uint32_t T_RH = 320, T_RL = 352;           // R^T, then (eta U)^T
constexpr uint32_t T_UB = 384;                       // U^T rounded once, for O
constexpr uint32_t T_O = 416;

struct Args {
    Seqs seqs;
    const uint8_t* rec;
    const float* h0;
    float* hT;
    __nv_bfloat16* o;
    int HK, HV;
    float scale;
    uint64_t wait_ns;
};

}  // namespace fw

__global__ void __launch_bounds__(fw::NT, 1)
forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ fw::Args p)
{
    using namespace fw;
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[N_BAR];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.x % p.HV, n = blockIdx.x / p.HV;
    const int hk = hv / (p.HV / p.HK);
    int begin, end;
    seq_range(p.seqs, n, begin, end);
    const int chunks = (end - begin + C - 1) / C;
    const int row = state_row(p.seqs, n);
    const int64_t slot0 = (int64_t)(begin / C) + n;
    auto bar = [&](int b) { return smem_u32(&bars[b]); };

    if (tid == 0) {
        for (int b = 0; b < N_BAR; ++b) {
            const int count = b >= B_EMPTY && b < B_EMPTY + 2 ? N_CHAIN + N_OUT
                            : b == B_S0 || b == B_S1 || b == B_R || b == B_U ? N_CHAIN : b == B_OFREE ? N_OUT : 1;
            mbar_init(bar(b), count);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == W_MMA) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    const Waits wait = {&s_abort, &g_fwd_status, p.wait_ns};

    if (warp < N_CHAIN) {
        const int sp = warp & 3, half = warp >> 2, j = 32 * sp + lane;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
        float S[2][32];                              // S[b][i]: d_k = 64 b + 32 half + i
        const float* h = p.h0 && row >= 0 ? p.h0 + ((int64_t)row * p.HV + hv) * D * D + j : nullptr;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 32; ++i) S[b][i] = h ? h[(int64_t)(64 * b + 32 * half + i) * D] : 0.f;
        auto put = [&](uint32_t hi_col, uint32_t lo_col, const float (&x)[32]) {
            float hi[16], lo[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) split_bf16(x[2 * i], x[2 * i + 1], hi[i], lo[i]);
            tmem_st16(t + hi_col + 16 * half, hi);
            tmem_st16(t + lo_col + 16 * half, lo);
        };
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        auto give_state = [&](int b) {
            put(T_SH + 32 * b, T_SL + 32 * b, S[b]);
            wait_st();
            fence_before_sync();
            arrive(B_S0 + b);
        };
        if (chunks > 0) {
            give_state(0);
            give_state(1);
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const uint8_t* st = sm + s * STAGE;
            const float* gam = reinterpret_cast<const float*>(st + S_REC + REC_GAM) + 32 * half;
            const float* eta = reinterpret_cast<const float*>(st + S_REC + REC_ETA) + 32 * half;
            const float* bet = reinterpret_cast<const float*>(st + S_REC + REC_BETA) + 32 * half;
            const __nv_bfloat16* V = reinterpret_cast<const __nv_bfloat16*>(st + S_V) + 32 * half * D + j;
            wait(bar(B_FULL + s), (c >> 1) & 1);
            wait(bar(B_READY + s), (c >> 1) & 1);
            const float last = *reinterpret_cast<const float*>(st + S_REC + REC_LAST);
            float x[32];
            wait(bar(B_MX), c & 1);
            fence_after_sync();
            tmem_ld32(t + T_XK + 32 * half, x);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(gam + i), b4 = *reinterpret_cast<const float4*>(bet + i);
                x[i] = b4.x * fmaf(-g4.x, x[i], to_f32(V[(i + 0) * D]));
                x[i + 1] = b4.y * fmaf(-g4.y, x[i + 1], to_f32(V[(i + 1) * D]));
                x[i + 2] = b4.z * fmaf(-g4.z, x[i + 2], to_f32(V[(i + 2) * D]));
                x[i + 3] = b4.w * fmaf(-g4.w, x[i + 3], to_f32(V[(i + 3) * D]));
            }
            put(T_RH, T_RL, x);
            wait_st();
            fence_before_sync();
            arrive(B_R);

            wait(bar(B_MU), c & 1);
            fence_after_sync();
            tmem_ld32(t + T_U + 32 * half, x);
            wait_ld();
            {
                float ub[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) ub[i] = __uint_as_float(pack_bf16(x[2 * i], x[2 * i + 1]));
                tmem_st16(t + T_UB + 16 * half, ub);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 e4 = *reinterpret_cast<const float4*>(eta + i);
                x[i] *= e4.x; x[i + 1] *= e4.y; x[i + 2] *= e4.z; x[i + 3] *= e4.w;
            }
            put(T_RH, T_RL, x);
            wait_st();
            fence_before_sync();
            arrive(B_U);
            arrive(B_EMPTY + s);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                wait(bar(B_MD0 + b), c & 1);
                fence_after_sync();
                tmem_ld32(t + T_D + 64 * b + 32 * half, x);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) S[b][i] = fmaf(last, S[b][i], x[i]);
                if (c + 1 < chunks) give_state(b);
            }
        }
        if (p.hT && row >= 0) {
            float* hT = p.hT + ((int64_t)row * p.HV + hv) * D * D + j;
            const bool bad = s_abort != 0;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    hT[(int64_t)(64 * b + 32 * half + i) * D] = bad ? __int_as_float(0x7fc00000) : S[b][i];
        }
    } else if (warp < W_MMA) {
        const int sp = warp & 3, j = 32 * sp + lane, ot = tid - 32 * N_CHAIN;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
        __nv_bfloat16* so = reinterpret_cast<__nv_bfloat16*>(sm + OST);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const uint8_t* st = sm + s * STAGE;
            const float* gam = reinterpret_cast<const float*>(st + S_REC + REC_GAM);
            const int t0 = begin + c * C, nv = min(C, end - t0);
            wait(bar(B_FULL + s), (c >> 1) & 1);
            wait(bar(B_MO), c & 1);
            fence_after_sync();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x[32], y[32];
                tmem_ld32(t + T_XQ + 32 * q, x);
                tmem_ld32(t + T_O + 32 * q, y);
                wait_ld();
                if (q == 1) {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_OFREE));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    so[(32 * q + i) * D + j] = __float2bfloat16_rn(fmaf(p.scale * gam[32 * q + i], x[i], y[i]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_EMPTY + s));
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int e = 0; e < C * D / 8 / 128; ++e) {
                const int i = ot + 128 * e, r = i / (D / 8), c8 = i % (D / 8);
                if (r < nv)
                    *reinterpret_cast<uint4*>(p.o + ((int64_t)(t0 + r) * p.HV + hv) * D + 8 * c8) =
                        *reinterpret_cast<const uint4*>(so + r * D + 8 * c8);
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
        }
    } else if (warp == W_MMA) {
        const uint32_t id_n64 = idesc_bf16(128, 64), id_d = idesc_bf16(128, 64, false, true);
        uint32_t issued = 0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            uint8_t* st = sm + s * STAGE;
            const uint32_t base = smem_u32(st), rec = base + S_REC;
            const int nv = min(C, end - (begin + c * C));
            auto ok = [&](int b, uint32_t parity) {   // every lane sees the same outcome
                const bool w = wait(bar(b), parity);
                return __all_sync(0xffffffffu, w) != 0;
            };
            bool go = ok(B_FULL + s, (c >> 1) & 1);
            if (nv < C) {      // rows behind the sequence count as zero, whatever they hold
                for (int e = lane; e < (C - nv) * 4 * 8; e += 32) {
                    const int piece = e & 7, box = (e >> 3) & 3, r = nv + (e >> 5);
                    *reinterpret_cast<uint4*>(st + box * 8192 + r * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                for (int e = lane; e < (C - nv) * 16; e += 32)
                    *reinterpret_cast<uint4*>(st + S_V + nv * D * 2 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_smem_to_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_READY + s));
            // (x S)^T for the K rows (box 0) or the Q rows (box 1): d_k steps [k0, k1)
            auto state_product = [&](uint32_t d, uint32_t a, int box, int k0, int k1, bool first) {
#pragma unroll
                for (int ks = k0; ks < k1; ++ks)
                    mma_f16_ts_w(tm + d, tm + a + 8 * ks,
                                 sdesc_sw128(base + (2 * (ks / 4) + box) * 8192) + (uint64_t)(2 * (ks % 4)), id_n64,
                                 first && ks == k0 ? 0u : 1u);
            };
            go = go && ok(B_S0, c & 1);
            fence_after_sync();
            if (go) {
                state_product(T_XK, T_SH, 0, 0, 4, true);
                state_product(T_XK, T_SL, 0, 0, 4, false);
            }
            go = go && ok(B_S1, c & 1);
            fence_after_sync();
            if (go) {
                state_product(T_XK, T_SH, 0, 4, 8, false);
                state_product(T_XK, T_SL, 0, 4, 8, false);
                mma_commit_w(bar(B_MX));
            }
            if (c > 0) go = go && ok(B_OFREE, (c - 1) & 1);
            fence_after_sync();
            if (go) state_product(T_XQ, T_SH, 1, 0, 8, true);
            // U^T = R^T X^T (K = tokens): R_hi X_hi + R_lo X_hi + R_hi X_lo
            auto token_product = [&](uint32_t d, uint32_t a, uint32_t b, bool first) {
                const uint64_t bd = sdesc(b, 128, 1024);
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
                    mma_f16_ts_w(tm + d, tm + a + 8 * ks, bd + (uint64_t)(16 * ks), id_n64, first && ks == 0 ? 0u : 1u);
            };
            go = go && ok(B_R, c & 1);
            fence_after_sync();
            if (go) {
                token_product(T_U, T_RH, rec + REC_XH, true);
                token_product(T_U, T_RL, rec + REC_XH, false);
                token_product(T_U, T_RH, rec + REC_XL, false);
                mma_commit_w(bar(B_MU));
            }
            go = go && ok(B_U, c & 1);
            fence_after_sync();
            if (go) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {         // (K^T U)^T, 64 values of d_k each
                    const uint64_t kd = sdesc_sw128(base + 2 * b * 8192);
#pragma unroll
                    for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                        for (int ks = 0; ks < C / 16; ++ks)
                            mma_f16_ts_w(tm + T_D + 64 * b, tm + (hl ? T_RL : T_RH) + 8 * ks, kd + (uint64_t)(128 * ks),
                                         id_d, hl == 0 && ks == 0 ? 0u : 1u);
                    mma_commit_w(bar(B_MD0 + b));
                }
                token_product(T_O, T_UB, rec + REC_P, true);
                mma_commit_w(bar(B_MO));
            }
            issued = c + 1;
            if (!go) break;
        }
        if (issued > 0) {                             // what was issued ends before its memory goes
            mma_commit_w(bar(B_DRAIN));
            mbar_wait(bar(B_DRAIN), 0, DRAIN_NS);
        }
    } else {
        const uint32_t bytes = 4 * 8192 + C * D * 2 + REC_BYTES;
        int loaded = 0;
        if (lane == 0) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int s = c & 1;
                if (c >= 2 && !wait(bar(B_EMPTY + s), ((c >> 1) - 1) & 1)) break;
                if (*(volatile int*)&s_abort) break;
                const uint32_t base = smem_u32(sm + s * STAGE), full = bar(B_FULL + s);
                const int y = begin + c * C;
                mbar_arrive_expect_tx(full, bytes);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tma_load_2d(base + 2 * b * 8192, &mk, hk * D + 64 * b, y, full);
                    tma_load_2d(base + (2 * b + 1) * 8192, &mq, hk * D + 64 * b, y, full);
                }
                tma_load_2d(base + S_V, &mv, hv * D, y, full);
                bulk_load(base + S_REC, p.rec + ((slot0 + c) * p.HV + hv) * REC_BYTES, REC_BYTES, full);
                loaded = c + 1;
            }
            for (int c = max(0, loaded - 2); c < loaded; ++c)          // everything loaded has landed before the end
                mbar_wait(bar(B_FULL + (c & 1)), (c >> 1) & 1, DRAIN_NS);
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    if (warp == W_MMA) {
        fence_after_sync();
        tmem_dealloc(tm, 512);
    }
    if (s_abort) {             // a wait expired: no partial result passes for a real one
        const __nv_bfloat16 nan = __float2bfloat16_rn(__int_as_float(0x7fc00000));
        for (int64_t e = tid; e < (int64_t)(end - begin) * D; e += NT)
            p.o[((int64_t)(begin + e / D) * p.HV + hv) * D + e % D] = nan;
        if (p.hT && row >= 0)
            for (int e = tid; e < D * D; e += NT) p.hT[((int64_t)row * p.HV + hv) * D * D + e] = __int_as_float(0x7fc00000);
    }
}

static DeviceFlags g_fwd_attr_done;

}  // namespace gdn

cudaError_t gdn_forward_launch(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* h0, void* o, float* hT, const int* cu, const int* slots, int n_slots,
                               float scale, int N, int T, int HK, int HV, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, bool gate_f32, cudaStream_t stream)
{
    using namespace gdn;
    fw::Args a = {};
    a.seqs.cu = cu;
    a.seqs.slots = slots;
    a.seqs.n_seq = N;
    a.seqs.n_slots = slots ? n_slots : N;
    a.seqs.len = T;
    a.seqs.tokens = cu ? T : (int64_t)N * T;
    a.h0 = h0;
    a.hT = hT;
    a.o = (__nv_bfloat16*)o;
    a.HK = HK;
    a.HV = HV;
    a.scale = scale;
    a.wait_ns = bounded_wait_limit_ns();
    cudaError_t e = once_per_device(g_fwd_attr_done, [](int) {
        return cudaFuncSetAttribute(forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fw::SMEM);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap mq = {}, mk = {}, mv = {};
    uint8_t* rec = nullptr;
    const int64_t tokens = a.seqs.tokens;
    if (tokens > 0) {
        if (!make_token_map(&mq, q, tokens, (int64_t)HK * D, q_stride, 64) ||
            !make_token_map(&mk, k, tokens, (int64_t)HK * D, k_stride, 64) ||
            !make_token_map(&mv, v, tokens, (int64_t)HV * D, v_stride, D))
            return cudaErrorInvalidValue;
        keep_pool_memory();
        e = cudaMallocAsync(reinterpret_cast<void**>(&rec), (size_t)slot_count(a.seqs) * HV * REC_BYTES, stream);
        if (e != cudaSuccess) return e;
        e = prep_launch(mq, mk, g, beta, a.seqs, rec, scale, HK, HV, gate_f32, stream);
    }
    a.rec = rec;
    if (e == cudaSuccess) {
        forward_kernel<<<(unsigned)((int64_t)N * HV), fw::NT, fw::SMEM, stream>>>(mq, mk, mv, a);
        note_launches(1);
        e = cudaGetLastError();
    }
    if (rec) {
        const cudaError_t ef = cudaFreeAsync(rec, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

int gdn_forward_status(cudaStream_t stream)
{
    int st = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&st, gdn::g_fwd_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(gdn::g_fwd_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return KDA_ERR_CUDA;
    return st;
}

}  // namespace kda
