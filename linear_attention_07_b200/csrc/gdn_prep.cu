// Gated delta rule, one decay per head: the part of a chunk that needs no
// state, for every chunk at once (one CTA per value head and chunk slot):
// X = (I + A)^-1, P and the gate factors (gdn_chunk.cuh).
//
// K K^T and Q K^T are one tensor-core product of M = 128 ([K; Q]), N = 64,
// K = 128 from the TMA-staged rows.  The running sums of g and their
// differences are taken in 64 bits: a sum over 64 tokens reaches thousands
// when tokens reset the state, and fp32 would then lose the decay between
// neighbours.  X comes from forward substitution in fp32: the four 16 x 16
// diagonal blocks by columns, then X10 = -X11 A10 X00 for blocks of 16 and of
// 32 (a row-by-row substitution of 64 rows would be one long chain, powers of
// A would lose digits when keys repeat).
#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

__device__ int g_prep_status;

namespace prep {
constexpr int NT = 256;
constexpr int LD = C + 1;
// K and Q rows (two boxes of 64 channels each: K0 Q0 K1 Q1), then A, X and
// the product between the blocks in their place
constexpr uint32_t KQ_BYTES = 2 * C * D * 2;
constexpr uint32_t A_OFF = 0;
constexpr uint32_t X_OFF = A_OFF + C * LD * 4;
constexpr uint32_t Y_OFF = X_OFF + C * LD * 4;
constexpr uint32_t BODY = Y_OFF + 32 * 33 * 4;
static_assert(BODY >= KQ_BYTES, "one body for both");
constexpr uint32_t SMEM = BODY + 1024;               // room to align the tiles to 1024 bytes
}  // namespace prep

__global__ void __launch_bounds__(prep::NT, 4)
prep_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const void* __restrict__ g,
            const void* __restrict__ beta, const Seqs seqs, uint8_t* __restrict__ rec_all, float scale, int HK, int HV,
            bool gate_f32, uint64_t wait_ns)
{
    using namespace prep;
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ double sG[C];
    __shared__ float sB[C];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x / HV;             // heads next to one another: they share K and Q in L2
    const int hv = (int)(blockIdx.x % HV), hk = hv / (HV / HK);
    int n, chunk, begin, end;
    if (!slot_chunk(seqs, slot, n, chunk, begin, end)) return;
    const int t0 = begin + chunk * C, nv = min(C, end - t0);
    uint8_t* rec = rec_all + (slot * HV + hv) * REC_BYTES;
    const uint32_t tile = smem_u32(sm), full = smem_u32(&bars[0]), done = smem_u32(&bars[1]);

    if (tid == 0) {
        mbar_init(full, 1);
        mbar_init(done, 1);
        fence_mbar_init();
        s_abort = 0;
        mbar_arrive_expect_tx(full, KQ_BYTES);
        for (int b = 0; b < 2; ++b) {
            tma_load_2d(tile + b * 16384, &mk, hk * D + 64 * b, t0, full);
            tma_load_2d(tile + b * 16384 + 8192, &mq, hk * D + 64 * b, t0, full);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), 64);
        tmem_relinquish();
    }
    if (warp == 2) {                                  // running sum of g in 64 bits, two tokens per lane
        double x[2];
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const int64_t at = (int64_t)(t0 + r) * HV + hv;
            x[i] = r < nv ? (double)cut_decay(gate(g, at, gate_f32)) : 0.0;
            sB[r] = r < nv ? gate(beta, at, gate_f32) : 0.f;
        }
        const double both = x[0] + x[1];
        double sum = both;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += y;
        }
        sG[2 * lane] = sum - both + x[0];
        sG[2 * lane + 1] = sum;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    const Waits wait = {&s_abort, &g_prep_status, wait_ns};
    if (warp == 0) {
        const bool here = wait(full, 0);
        if (!here) mbar_wait(full, 0, DRAIN_NS);      // the loads land before their space is used again
        if (nv < C) {                                 // rows behind the sequence: whatever is there counts as zero
            for (int e = lane; e < (C - nv) * 4 * 8; e += 32) {
                const int piece = e & 7, row = nv + (e >> 5), box = (e >> 3) & 3;
                *reinterpret_cast<uint4*>(sm + box * 8192 + row * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_smem_to_async();
            __syncwarp();
        }
        if (__all_sync(0xffffffffu, here)) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t d = sdesc_sw128(tile + (ks / 4) * 16384) + (uint64_t)(2 * (ks % 4));
                mma_f16_ss_w(tm, d, d, idesc_bf16(128, C), ks > 0 ? 1u : 0u);
            }
            mma_commit_w(done);
            if (!wait(done, 0)) mbar_wait(done, 0, DRAIN_NS);
        }
    }
    __syncthreads();
    fence_after_sync();
    float* sA = reinterpret_cast<float*>(sm + A_OFF);
    float* sX = reinterpret_cast<float*>(sm + X_OFF);
    float* sY = reinterpret_cast<float*>(sm + Y_OFF);
    {   // thread: one row of [K K^T; Q K^T], 32 columns
        float x[32];
        const int sp = warp & 3, col = 32 * (warp >> 2), r = (sp & 1) * 32 + lane;
        tmem_ld32(tm + ((uint32_t)(32 * sp) << 16) + col, x);
        wait_ld();
        const double Gr = sG[r];
        if (sp < 2) {
            const float b = sB[r];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int c = col + i;
                sA[r * LD + c] = c < r ? b * expf((float)(Gr - sG[c])) * x[i] : 0.f;
            }
        } else {
            uint8_t* dst = rec + REC_P + (r / 8) * 1024 + (r % 8) * 16;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 8 * p + 2 * e, c = col + i;
                    const float lo = c <= r ? scale * expf((float)(Gr - sG[c])) * x[i] : 0.f;
                    const float hi = c + 1 <= r ? scale * expf((float)(Gr - sG[c + 1])) * x[i + 1] : 0.f;
                    w[e] = pack_bf16(lo, hi);
                }
                *reinterpret_cast<uint4*>(dst + (col / 8 + p) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (tid < C) {
        const double Gl = sG[C - 1], Gr = sG[tid];
        reinterpret_cast<float*>(rec + REC_GAM)[tid] = expf((float)Gr);
        reinterpret_cast<float*>(rec + REC_ETA)[tid] = expf((float)(Gl - Gr));
        reinterpret_cast<float*>(rec + REC_BETA)[tid] = sB[tid];
        if (tid == 0) *reinterpret_cast<float*>(rec + REC_LAST) = expf((float)Gl);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tm, 64);
    }
    // X: the 16 x 16 diagonal blocks, one column per thread
    if (tid < C) {
        const int b = tid / 16, j = tid % 16;
        const float* a = sA + (16 * b) * LD + 16 * b;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < r; ++i) s[i & 3] = fmaf(a[r * LD + i], x[i], s[i & 3]);
            x[r] = r == j ? 1.f : r > j ? -((s[0] + s[1]) + (s[2] + s[3])) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) sX[(16 * b + r) * LD + 16 * b + j] = x[r];
    }
    __syncthreads();
    // blocks of S next to one another: X10 = -X11 (A10 X00), S = 16 then 32;
    // the block of S x S results is spread over the threads of its pair
    auto join = [&](auto size) {
        constexpr int S = decltype(size)::value;
        constexpr int PAIRS = C / (2 * S), TP = NT / PAIRS, PER = S * S / TP;      // results per thread
        const int pair = tid / TP, t = tid % TP;
        const int col = t % S, row0 = (t / S) * PER;
        const int base = 2 * S * pair;
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 8
        for (int k = 0; k < S; ++k) {                 // Y = A10 X00
            const float x = k >= col ? sX[(base + k) * LD + base + col] : 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = fmaf(sA[(base + S + row0 + i) * LD + base + k], x, acc[i]);
        }
        float* y = sY + pair * (S * (S + 1));
#pragma unroll
        for (int i = 0; i < PER; ++i) y[(row0 + i) * (S + 1) + col] = acc[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 8
        for (int k = 0; k < S; ++k) {
            const float v = y[k * (S + 1) + col];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                acc[i] = fmaf(k <= row0 + i ? sX[(base + S + row0 + i) * LD + base + S + k] : 0.f, v, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) sX[(base + S + row0 + i) * LD + base + col] = -acc[i];
        __syncthreads();
    };
    join(std::integral_constant<int, 16>());
    join(std::integral_constant<int, 32>());
    {   // X as two bf16 numbers, in the operand layout: one row and 16 columns per thread
        const int r = tid % C, c0 = (tid / C) * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = c0 + 8 * p + 2 * e;
                // above the diagonal blocks sX was never written
                const float a = c <= r ? sX[r * LD + c] : 0.f, b = c + 1 <= r ? sX[r * LD + c + 1] : 0.f;
                float h, l;
                split_bf16(a, b, h, l);
                hi[e] = __float_as_uint(h);
                lo[e] = __float_as_uint(l);
            }
            const uint32_t at = (r / 8) * 1024 + (c0 / 8 + p) * 128 + (r % 8) * 16;
            *reinterpret_cast<uint4*>(rec + REC_XH + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(rec + REC_XL + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if (s_abort && tid < C) reinterpret_cast<float*>(rec + REC_GAM)[tid] = __int_as_float(0x7fc00000);
}

bool make_token_map(CUtensorMap* map, const void* base, int64_t tokens, int64_t cols, int64_t stride, int box_cols)
{
    typedef CUresult (*encode_fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const encode_fn encode = []() -> encode_fn {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return (encode_fn)fn;
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)tokens};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)C};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static DeviceFlags g_prep_attr_done;

cudaError_t prep_launch(const CUtensorMap& mq, const CUtensorMap& mk, const void* g, const void* beta, const Seqs& seqs,
                        uint8_t* rec, float scale, int HK, int HV, bool gate_f32, cudaStream_t stream)
{
    const cudaError_t e = once_per_device(g_prep_attr_done, [](int) {
        return cudaFuncSetAttribute(prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep::SMEM);
    });
    if (e != cudaSuccess) return e;
    prep_kernel<<<(unsigned)(slot_count(seqs) * HV), prep::NT, prep::SMEM, stream>>>(
        mq, mk, g, beta, seqs, rec, scale, HK, HV, gate_f32, bounded_wait_limit_ns());
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace gdn

int gdn_prep_status(cudaStream_t stream)
{
    int st = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&st, gdn::g_prep_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(gdn::g_prep_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return KDA_ERR_CUDA;
    return st;
}

}  // namespace kda
