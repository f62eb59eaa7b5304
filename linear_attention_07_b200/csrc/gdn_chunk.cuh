// Chunked form of the gated delta rule with one decay per head (d_k = d_v =
// 128): what the forward and the backward share.
//
// A chunk is C = 64 tokens.  With G_r the running sum of g inside the chunk,
// gam = exp(G), eta_r = exp(G_last - G_r), D_ri = exp(G_r - G_i):
//     A  = strict_lower(beta_r D_ri k_r . k_i),   X = (I + A)^-1
//     T  = X diag(beta),   W = T diag(gam) K,   U = T V - W S0
//     O  = scale gam Q S0 + P U,  P = scale lower(D_ri q_r . k_i)
//     S1 = gam_last S0 + K^T (eta U)
// One decay per head is one factor per token pair or token: K, Q and V enter
// every product as they are in memory, exact in bf16.  Everything else (the
// state, T, W, P, U) is fp32 and enters as the sum of two bf16 numbers (16
// significant bits; the products hi hi, hi lo and lo hi are kept), so the
// state carries about fp32 accuracy through bf16 tensor-core products (and so
// do the outputs, whose sums over U cancel where keys repeat).
//
// Sequences are cut into chunks at their own begins.  Chunk c of sequence n,
// which begins at token a, has the workspace slot a / 64 + n + c: a sequence
// of L tokens from a needs ceil(L / 64) <= (a + L) / 64 - a / 64 + 1 of them,
// so slots never collide, and no prefix sum over the lengths is needed.
#pragma once
#include <cuda.h>

#include "gdn_common.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace gdn {

constexpr int C = 64;
constexpr int D = 128;

// What the prep kernel leaves per (slot, value head), in bytes.  W is stored
// as a TMA box with the 128-byte swizzle would be (two boxes of 64 channels),
// negated; T and P as the no-swizzle operand layout wants them: element (r, i)
// at (r / 8) * 1024 + (i / 8) * 128 + (r % 8) * 16 + (i % 8) * 2.
constexpr uint32_t BOX = C * 64 * 2;
constexpr uint32_t REC_WH = 0;                       // -W, upper 8 bits   [2][64 x 64] bf16
constexpr uint32_t REC_WL = REC_WH + 2 * BOX;        // and the rest
constexpr uint32_t REC_TH = REC_WL + 2 * BOX;        // T, likewise   [64 x 64]
constexpr uint32_t REC_TL = REC_TH + BOX;
constexpr uint32_t REC_NGAM = REC_TL + BOX;          // -gam_r   [64] fp32
constexpr uint32_t REC_ETA = REC_NGAM + C * 4;       // eta_r (forward: times ETA_SCALE, and P divided by it)
constexpr uint32_t REC_GQ = REC_ETA + C * 4;         // scale gam_r
constexpr uint32_t REC_BETA = REC_GQ + C * 4;        // beta_r (0 behind the sequence)
constexpr uint32_t REC_PH = REC_BETA + C * 4;        // P, likewise
constexpr uint32_t REC_PL = REC_PH + BOX;
constexpr uint32_t REC_BYTES = REC_PL + BOX;
constexpr uint32_t REC_W_BYTES = REC_PH;             // W, T and the gates; P is needed at another time
constexpr uint32_t GATE_BYTES = REC_PH - REC_NGAM;
constexpr uint32_t P_BYTES = REC_BYTES - REC_PH;
static_assert(REC_BYTES == 66560 && REC_W_BYTES % 1024 == 0, "record");

// The forward multiplies P with eta U, which it has as an operand anyway, so
// there P's columns are divided by eta.  eta is held above 2^-100 for that: a
// token whose write has decayed further leaves 2^-100 of it in the state.  So
// that eta U stays in bf16's range with such an eta too (values below 1e-6 lost
// digits in chunks that decay far), the forward's eta is 2^50 times as large and
// P / eta that much smaller; K^T (eta U) is divided by it.  U may be between 2^-60
// (where both planes of eta U are still normal numbers) and 2^77.
constexpr float ETA_FLOOR_LOG2 = -100.f;
constexpr float ETA_SCALE = 0x1p50f, ETA_UNSCALE = 0x1p-50f;

__host__ __device__ inline int64_t slot_count(const Seqs& s) { return s.tokens / C + s.n_seq; }

__device__ __forceinline__ int64_t first_slot(const Seqs& s, int n)
{
    int a, b;
    seq_range(s, n, a, b);
    return (int64_t)(a / C) + n;
}

// Chunk of a slot in sequence n; false if it has none there.
__device__ __forceinline__ bool chunk_of(int64_t slot, int n, int begin, int end, int& chunk)
{
    const int64_t c = slot - ((int64_t)(begin / C) + n);
    chunk = (int)c;
    return c >= 0 && c * C < end - begin;
}

// The last sequence n with first_slot(n) <= slot, or 0; by whole warps.  32
// sequences are looked at at once, a trip to memory for each factor of 32 in
// their number.
__device__ __forceinline__ int find_sequence(const Seqs& s, int64_t slot)
{
    int lo = 0;
    for (int count = s.n_seq; count > 1;) {
        const int step = (count + 31) / 32, at = (int)(threadIdx.x & 31) * step;
        const bool before = at < count && first_slot(s, lo + at) <= slot;
        const int last = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0) * step;
        lo += last;
        count = min(step, count - last);
    }
    return lo;
}

// Sequence and chunk of a slot; false if the slot belongs to none.  By whole warps.
__device__ __forceinline__ bool slot_chunk(const Seqs& s, int64_t slot, int& n, int& chunk, int& begin, int& end)
{
    n = find_sequence(s, slot);
    seq_range(s, n, begin, end);
    return chunk_of(slot, n, begin, end, chunk);
}

__device__ __forceinline__ int chunk_count(const Seqs& s, int n)
{
    int begin, end;
    seq_range(s, n, begin, end);
    return (end - begin + C - 1) / C;
}

// The l-th sequence of min_chunks chunks or more, or -1; by whole warps.
__device__ __forceinline__ int long_sequence(const Seqs& s, int min_chunks, int l)
{
    for (int first = 0; first < s.n_seq; first += 32) {
        const int n = first + (int)(threadIdx.x & 31);
        uint32_t m = __ballot_sync(0xffffffffu, n < s.n_seq && chunk_count(s, n) >= min_chunks);
        const int count = __popc(m);
        if (l < count) {
            for (; l > 0; --l) m &= m - 1;
            return first + __ffs(m) - 1;
        }
        l -= count;
    }
    return -1;
}

// Long sequences of few heads run in segments at the same time: from MIN_CHUNKS
// chunks on.  The start states follow from the states that the segments reach
// from zero (N) and their transitions (M), start_{k+1} = M_k start_k + N_k with
// start_0 = first; before_last is what the last step gives.  All [n_long]
// [between][HV][D][D] fp32, first and before_last [n_long][HV][D][D].
constexpr int MIN_CHUNKS = 32;
struct JoinSet {
    const float *M, *N, *first;
    float *start, *before_last;
};
struct JoinArgs {
    Seqs seqs;
    JoinSet set[2];
    int HV, between, min_chunks;
};
cudaError_t join_launch(const JoinArgs& a, int sets, int64_t heads, cudaStream_t stream);

// Descriptor of a 128-byte-swizzled tile of 128-byte rows (as a TMA box of 64
// bf16 columns leaves it, 1024-byte aligned): groups of 8 rows are 1024 bytes
// apart.  K-major (the row is a vector along K): 16 elements of K further are
// 32 bytes further.  MN-major (the row is a vector along M or N): 16 rows
// further along K are 2048 bytes further.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(1024 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor, kind::f16 with bf16 A and B and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn = false, bool b_mn = false)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Four K steps of one product by a converged warp (one elected lane issues).
// A from tensor memory (16 columns per step: 8 of the upper and 8 of the lower
// plane, written by one store) or shared memory, B from shared memory, its steps
// in descriptor units (16 bytes), which change a descriptor's lower word only.
// Issuing is close to what bounds the chains, so it is kept to few instructions:
// warp-uniform operands, one election for four.
template <uint32_t B_STEP>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t more)
{
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 l, h;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|p, 0xffffffff;\n\tsetp.ne.b32 q, %7, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 {l, h}, %5;\n\t"
        "add.u32 l, l, %8;\n\tmov.b64 b1, {l, h};\n\tadd.u32 l, l, %8;\n\tmov.b64 b2, {l, h};\n\t"
        "add.u32 l, l, %8;\n\tmov.b64 b3, {l, h};\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %6, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], b1, %6, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], b2, %6, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], b3, %6, t;\n\t}\n"
        :: "r"(d), "r"(a), "r"(a + 16), "r"(a + 32), "r"(a + 48), "l"(b), "r"(idesc), "r"(more), "n"(B_STEP) : "memory");
}
template <uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t more)
{
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 l, h, m, g;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|p, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 {l, h}, %2;\n\tmov.b64 {m, g}, %1;\n\t"
        "add.u32 l, l, %6;\n\tmov.b64 b1, {l, h};\n\tadd.u32 l, l, %6;\n\tmov.b64 b2, {l, h};\n\t"
        "add.u32 l, l, %6;\n\tmov.b64 b3, {l, h};\n\t"
        "add.u32 m, m, %5;\n\tmov.b64 a1, {m, g};\n\tadd.u32 m, m, %5;\n\tmov.b64 a2, {m, g};\n\t"
        "add.u32 m, m, %5;\n\tmov.b64 a3, {m, g};\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(more), "n"(A_STEP), "n"(B_STEP) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int x, int y, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar) : "memory");
}
// The same data on its way to L2.
__device__ __forceinline__ void tma_prefetch_2d(const void* map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(mbar) : "memory");
}

// Packed fp32 pairs: one instruction for two values.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// 2^x, below 2^-126 zero.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values as packed bf16 pairs hi and lo with x ~ hi + lo (each
// rounded to nearest: 16 significant bits together).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void split_bf16(float a, float b, float& hi, float& lo)
{
    const uint32_t h = pack_bf16(a, b);
    hi = __uint_as_float(h);
    const float2 r = fma2(make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), make_float2(-1.f, -1.f),
                          make_float2(a, b));         // exact
    lo = __uint_as_float(pack_bf16(r.x, r.y));
}

// 16 values of one lane as two planes of an operand in tensor memory: the upper
// bf16 pairs in columns [0, 8), the lower in [8, 16).
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const float (&x)[16], float (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) split_bf16(x[2 * i], x[2 * i + 1], w[i], w[8 + i]);
    tc::tmem_st16(taddr, w);
}

// A bounded wait of one role.  All lanes of a warp poll with try_wait, which
// suspends them: polling by one lane, or with test_wait, made the forward's
// chain 1.4 to 2.5 times slower.  Once any wait of the CTA has expired, every
// later one returns at once: the roles run to their ends without issuing.
struct Waits {
    volatile int* abort;
    int* status;
    uint64_t ns;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        if (ns != 0 && tc::mbar_try_wait(bar, parity)) return true;
        return slow(bar, parity);
    }
    // The same without a call: kernels that move registers between their warps may not make one.
    __device__ __forceinline__ bool inlined(uint32_t bar, uint32_t parity) const
    {
        return (ns != 0 && tc::mbar_try_wait(bar, parity)) || expire(bar, parity);
    }
    __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity) const { return expire(bar, parity); }
    __device__ __forceinline__ bool expire(uint32_t bar, uint32_t parity) const
    {
        if (ns == 0 && tc::mbar_test_wait(bar, parity)) return true;
        // by the SM's clock (2 cycles per ns at most): reading the global timer takes about as long as its 1 us step,
        // and every wait of the chain would end that much later
        const long long t0 = clock64();
        while (ns != 0 && !*abort) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)              // each try may itself block for a while
                if (tc::mbar_try_wait(bar, parity)) return true;
            if ((uint64_t)(clock64() - t0) > 2 * ns) break;
        }
        *abort = 1;
        atomicExch(status, (int)KDA_ERR_TIMEOUT);
        return false;
    }
};
constexpr uint64_t DRAIN_NS = 20000000ull;           // after an expired wait: 20 ms for what is in flight

// Bulk store of shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" :: "l"(dst), "r"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_store_2d(const void* map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(src) : "memory");
}

// Host: bf16 [tokens][cols] with a row stride in elements; boxes of 64 rows by
// 64 columns with the 128-byte swizzle (loads), or of 32 rows by 128 columns
// without (stores).
bool make_token_map(CUtensorMap* map, const void* base, int64_t tokens, int64_t cols, int64_t stride, bool store = false);

// offsets: where the sequences' offsets go in order ([n_seq + 1]), which the kernels behind the prep take for cu; null
// without cu.  order_launch puts those of 32 sequences or more there and into seqs (one launch), prep_launch fewer.
cudaError_t order_launch(Seqs& seqs, int* offsets, cudaStream_t stream);
cudaError_t prep_launch(const CUtensorMap& mq, const CUtensorMap& mk, const void* g, const void* beta, const Seqs& seqs,
                        int* offsets, uint8_t* rec, float scale, int HK, int HV, int f32_gates, bool backward, cudaStream_t stream);

}  // namespace gdn
}  // namespace kda
