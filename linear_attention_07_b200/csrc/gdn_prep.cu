// Gated delta rule, one decay per head: the part of a chunk that needs no
// state, for every chunk at once (one CTA per value head and chunk slot):
// T = (I + A)^-1 diag(beta), W, P and the gate factors (gdn_chunk.cuh).
//
// K K^T and Q K^T are one tensor-core product of M = 128 ([K; Q]), N = 64,
// K = 128 from the TMA-staged rows.  The running sums of g are taken in 64
// bits and kept as two fp32 numbers: a sum over 64 tokens reaches thousands
// when tokens reset the state, and fp32 would then lose the decay between
// neighbours.  X comes from forward substitution (powers of A would lose
// digits when keys repeat): the 16 x 16 diagonal blocks in fp32, then X10 =
// -X11 (A10 X00) for blocks of 16 and of 32 as small tensor-core products of
// fp32 accuracy (three tf32 products each): with fp32 FMAs those read shared
// memory once per multiply, which bound the kernel.
//
// 85 us for 8192 tokens x 32 heads, 611 us for 4 x 16384 x 32 (a record of
// 66,560 bytes each: 3.7 TB/s).  Bound by a CTA's 15 us of dependent phases
// against six CTAs per SM: issue slots are half full, shared memory's port as
// much, no phase above 15 % of the time.  Four CTAs of 52 KB took 818 us; with
// 2-byte stores of W, a substitution on all four warps and the gates in front
// of the products it was 708 us.
#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

__device__ int g_prep_status;

namespace prep {
constexpr int NT = 128;
// K and Q rows (boxes of 64 channels: K0 Q0 K1 Q1); then the lower triangle of
// A, which becomes X in place, where Q was: three blocks of 32 x 32; then
// -T diag(gam) as two planes there; at the end W's two planes over all of it.
// No more than that, and 64 columns of tensor memory: six CTAs of an SM hide
// one another's latency.
constexpr int BLK = 32 * 32;                         // fp32 values of a block
constexpr uint32_t B00 = BOX, B10 = BOX + 4 * BLK, B11 = 3 * BOX;
constexpr uint32_t SMEM = 4 * BOX + 1024;            // room to align the tiles to 1024 bytes

// Element (r, c) of a block: rows of 32, their groups of four columns permuted
// so that neither rows of a column nor the matrix fragments meet in a bank.
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }
__device__ __forceinline__ int at(int r, int c) { return r * 32 + (((c >> 2) ^ swz(r)) << 2) + (c & 3); }

// 16 columns of row r as pairs of bf16, in the operand layout.
__device__ __forceinline__ void store_split(uint8_t* hi_dst, uint8_t* lo_dst, int r, int col, const float* x)
{
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16(x[8 * p + 2 * e], x[8 * p + 2 * e + 1], hi[e], lo[e]);
        const uint32_t o = (r / 8) * 1024 + (col / 8 + p) * 128 + (r % 8) * 16;
        *reinterpret_cast<float4*>(hi_dst + o) = make_float4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<float4*>(lo_dst + o) = make_float4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// Warps 0 and 1.
__device__ __forceinline__ void front_sync() { asm volatile("bar.sync 1, 64;" ::: "memory"); }

// 16 lanes x 32 columns of tensor memory as matrix fragments: x[4 k ..] are the
// lanes l / 4 (two columns 8 k + 2 (l % 4) ..) and l / 4 + 8 (likewise) of thread l.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, float (&x)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
                   "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
                 : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit values, transposed; thread l has the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, float a, float b, float c, float d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)) : "memory");
}

// fp32 products on the tensor cores: x = hi + lo with 11 significant bits in
// hi, and hi hi + hi lo + lo hi.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo)
{
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// (16 MT x 16 MT at (mr, mc) of block m) times (16 MT x 8 at (xr, xc) of block x).
template <int MT>
__device__ __forceinline__ void block_product(const float* m, int mr, int mc, const float* x, int xr, int xc, int lane,
                                              float (&d)[MT][4])
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k) {
        uint32_t bh[2], bl[2];
        split_tf32(x[at(xr + 8 * k + t, xc + g)], bh[0], bl[0]);
        split_tf32(x[at(xr + 8 * k + t + 4, xc + g)], bh[1], bl[1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = mr + 16 * i + g, c = mc + 8 * k + t;
            uint32_t ah[4], al[4];
            split_tf32(m[at(r, c)], ah[0], al[0]);
            split_tf32(m[at(r, c) + 8 * 32], ah[1], al[1]);
            split_tf32(m[at(r, c + 4)], ah[2], al[2]);
            split_tf32(m[at(r, c + 4) + 8 * 32], ah[3], al[3]);
            mma_tf32(d[i], al, bh);
            mma_tf32(d[i], ah, bl);
            mma_tf32(d[i], ah, bh);
        }
    }
}
template <int MT>
__device__ __forceinline__ void put(float* x, int xr, int xc, int lane, float sign, const float (&d)[MT][4])
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        float* y = x + at(xr + 16 * i + g, xc + 2 * t);
        *reinterpret_cast<float2*>(y) = make_float2(sign * d[i][0], sign * d[i][1]);
        *reinterpret_cast<float2*>(y + 8 * 32) = make_float2(sign * d[i][2], sign * d[i][3]);
    }
}
// Columns [c, c + 8) of X10 = -X11 (A10 X00), in A10's place; all threads take part.
template <int MT>
__device__ __forceinline__ void join(const float* x00, float* a10, int ar, const float* x11, int xc, int c, int lane)
{
    float d[MT][4];
    block_product<MT>(a10, ar, 0, x00, 0, c, lane, d);
    __syncthreads();                                  // every warp has read A10
    put<MT>(a10, ar, c, lane, 1.f, d);
    __syncwarp();
    block_product<MT>(x11, ar, xc, a10, ar, c, lane, d);
    __syncwarp();
    put<MT>(a10, ar, c, lane, -1.f, d);
    __syncthreads();
}

// slot_chunk by the caller's offsets of fewer than 32 sequences, which may go
// back: offset n is the largest up to n.  A lane has each of them, so that they
// are put in order only where they are not.  (For more, order_kernel does it: to
// look at all offsets in every CTA made calls of 100 and 1000 sequences 4 % longer.)
__device__ __forceinline__ bool given_slot_chunk(const Seqs& s, int slot, int& n, int& chunk, int& begin, int& end)
{
    if (s.n_seq == 1) {
        n = 0;
        seq_range(s, 0, begin, end);
    } else {
        const int lane = (int)(threadIdx.x & 31);
        int v = cut_offset(s, lane <= s.n_seq ? s.cu[lane] : 0x7fffffff);
        if (!__all_sync(0xffffffffu, v <= __shfl_down_sync(0xffffffffu, v, 1)))
#pragma unroll 1
            for (int off = 1; off < 32; off <<= 1) v = max(v, __shfl_sync(0xffffffffu, v, max(lane - off, 0)));
        n = max(__popc(__ballot_sync(0xffffffffu, lane < s.n_seq && v / C + lane <= slot)) - 1, 0);
        begin = __shfl_sync(0xffffffffu, v, n);
        end = __shfl_sync(0xffffffffu, v, n + 1);
    }
    return chunk_of(slot, n, begin, end, chunk);
}
}  // namespace prep

// The caller's offsets in order: offset n is the largest of cu[0 .. n], cut to [0, tokens].  One CTA: 3 us up to 1000
// sequences, 14 us for 16000.
constexpr int ORDER_NT = 1024;
__global__ void __launch_bounds__(ORDER_NT) order_kernel(const Seqs s, int* __restrict__ offsets)
{
    __shared__ int most[2][ORDER_NT / 32];            // of each warp; two sets in turn: one barrier a pass
    const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
    int before = 0;
    for (int first = 0, set = 0; first <= s.n_seq; first += ORDER_NT, set ^= 1) {
        const int i = first + (int)threadIdx.x;
        int v = i <= s.n_seq ? cut_offset(s, s.cu[i]) : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) v = max(v, __shfl_sync(0xffffffffu, v, max(lane - off, 0)));
        if (lane == 31) most[set][warp] = v;
        __syncthreads();
        const int w = most[set][lane];
        v = max(v, max(before, __reduce_max_sync(0xffffffffu, lane < warp ? w : 0)));
        if (i <= s.n_seq) offsets[i] = v;
        before = max(before, __reduce_max_sync(0xffffffffu, w));
    }
}

__global__ void __launch_bounds__(prep::NT, 6)
prep_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const void* __restrict__ g,
            const void* __restrict__ beta, const Seqs seqs, int* __restrict__ offsets, uint8_t* __restrict__ rec_all,
            float scale, int HK, int HV, int f32_gates, bool backward, uint64_t wait_ns)
{
    using namespace prep;
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2];
    // the running sum of g in units of log 2, as two fp32 numbers
    __shared__ __align__(16) float sGh[C], sGl[C];
    __shared__ __align__(16) float sCh[C], sCl[C];    // what P's columns are measured from, likewise
    __shared__ __align__(16) float sNG[C];            // -gam
    __shared__ __align__(16) float sB[C];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x / HV;             // heads next to one another: they share K and Q in L2
    const int hv = (int)(blockIdx.x % HV), hk = hv / (HV / HK);
    int n, chunk, begin, end;
    const bool has_tokens = offsets ? given_slot_chunk(seqs, (int)slot, n, chunk, begin, end) : slot_chunk(seqs, slot, n, chunk, begin, end);
    if (offsets && hv == 0 && tid == 0 && slot == begin / C + n) {           // every sequence has this slot, if an empty one
        offsets[n] = begin;
        if (n + 1 == seqs.n_seq) offsets[n + 1] = end;
    }
    if (!has_tokens) return;
    const int t0 = begin + chunk * C, nv = min(C, end - t0);
    uint8_t* rec = rec_all + (slot * HV + hv) * REC_BYTES;
    const uint32_t tile = smem_u32(sm), full = smem_u32(&bars[0]), done = smem_u32(&bars[1]);

    bool issued = false;
    const Waits wait = {&s_abort, &g_prep_status, wait_ns};
    if (warp == 0) {                                  // [K; Q] K^T, while warp 2 has the gates
        if (lane == 0) {
            mbar_init(full, 1);
            mbar_init(done, 1);
            fence_mbar_init();
            s_abort = 0;
            mbar_arrive_expect_tx(full, 4 * BOX);
            for (int b = 0; b < 2; ++b) {
                tma_load_2d(tile + 2 * b * BOX, &mk, hk * D + 64 * b, t0, full);
                tma_load_2d(tile + (2 * b + 1) * BOX, &mq, hk * D + 64 * b, t0, full);
            }
        }
        front_sync();                                 // tensor memory is there
        fence_after_sync();
        const bool here = wait(full, 0);
        if (!here) mbar_wait(full, 0, DRAIN_NS);      // the loads land before their space is used again
        if (nv < C) {                                 // rows behind the sequence: whatever is there counts as zero
            for (int e = lane; e < (C - nv) * 4 * 8; e += 32) {
                const int piece = e & 7, row = nv + (e >> 5), box = (e >> 3) & 3;
                *reinterpret_cast<uint4*>(sm + box * BOX + row * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_smem_to_async();
            __syncwarp();
        }
        if (__all_sync(0xffffffffu, here)) {          // K K^T in lanes 0-63, Q K^T in lanes 64-127
            constexpr uint32_t id = idesc_bf16(128, C);
            const uint32_t d = s_tmem;
            mma4_ss<2, 2>(d, sdesc_sw128(tile), sdesc_sw128(tile), id, 0u);
            mma4_ss<2, 2>(d, sdesc_sw128(tile + 2 * BOX), sdesc_sw128(tile + 2 * BOX), id, 1u);
            mma_commit_w(done);
            if (!wait(done, 0)) mbar_wait(done, 0, DRAIN_NS);
            issued = true;
        }
    } else if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), C);
        tmem_relinquish();
        fence_before_sync();
        front_sync();
    } else if (warp == 2) {                           // running sum of g in 64 bits, two tokens per lane
        const int64_t at = (int64_t)(t0 + 2 * lane) * HV + hv;
        const bool real[2] = {2 * lane < nv, 2 * lane + 1 < nv};
        float gi[2] = {0.f, 0.f}, bi[2] = {0.f, 0.f};
        auto load = [&](bool g_f32, bool beta_f32) {  // all loads at once, whatever the types
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (real[i]) gi[i] = gate(g, at + i * HV, g_f32), bi[i] = gate(beta, at + i * HV, beta_f32);
        };
        if (f32_gates == 0) load(false, false);
        else if (f32_gates == G_F32) load(true, false);
        else load(true, true);
        const double x0 = (double)cut_decay(gi[0]), x1 = (double)cut_decay(gi[1]);
        double sum = x0 + x1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += y;
        }
        const double last = __shfl_sync(0xffffffffu, sum, 31) * 1.4426950408889634;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const double G = (i == 0 ? sum - x1 : sum) * 1.4426950408889634;
            // P / eta: exp(G_r - G_i) / exp(G_last - G_i), the latter not below its floor
            const double c = backward ? G : last - G > (double)ETA_FLOOR_LOG2 ? last : G + (double)ETA_FLOOR_LOG2;
            sGh[r] = (float)G;
            sGl[r] = (float)(G - (double)(float)G);
            sCh[r] = (float)c;
            sCl[r] = (float)(c - (double)(float)c);
            // the backward divides by beta: not below 2^-30
            sB[r] = backward && real[i] && fabsf(bi[i]) < 0x1p-30f ? copysignf(0x1p-30f, bi[i]) : bi[i];
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    float* x00 = reinterpret_cast<float*>(sm + B00);
    float* x10 = reinterpret_cast<float*>(sm + B10);
    float* x11 = reinterpret_cast<float*>(sm + B11);
    {   // thread: one row of [K K^T; Q K^T]; warps 0-1 make A, warps 2-3 P
        const int r = tid % C;
        const float gh = sGh[r], gl = sGl[r], f = warp < 2 ? sB[r] : backward ? scale : scale * ETA_UNSCALE;
        const float* from_h = warp < 2 ? sGh : sCh;
        const float* from_l = warp < 2 ? sGl : sCl;
        const int last = warp < 2 ? r - 1 : r;        // the row's last column
        const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll 1
        for (int col = 0; col < C; col += 16) {
            float x[16];
            if (col > (r | 31)) {                     // a block above the diagonal (warp-uniform): A's is never read
                if (warp >= 2) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = 0.f;
                    store_split(rec + REC_PH, rec + REC_PL, r, col, x);
                }
                continue;
            }
            tmem_ld16(tm + ((uint32_t)(32 * warp) << 16) + col, x);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 ch = *reinterpret_cast<const float4*>(from_h + col + i), cl = *reinterpret_cast<const float4*>(from_l + col + i);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 h = e ? make_float2(ch.z, ch.w) : make_float2(ch.x, ch.y);
                    const float2 l = e ? make_float2(cl.z, cl.w) : make_float2(cl.x, cl.y);
                    const float2 d = add2(fma2(h, minus, make_float2(gh, gh)), fma2(l, minus, make_float2(gl, gl)));
                    const float2 y = mul2(mul2(make_float2(exp2_fast(d.x), exp2_fast(d.y)), make_float2(f, f)),
                                          make_float2(x[i + e], x[i + e + 1]));
                    x[i + e] = col + i + e <= last ? y.x : 0.f;
                    x[i + e + 1] = col + i + e + 1 <= last ? y.y : 0.f;
                }
            }
            if (warp < 2) {
                float* a = warp == 0 ? x00 : col < 32 ? x10 : x11;
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(a + at(lane, col % 32 + i)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else {
                store_split(rec + REC_PH, rec + REC_PL, r, col, x);
            }
        }
    }
    if (warp < 2) {
        // the 16 x 16 diagonal blocks of this warp's rows: forward substitution, one column per lane, its values in
        // registers and the rows of A as broadcast reads (half h is 16 rows and 16 columns on, where the groups of
        // columns are permuted by 4 more)
        __syncwarp();
        float* blk = warp ? x11 : x00;
        const int h = lane >> 4, j = lane & 15;
        const float* up = blk + h * (16 * 32 + 16);
        const float* down = blk + h * (16 * 32 - 16);
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < r; i += 4) {
                const int piece = (i >> 2) ^ swz(r);
                const float4 v = *reinterpret_cast<const float4*>((piece & 4 ? down : up) + r * 32 + 4 * piece);
                s[0] = fmaf(v.x, x[i], s[0]);
                if (i + 1 < r) s[1] = fmaf(v.y, x[i + 1], s[1]);
                if (i + 2 < r) s[2] = fmaf(v.z, x[i + 2], s[2]);
                if (i + 3 < r) s[3] = fmaf(v.w, x[i + 3], s[3]);
            }
            x[r] = r == j ? 1.f : r > j ? -((s[0] + s[1]) + (s[2] + s[3])) : 0.f;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 16; ++r) blk[at(16 * h + r, 16 * h + j)] = x[r];
    } else {
        const int r = tid - C;
        const float gh = sGh[r], gl = sGl[r], gam = exp2f(gh + gl);
        const float eta = (sGh[C - 1] - gh) + (sGl[C - 1] - gl);
        reinterpret_cast<float*>(rec + REC_NGAM)[r] = -gam;
        // powers of two after the exponentials, so that these keep their digits
        reinterpret_cast<float*>(rec + REC_ETA)[r] = backward ? exp2f(eta) : ETA_SCALE * exp2f(eta > ETA_FLOOR_LOG2 ? eta : ETA_FLOOR_LOG2);
        reinterpret_cast<float*>(rec + REC_GQ)[r] = scale * gam;
        reinterpret_cast<float*>(rec + REC_BETA)[r] = sB[r];
        sNG[r] = -gam;
    }
    fence_before_sync();
    __syncthreads();
    // blocks next to one another: X10 = -X11 (A10 X00), of 16 and then of 32; every warp takes 8 columns
    {
        float* blk = warp < 2 ? x00 : x11;
        join<1>(blk, blk, 16, blk, 16, 8 * (warp & 1), lane);
    }
    join<2>(x00, x10, 0, x11, 0, 8 * warp, lane);
    {   // T = X diag(beta) as two bf16 numbers, in the operand layout: one row and 32 columns per thread
        const int r = tid % C, half = tid / C, col = 32 * half;
        const float* blk = half ? x11 : r < 32 ? x00 : x10;
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(blk + at(lane, i)), b = *reinterpret_cast<const float4*>(sB + col + i);
            x[i] = v.x * b.x; x[i + 1] = v.y * b.y; x[i + 2] = v.z * b.z; x[i + 3] = v.w * b.w;
        }
        if (r < col) {                                // above the diagonal (warp-uniform): not kept
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        store_split(rec + REC_TH, rec + REC_TL, r, col, x);
        store_split(rec + REC_TH, rec + REC_TL, r, col + 16, x + 16);
        __syncthreads();                              // X has been read
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(sNG + col + i);
            x[i] *= v.x; x[i + 1] *= v.y; x[i + 2] *= v.z; x[i + 3] *= v.w;
        }
        store_split(sm + BOX, sm + 3 * BOX, r, col, x);
        store_split(sm + BOX, sm + 3 * BOX, r, col + 16, x + 16);
    }
    fence_smem_to_async();
    __syncthreads();
    // -W^T = K^T (-T diag(gam))^T, d_k as M
    if (warp == 0) {
        fence_after_sync();
        if (issued) {
            constexpr uint32_t id = idesc_bf16(128, C, true);
            const uint64_t kd = (sdesc_sw128(tile) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(2 * BOX >> 4) << 16);
            mma4_ss<128, 16>(tm, kd, sdesc(tile + BOX, 128, 1024), id, 0u);
            mma4_ss<128, 16>(tm, kd, sdesc(tile + 3 * BOX, 128, 1024), id, 1u);
            mma_commit_w(done);
            if (!wait(done, 1)) mbar_wait(done, 1, DRAIN_NS);
        }
    }
    __syncthreads();
    fence_after_sync();
    {   // -W^T to two planes of swizzled boxes, 8 channels x 8 tokens at a time through transposing matrix stores: a
        // thread has two neighbouring tokens of a channel, of one 8 channels on, and of both the lower plane
        const int token = lane & 7, octet = (lane >> 3) & 1, plane = lane >> 4;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            const int ch = 32 * warp + 16 * (q >> 1), col = 32 * (q & 1);
            const uint32_t dst = tile + (2 * plane + ch / 64) * BOX + (col + token) * 128 + ((((ch % 64) / 8 + octet) ^ token) * 16);
            float x[16];
            tmem_ld_16x256b(tm + ((uint32_t)ch << 16) + col, x);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float hi[2], lo[2];
                split_bf16(x[4 * k], x[4 * k + 1], hi[0], lo[0]);
                split_bf16(x[4 * k + 2], x[4 * k + 3], hi[1], lo[1]);
                store_transposed(dst + k * 8 * 128, hi[0], hi[1], lo[0], lo[1]);
            }
        }
    }
    fence_smem_to_async();
    fence_before_sync();
    __syncthreads();
    if (tid == 0) {
        bulk_store(rec + REC_WH, tile, 4 * BOX);
        bulk_commit();
        bulk_wait_read_all();
    }
    // a wait that expired leaves NaN in the state, the outputs and the gradients
    if (s_abort && tid >= C) {
        for (uint32_t at : {REC_NGAM, REC_ETA, REC_GQ}) reinterpret_cast<float*>(rec + at)[tid - C] = __int_as_float(0x7fc00000);
    }
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tm, C);
    }
}

bool make_token_map(CUtensorMap* map, const void* base, int64_t tokens, int64_t cols, int64_t stride, bool store)
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
    const cuuint32_t box[2] = {store ? 128u : 64u, store ? 32u : (cuuint32_t)C};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, store ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t order_launch(Seqs& seqs, int* offsets, cudaStream_t stream)
{
    if (seqs.n_seq < 32) return cudaSuccess;
    order_kernel<<<1, ORDER_NT, 0, stream>>>(seqs, offsets);
    note_launches(1);
    seqs.cu = offsets;
    return cudaGetLastError();
}

static DeviceFlags g_prep_attr_done;

cudaError_t prep_launch(const CUtensorMap& mq, const CUtensorMap& mk, const void* g, const void* beta, const Seqs& seqs,
                        int* offsets, uint8_t* rec, float scale, int HK, int HV, int f32_gates, bool backward, cudaStream_t stream)
{
    const cudaError_t e = once_per_device(g_prep_attr_done, [](int) {
        return cudaFuncSetAttribute(prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep::SMEM);
    });
    if (e != cudaSuccess) return e;
    if (seqs.cu == offsets) offsets = nullptr;        // in order already
    prep_kernel<<<(unsigned)(slot_count(seqs) * HV), prep::NT, prep::SMEM, stream>>>(
        mq, mk, g, beta, seqs, offsets, rec, scale, HK, HV, f32_gates, backward, bounded_wait_limit_ns());
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
