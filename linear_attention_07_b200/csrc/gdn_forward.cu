// Gated delta rule, one decay per head: chunked forward, after the prep kernel
// (gdn_prep.cu).  One CTA per sequence and value head carries the state
// through the chunks; per chunk (gdn_chunk.cuh)
//     U = T V - W S,   O = scale gam Q S + P U,   S <- gam_last S + K^T (eta U).
// Every product is computed transposed, with d_v as the M = 128 of the MMA:
//     U^T = V^T T^T - S^T W^T,  X_Q^T = S^T Q^T,  O^T = (eta U)^T (P / eta)^T,
//     S^T += (eta U)^T K,
// so the left operands that are computed here (S, eta U: fp32 values as two
// bf16) go from registers to tensor memory, everything that is in memory (K,
// Q, V, T, W, P: bf16) is read by the MMA as TMA left it, and thread j owns
// column j of S, U and O throughout: nothing the chain computes passes through
// shared memory.  Sums are fp32; the state is updated in fp32 registers (never
// accumulated in tensor memory, whose additions need not round to nearest).
//
// Long sequences of few heads run in segments, as the chunks of one head are a
// chain: every segment from zero and its transition at the same time, the start
// states joined, and every segment again with its outputs.
//
// Roles (22 warps):
//   warps 0-15  chain: thread (j, part) holds S[dk][j] for 16 + 16 values of
//               dk and takes 16 of the chunk's tokens; eta U, the state
//               update, and their split into bf16 pairs
//   warps 16-19 output: thread j takes O^T's row j, 64 tokens, through
//               shared memory to tensor stores, off the chain's path
//   warp 20     issues every MMA
//   warp 21     loads: K, Q, V (128-byte swizzle), W and T into two stages, P
//               into one buffer, the gates into four slots; prefetches to L2
// The chain waits for two products in turn (W S, K^T U) and converts between
// them; splitting fp32 values into bf16 pairs is most of what the SM issues.
// What the chain does not wait for (T V, X_Q, O) is issued where the tensor
// cores would be idle.  The state goes in two halves of d_k, so that a product
// runs on one while the other is converted (halves of the tokens gain nothing:
// an MMA of N = 32 takes as long as one of N = 64).
//
// A chunk takes 2.5 us (about 4,500 cycles; 2.8 us when more than half of the
// SMs run one, 2.2 us without outputs), whatever its head: a chain of two
// products of 0.4 us each, four passes between tensor memory and registers and
// the splits.  4 x 16384 tokens x 32 heads: 742 us on 128 SMs.  History of a
// chunk at 8192 tokens x 32 heads: 3.4 us with three products in turn (T R after
// V - K S), 3.3 with stages freed late, 2.6 with W formed before.
#include <algorithm>
#include <cmath>

#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

__device__ int g_fwd_status;

namespace fw {

constexpr int N_CHAIN = 16, N_OUT = 4;               // warps
constexpr int W_MMA = N_CHAIN + N_OUT, W_LOAD = W_MMA + 1;
constexpr int NT = 32 * (W_LOAD + 1);

// a stage: K0 Q0 K1 Q1 V0 V1 (boxes of 64 tokens x 64 channels), W and T
constexpr int STAGES = 2, GATE_SLOTS = 4;
constexpr uint32_t S_V = 4 * BOX;
constexpr uint32_t S_REC = 6 * BOX;
constexpr uint32_t STAGE = S_REC + REC_NGAM;
static_assert(STAGE % 1024 == 0, "swizzled tiles are 1024-byte aligned");
constexpr uint32_t S_P = STAGES * STAGE;             // P, one buffer
constexpr uint32_t S_GATE = S_P + P_BYTES;           // the gates, which the output warps read later than the rest
constexpr uint32_t S_OUT = S_GATE + GATE_SLOTS * GATE_BYTES;   // o staging [32][128] bf16
constexpr uint32_t SMEM = S_OUT + 32 * D * 2 + 1024;

// barriers (a pair where the work goes in halves)
// A wait by parity may not fall two completions behind: the gates, whose
// readers may still be at chunk c while the stage takes chunk c + 2, have
// barriers of their own.
enum { B_FULL = 0, B_GATE = STAGES, B_MU = B_GATE + GATE_SLOTS, B_MD, B_MO = B_MD + 2, B_S, B_U = B_S + 2, B_OFREE,
       B_DRAIN, N_BAR };

// tensor memory columns
// operands by 16 values: 8 columns of the upper plane (two values each), 8 of the lower
constexpr uint32_t LOWER = 8;
constexpr uint32_t T_S = 0;                          // S^T
constexpr uint32_t T_U = 128;                        // U^T
constexpr uint32_t T_UE = 192;                       // (eta U)^T
constexpr uint32_t T_XQ = 256, T_O = 320;
constexpr uint32_t T_D = 384;                        // (K^T eta U)^T

// A sequence runs in one piece; or, if it has min_chunks chunks, in segments, of
// which the first of two launches runs segment 0 and, for each of the segments
// between it and the last, the state that it reaches from zero and its
// transition (from the identity with V = 0; neither has outputs).
// join_launch makes the start states of these, and the second launch runs all
// but segment 0 from them.  The first launch has the sequences in one piece
// behind those in segments.
enum Pass { WHOLE, FIRST, SECOND };
// Segment 0 counts 8 of the others' 10: its outputs are made while theirs are not.
constexpr int SEG_FIRST = 8, SEG_OTHER = 10;

struct Args {
    Seqs seqs;
    const uint8_t* rec;
    const float* h0;
    float* hT;
    __nv_bfloat16* o;
    // [n_long][HV][D][D] the state behind segment 0 and that before the last; [n_long][segments - 2][HV][D][D] the
    // transitions, the states reached from zero and the start states of those between
    float *end0, *before_last, *M, *N, *start;
    int pass, segments, min_chunks, n_long;          // at most n_long sequences are in segments
    int HK, HV;
    uint64_t wait_ns;
};

}  // namespace fw

__global__ void __launch_bounds__(fw::NT, 1)
forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
               const __grid_constant__ fw::Args p)
{
    using namespace fw;
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[N_BAR];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.x % p.HV, between = p.segments - 2;
    const int tasks = p.pass == WHOLE ? 0 : p.pass == FIRST ? 1 + 2 * between : between + 1;
    const int in_segments = p.n_long * tasks, at = blockIdx.x / p.HV - in_segments;
    const bool whole = at >= 0;
    const int l = whole ? 0 : (at + in_segments) / tasks, task = whole ? 0 : (at + in_segments) % tasks;
    const int n = whole ? at : long_sequence(p.seqs, p.min_chunks, l);
    if (n < 0 || (whole && p.pass == FIRST && chunk_count(p.seqs, n) >= p.min_chunks)) return;
    const int hk = hv / (p.HV / p.HK);
    int begin, end;
    seq_range(p.seqs, n, begin, end);
    int chunks = (end - begin + C - 1) / C;
    int64_t slot0 = (int64_t)(begin / C) + n;
    const int row = state_row(p.seqs, n);
    const int64_t head = ((int64_t)l * p.HV + hv) * D * D, pool = ((int64_t)row * p.HV + hv) * D * D;
    // where the state comes from and goes to; whether outputs are made, and whether V counts as zero and the state
    // begins as the identity
    const float* from = p.h0 && row >= 0 ? p.h0 + pool : nullptr;
    float* to = p.hT && row >= 0 ? p.hT + pool : nullptr;
    bool outputs = true, transition = false;
    if (!whole) {
        const int seg = p.pass == SECOND ? 1 + task : (task + 1) / 2;
        const int64_t mid = (((int64_t)l * between + seg - 1) * p.HV + hv) * D * D;
        if (p.pass == SECOND) {
            from = seg <= between ? p.start + mid : p.before_last + head;
            if (seg <= between) to = nullptr;
        } else if (seg == 0) {
            to = p.end0 + head;
        } else {
            outputs = false;
            transition = task % 2 == 0;
            from = nullptr;
            to = (transition ? p.M : p.N) + mid;
        }
        auto first_chunk = [&](int x) {
            constexpr int less = SEG_OTHER - SEG_FIRST;
            return x == 0 ? 0 : (int)((int64_t)chunks * (SEG_OTHER * x - less) / (SEG_OTHER * p.segments - less));
        };
        const int c0 = first_chunk(seg), c1 = first_chunk(seg + 1);
        end = min(end, begin + c1 * C);
        begin += c0 * C;
        slot0 += c0;
        chunks = c1 - c0;
    }
    auto bar = [&](int b) { return smem_u32(&bars[b]); };

    if (tid == 0) {
        for (int b = 0; b < N_BAR; ++b) {
            const int count = b == B_S || b == B_S + 1 ? N_CHAIN : b == B_U ? N_CHAIN + 1 : b == B_OFREE ? N_OUT : 1;
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
    constexpr uint32_t tm = 0;                       // all of tensor memory is this CTA's
    const Waits wait = {&s_abort, &g_fwd_status, p.wait_ns};

    if (warp < N_CHAIN) {
        const int sp = warp & 3, part = warp >> 2, j = 32 * sp + lane;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
        float S[2][16];                              // S[b][i]: d_k = 64 b + 16 part + i
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int dk = 64 * b + 16 * part + i;
                S[b][i] = from ? from[dk * D + j] : transition && dk == j ? 1.f : 0.f;
            }
        auto put = [&](uint32_t col, const float (&x)[16]) {     // this part's 16 values of an operand
            float w[16];
            tmem_put16(t + col + 16 * part, x, w);
        };
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        auto give = [&](int b) {                     // what this warp put is there
            wait_st();
            fence_before_sync();
            arrive(b);
        };
        if (chunks > 0)
            for (int b = 0; b < 2; ++b) {
                put(T_S + 64 * b, S[b]);
                give(B_S + b);
            }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const float* gates = reinterpret_cast<const float*>(sm + S_GATE + (c % GATE_SLOTS) * GATE_BYTES);
            wait(bar(B_GATE + c % GATE_SLOTS), (c / GATE_SLOTS) & 1);
            const float last = -gates[C - 1];
            float4 eta[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) eta[i] = reinterpret_cast<const float4*>(gates + C + 16 * part)[i];
            float x[16];
            wait(bar(B_MU), c & 1);
            fence_after_sync();
            tmem_ld16(t + T_U + 16 * part, x);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = mul2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(eta[i].x, eta[i].y));
                const float2 b = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(eta[i].z, eta[i].w));
                x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
            }
            put(T_UE, x);
            give(B_U);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                wait(bar(B_MD + b), c & 1);
                fence_after_sync();
                tmem_ld16(t + T_D + 64 * b + 16 * part, x);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 d = mul2(make_float2(x[i], x[i + 1]), make_float2(ETA_UNSCALE, ETA_UNSCALE));
                    const float2 y = fma2(make_float2(last, last), make_float2(S[b][i], S[b][i + 1]), d);
                    S[b][i] = y.x;
                    S[b][i + 1] = y.y;
                }
                if (c + 1 < chunks) {
                    put(T_S + 64 * b, S[b]);
                    give(B_S + b);
                }
            }
        }
        if (to)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) to[(64 * b + 16 * part + i) * D + j] = S[b][i];
    } else if (warp < W_MMA) {
        const int sp = warp & 3, j = 32 * sp + lane;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
        const int ot = tid - 32 * N_CHAIN;
        __nv_bfloat16* so = reinterpret_cast<__nv_bfloat16*>(sm + S_OUT);
#pragma unroll 1
        for (int c = 0; c < chunks && outputs; ++c) {
            const float2* gq = reinterpret_cast<const float2*>(sm + S_GATE + (c % GATE_SLOTS) * GATE_BYTES + (REC_GQ - REC_NGAM));
            wait(bar(B_GATE + c % GATE_SLOTS), (c / GATE_SLOTS) & 1);
            wait(bar(B_MO), c & 1);
            fence_after_sync();
            float x[32], y[32];
            tmem_ld32(t + T_XQ, x);
            tmem_ld32(t + T_O, y);
            wait_ld();
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int t0 = begin + c * C + 32 * q;
                if (ot == 0) bulk_wait_read_all();    // the staging's last store has read it
                asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 v = fma2(gq[16 * q + i / 2], make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]));
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v.x, v.y);
                    so[i * D + j] = b2.x;
                    so[(i + 1) * D + j] = b2.y;
                }
                if (q == 0) {                        // the second half, so that the next products may begin
                    tmem_ld32(t + T_XQ + 32, x);
                    tmem_ld32(t + T_O + 32, y);
                    wait_ld();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_OFREE));
                }
                fence_smem_to_async();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (t0 + 32 <= end) {
                    if (ot == 0) {
                        tma_store_2d(&mo, hv * D, t0, smem_u32(so));
                        bulk_commit();
                    }
                } else {                             // rows behind the sequence are not stored
                    for (int e = ot; e < 32 * D / 8; e += 128) {
                        const int r = e / (D / 8), c8 = e % (D / 8);
                        if (t0 + r < end)
                            *reinterpret_cast<uint4*>(p.o + ((int64_t)(t0 + r) * p.HV + hv) * D + 8 * c8) =
                                *reinterpret_cast<const uint4*>(so + r * D + 8 * c8);
                    }
                }
            }
        }
        if (ot == 0) bulk_wait_all();
    } else if (warp == W_MMA) {
        const uint32_t id_n64 = idesc_bf16(128, 64), id_d = idesc_bf16(128, 64, false, true);
        const uint32_t id_v = idesc_bf16(128, 64, true);
        auto ok = [&](int b, uint32_t parity) {       // every lane sees the same outcome
            const bool w = wait(bar(b), parity);
            return __all_sync(0xffffffffu, w) != 0;
        };
        // chunk c is there: its rows behind the sequence count as zero, whatever they hold; U^T = V^T T^T
        auto begin_chunk = [&](int c) {
            const int s = c & 1;
            if (!ok(B_FULL + s, (c >> 1) & 1)) return false;
            uint8_t* st = sm + s * STAGE;
            const int nv = min(C, end - (begin + c * C));
            if (nv < C) {
                for (int e = lane; e < (C - nv) * 6 * 8; e += 32) {
                    const int piece = e & 7, box = (e >> 3) % 6, r = nv + (e >> 3) / 6;
                    *reinterpret_cast<uint4*>(st + box * BOX + r * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_smem_to_async();
                __syncwarp();
            }
            const uint32_t base = smem_u32(st);
            if (transition) return true;
            const uint64_t vd = (sdesc_sw128(base + S_V) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(BOX >> 4) << 16);
            mma4_ss<128, 16>(tm + T_U, vd, sdesc(base + S_REC + REC_TH, 128, 1024), id_v, 0u);
            mma4_ss<128, 16>(tm + T_U, vd, sdesc(base + S_REC + REC_TL, 128, 1024), id_v, 1u);
            return true;
        };
        if (chunks > 0) begin_chunk(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t base = smem_u32(sm + (c & 1) * STAGE);
            const uint64_t kq = sdesc_sw128(base), wd = sdesc_sw128(base + S_REC + REC_WH);
            auto w_product = [&](int b) {             // -(W S)^T over half b of d_k
                const uint64_t h = wd + (uint64_t)(b * (BOX >> 4)), l = h + (uint64_t)(2 * BOX >> 4);
                mma4_ts<2>(tm + T_U, tm + T_S + 64 * b, h, id_n64, transition && b == 0 ? 0u : 1u);
                mma4_ts<2>(tm + T_U, tm + T_S + 64 * b + LOWER, h, id_n64, 1u);
                mma4_ts<2>(tm + T_U, tm + T_S + 64 * b, l, id_n64, 1u);
            };
            if (!ok(B_S, c & 1)) break;
            fence_after_sync();
            w_product(0);
            if (!ok(B_S + 1, c & 1)) break;
            fence_after_sync();
            w_product(1);
            mma_commit_w(bar(B_MU));
            if (outputs) {
                if (c > 0 && !ok(B_OFREE, (c - 1) & 1)) break;
                fence_after_sync();
#pragma unroll
                for (int b = 0; b < 2; ++b) {         // (Q S)^T, before a new state replaces the old one
                    const uint64_t qd = kq + (uint64_t)((2 * b + 1) * (BOX >> 4));
                    mma4_ts<2>(tm + T_XQ, tm + T_S + 64 * b, qd, id_n64, b > 0 ? 1u : 0u);
                    mma4_ts<2>(tm + T_XQ, tm + T_S + 64 * b + LOWER, qd, id_n64, 1u);
                }
            }
            if (!ok(B_U, c & 1)) break;               // eta U, and P has landed
            fence_after_sync();
#pragma unroll
            for (int b = 0; b < 2; ++b) {             // (K^T eta U)^T, half b of d_k
                const uint64_t kd = kq + (uint64_t)(2 * b * (BOX >> 4));
                mma4_ts<128>(tm + T_D + 64 * b, tm + T_UE, kd, id_d, 0u);
                mma4_ts<128>(tm + T_D + 64 * b, tm + T_UE + LOWER, kd, id_d, 1u);
                mma_commit_w(bar(B_MD + b));
            }
            if (outputs) {
                const uint64_t ph = sdesc(smem_u32(sm + S_P), 128, 1024), pl = ph + (uint64_t)(BOX >> 4);
                mma4_ts<16>(tm + T_O, tm + T_UE, ph, id_n64, 0u);
                mma4_ts<16>(tm + T_O, tm + T_UE + LOWER, ph, id_n64, 1u);
                mma4_ts<16>(tm + T_O, tm + T_UE, pl, id_n64, 1u);
            }
            mma_commit_w(bar(B_MO));
            // T_U is free: the next chunk's U^T = V^T T^T
            if (c + 1 < chunks && !begin_chunk(c + 1)) break;
        }
        if (chunks > 0) {                             // what was issued ends before its memory goes
            mma_commit_w(bar(B_DRAIN));
            mbar_wait(bar(B_DRAIN), 0, DRAIN_NS);
        }
    } else if (lane == 0) {
        const uint8_t* rec = p.rec + (slot0 * p.HV + hv) * REC_BYTES;
        const int64_t rec_step = (int64_t)p.HV * REC_BYTES;
        int loaded = 0, loaded_p = 0;
        auto load_p = [&](int cp) {                   // one of the arrivals that chunk cp's U waits for
            loaded_p = cp + 1;
            if (!outputs) {
                mbar_arrive(bar(B_U));
                return;
            }
            mbar_arrive_expect_tx(bar(B_U), P_BYTES);
            bulk_load(smem_u32(sm + S_P), rec + cp * rec_step + REC_PH, P_BYTES, bar(B_U));
        };
        // Q is for the outputs; V is not for the transition
        const uint32_t stage_bytes = STAGE - (outputs ? 0 : 2 * BOX) - (transition ? 2 * BOX : 0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            // chunk c - 2's products (O's is the last) are complete: its stage is free, and P's buffer for chunk c - 1.
            // Its gates slot is that of chunk c + 2, which waits for a later output.
            if (c >= 2 && !wait(bar(B_MO), c & 1)) break;
            if (*(volatile int*)&s_abort) break;
            if (c >= 2) load_p(c - 1);
            const uint32_t base = smem_u32(sm + (c & 1) * STAGE), full = bar(B_FULL + (c & 1));
            const int y = begin + c * C;
            const uint8_t* r = rec + c * rec_step;
            mbar_arrive_expect_tx(full, stage_bytes);
            const uint32_t gate = bar(B_GATE + c % GATE_SLOTS);
            mbar_arrive_expect_tx(gate, GATE_BYTES);
            bulk_load(smem_u32(sm + S_GATE) + (c % GATE_SLOTS) * GATE_BYTES, r + REC_NGAM, GATE_BYTES, gate);
            if (!transition)
#pragma unroll
                for (int b = 0; b < 2; ++b) tma_load_2d(base + S_V + b * BOX, &mv, hv * D + 64 * b, y, full);
            bulk_load(base + S_REC, r, REC_NGAM, full);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tma_load_2d(base + 2 * b * BOX, &mk, hk * D + 64 * b, y, full);
                if (outputs) tma_load_2d(base + (2 * b + 1) * BOX, &mq, hk * D + 64 * b, y, full);
            }
            loaded = c + 1;
            if (c == 0) load_p(0);
            const int cn = c < 2 ? c + 2 : c + 1;     // what will be loaded next, on its way to L2
            if (cn < chunks && c >= 1) {
                const int yn = begin + cn * C;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (!transition) tma_prefetch_2d(&mv, hv * D + 64 * b, yn);
                    tma_prefetch_2d(&mk, hk * D + 64 * b, yn);
                    if (outputs) tma_prefetch_2d(&mq, hk * D + 64 * b, yn);
                }
                bulk_prefetch(rec + cn * rec_step, outputs ? REC_BYTES : REC_PH);
            }
        }
        if (loaded == chunks && chunks > 1 && wait(bar(B_MO), chunks & 1)) {     // the last chunk's P
            load_p(chunks - 1);
        }
        // everything loaded has landed before the end
        for (int c = max(0, loaded - STAGES); c < loaded; ++c)
            mbar_wait(bar(B_FULL + (c & 1)), (c >> 1) & 1, DRAIN_NS);
        for (int c = max(0, loaded - GATE_SLOTS); c < loaded; ++c)
            mbar_wait(bar(B_GATE + c % GATE_SLOTS), (c / GATE_SLOTS) & 1, DRAIN_NS);
        if (loaded_p > 0) mbar_wait(bar(B_U), (loaded_p - 1) & 1, DRAIN_NS);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == W_MMA) {
        fence_after_sync();
        tmem_dealloc(s_tmem, 512);
    }
    if (s_abort) {             // a wait expired: no partial result passes for a real one
        const __nv_bfloat16 nan = __float2bfloat16_rn(__int_as_float(0x7fc00000));
        if (outputs)
            for (int64_t e = tid; e < (int64_t)(end - begin) * D; e += NT)
                p.o[((int64_t)(begin + e / D) * p.HV + hv) * D + e % D] = nan;
        if (to)
            for (int e = tid; e < D * D; e += NT) to[e] = __int_as_float(0x7fc00000);
    }
}

static DeviceFlags g_fwd_attr_done;

// Segments of a call's long sequences: where all SMs take three CTAs and more
// per sequence and head (a CTA of this kernel fills one), as many as make the
// first launch one wave; and at most the square root of the sequences' average
// of chunks, as a segment costs about 4 us (its transition is joined to the
// others in turn) and a chunk 2.5 us.  Whole call, one sequence, in one piece
// and so, us: 8192 tokens 401 -> 318 at 32 heads, 343 -> 153 at 8, 322 -> 128 at
// 1 (8 segments 136, 16 139); 32768 tokens of 1 head 1231 -> 240; 2048 tokens
// 117 -> 111 at 32 heads, 100 -> 83 at 8; 1024 tokens 68 -> 74 and 63 -> 67: in
// one piece below 32 chunks on average (lengths are on the device).  With
// more heads a batch's longest sequences gained nothing so, even where they
// took most of the call (16 prompts x 16 heads with one of 4096 tokens, the next
// of 2500 and 2047: 173 us of this kernel in one piece, 220 in four segments).
static void choose_segments(fw::Args& a, int64_t heads, bool ragged)
{
    const int64_t chunks = a.seqs.tokens / C / a.seqs.n_seq;
    const int64_t segments = std::min((current_sm_count() / heads + 3) / 2, (int64_t)std::sqrt((double)chunks));
    if (chunks < MIN_CHUNKS || segments < 3) return;
    a.segments = (int)segments;
    a.min_chunks = MIN_CHUNKS;
    // all of equal lengths, or as many as the tokens can make
    a.n_long = ragged ? (int)std::min<int64_t>(a.seqs.n_seq, a.seqs.tokens / ((MIN_CHUNKS - 1) * C + 1)) : a.seqs.n_seq;
}

}  // namespace gdn

cudaError_t gdn_forward_launch(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* h0, void* o, float* hT, const int* cu, const int* slots, int n_slots,
                               float scale, int N, int T, int HK, int HV, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, int f32_gates, cudaStream_t stream)
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
    a.wait_ns = bounded_wait_limit_ns();
    cudaError_t e = once_per_device(g_fwd_attr_done, [](int) {
        return cudaFuncSetAttribute(forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fw::SMEM);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap mq = {}, mk = {}, mv = {}, mo = {};
    uint8_t* rec = nullptr;
    const int64_t tokens = a.seqs.tokens;
    if (tokens > 0) {
        if (!make_token_map(&mq, q, tokens, (int64_t)HK * D, q_stride) ||
            !make_token_map(&mk, k, tokens, (int64_t)HK * D, k_stride) ||
            !make_token_map(&mv, v, tokens, (int64_t)HV * D, v_stride) ||
            !make_token_map(&mo, o, tokens, (int64_t)HV * D, (int64_t)HV * D, true))
            return cudaErrorInvalidValue;
        keep_pool_memory();
        choose_segments(a, (int64_t)N * HV, cu != nullptr);
        const int64_t heads = (int64_t)a.n_long * HV, state = (int64_t)D * D, between = a.segments - 2;
        const size_t rec_bytes = (size_t)slot_count(a.seqs) * HV * REC_BYTES;
        const size_t states = heads > 0 ? (size_t)(heads * (2 + 3 * between) * state) : 0;
        const size_t offsets = cu ? ((size_t)N + 1) * sizeof(int) : 0;
        e = cudaMallocAsync(reinterpret_cast<void**>(&rec), rec_bytes + states * sizeof(float) + offsets, stream);
        if (e != cudaSuccess) return e;
        if (states) {
            a.end0 = reinterpret_cast<float*>(rec + rec_bytes);
            a.before_last = a.end0 + heads * state;
            a.M = a.before_last + heads * state;
            a.N = a.M + heads * between * state;
            a.start = a.N + heads * between * state;
        }
        int* in_order = cu ? reinterpret_cast<int*>(rec + rec_bytes + states * sizeof(float)) : nullptr;
        if (cu) e = order_launch(a.seqs, in_order, stream);
        if (e == cudaSuccess) e = prep_launch(mq, mk, g, beta, a.seqs, in_order, rec, scale, HK, HV, f32_gates, false, stream);
        a.seqs.cu = in_order;
    }
    a.rec = rec;
    auto launch = [&](int pass, int64_t blocks) {
        a.pass = pass;
        forward_kernel<<<(unsigned)blocks, fw::NT, fw::SMEM, stream>>>(mq, mk, mv, mo, a);
        note_launches(1);
        return cudaGetLastError();
    };
    if (e == cudaSuccess && a.n_long == 0) {
        e = launch(fw::WHOLE, (int64_t)N * HV);
    } else if (e == cudaSuccess) {
        const int64_t between = a.segments - 2, heads = (int64_t)a.n_long * HV;
        e = launch(fw::FIRST, heads * (1 + 2 * between) + (cu ? (int64_t)N * HV : 0));
        if (e == cudaSuccess) {
            JoinArgs j = {a.seqs, {{a.M, a.N, a.end0, a.start, a.before_last}}, HV, (int)between, a.min_chunks};
            e = join_launch(j, 1, heads, stream);
        }
        if (e == cudaSuccess) e = launch(fw::SECOND, heads * (between + 1));
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
