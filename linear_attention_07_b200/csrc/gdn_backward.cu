// Gated delta rule, one decay per head: backward of the chunked forward, after
// the prep kernel (gdn_prep.cu).  With dO~ = scale dO, dS1 = dL/dS1 and the
// chunk's quantities of gdn_chunk.cuh:
//     dU  = P^T dO + eta (K dS1)
//     dV  = T^T dU
//     dS0 = gam_last dS1 - W^T dU + Q^T (gam dO~)
// and, with E = U / beta and Z = dV / beta (A enters U through (I + A) U =
// beta (V - gam K S0), so dA = -Z U^T):
//     dkk_ri = -D_ri dV_r . U_i  (i < r),    dqk_ri = scale D_ri dO_r . U_i  (i <= r)
//     dQ  = gam dO~ S0^T + dqk K
//     dK  = [-gam dV S0^T + dkk K]  +  [eta U dS1^T + dkk^T K + dqk^T Q]
//     dbeta_r = Z_r . E_r = dV_r . U_r / beta_r^2
// The gradient of a log-decay collects every path across its token, without
// the cancellation of a sum over all tokens behind it:
//     dg_t = gam_last <dS1, S0>  +  sum_{r >= t} a_r  +  sum_{i < t} b_i  +  sum_{i < t <= r} w_ri
//     a_r  = gam_r (dO~_r . q_r S0 - dV_r . k_r S0)         read behind t what was there before the chunk
//     b_i  = eta_i U_i . k_i dS1                            written before t and kept to the chunk's end
//     w_ri = dqk_ri q_r . k_i + dkk_ri k_r . k_i            written before t, read behind it
// A write strength of zero would make dbeta 0 / 0: the backward takes |beta|
// as at least 2^-30 (below fp32's resolution of the state).
//
// Two launches after the prep (four where sequences run in segments):
//   1. chains_kernel: per sequence and value head two CTAs side by side, the
//      forward chain (states at the chunks' starts, U) and the reverse chain
//      (state gradients at the chunks' ends, dV, dh0); its transition over chunks
//      is the forward chain's, transposed;
//   2. local_kernel: per chunk and query/key head, dq, dk (summed over the
//      value heads of the group), dg, dbeta.
// All that passes between products is a pair of bf16, as in the forward: a
// single rounding would show in dg and dbeta, which are few numbers each from
// a long sum.
//
// 8192 tokens x 32 heads (16 query/key heads): chains 435 us (215 + 9 + 211; in
// one piece 560: 3.3 us a forward chunk, 4.2 us a reverse one, which has 96 KB
// to store, and an SM stores about 32 bytes a cycle), local 342 us (10 us per value head: the pair products and the states'
// read shared memory at its rate, 128 bytes a cycle, for 7,000 of 18,000 cycles,
// and the sums over the results take the rest).  The local kernel with one role
// that did everything in turn took 410 us; with 16 computing warps of 16 columns
// each in place of 8 of 32, 390 against 364 us at that time.
#include <algorithm>
#include <cmath>

#include "gdn_chunk.cuh"

namespace kda {
namespace gdn {

__device__ int g_back_status;

namespace bk {

// a state as two bf16 planes, each as the local kernel's left operand (M =
// d_k, K = d_v in two halves, MN-major without swizzle): element (i, j) at
// (j / 64) * 16384 + (i / 8) * 1024 + (j % 64) * 16 + (i % 8) * 2
constexpr uint32_t PLANE = D * D * 2, HALF = PLANE / 2;
constexpr uint32_t ST_SBO = 1024, ST_LBO = 128;
// U and dV as two planes each, as operands with the tokens as M or N and d_v
// as K (MN-major without swizzle): element (r, j) at (r / 8) * 2048 + j * 16 +
// (r % 8) * 2.  In both, the thread that owns column j writes 16 bytes, a warp
// 512 in a row.
constexpr uint32_t UPLANE = C * D * 2;
constexpr uint32_t U_SBO = 2048, U_LBO = 128;

// ------------------------------------------------------------------ chains --

constexpr int N_CHAIN = 16, N_OUT = 4;               // warps
constexpr int W_MMA = N_CHAIN + N_OUT, W_LOAD = W_MMA + 1;
constexpr int NT = 32 * (W_LOAD + 1);
// a stage: K0 Q0 K1 Q1, V0 V1 (reverse: dO), W, T and the gates
constexpr int STAGES = 2;
constexpr uint32_t S_V = 4 * BOX, S_REC = 6 * BOX;
constexpr uint32_t STAGE = S_REC + REC_W_BYTES;
static_assert(STAGE % 1024 == 0, "swizzled tiles are 1024-byte aligned");
constexpr uint32_t S_P = STAGES * STAGE;             // reverse: P, one buffer
constexpr uint32_t SMEM = S_P + P_BYTES + 1024;

// A wait by parity may not fall two completions behind, so what a slower role
// waits for goes by chunk parity: a stage's last product (B_FREE, the loads),
// U or dV (B_MV, the output warps) and its having been read (B_OFREE).
enum { B_FULL = 0, B_FREE = STAGES, B_P = 2 * STAGES, B_MU, B_MD, B_MV = B_MD + 2, B_S = B_MV + 2, B_U = B_S + 2, B_DO,
       B_OFREE, B_DRAIN = B_OFREE + 2, N_BAR };

// operands by 16 values: 8 columns of the upper plane (two values each), 8 of the lower
constexpr uint32_t LOWER = 8;
constexpr uint32_t T_S = 0;
constexpr uint32_t T_U = 128;                        // forward: U^T, by chunk parity here or in T_U2; reverse: (K dS1)^T, then dV^T
constexpr uint32_t T_U2 = 256;
constexpr uint32_t T_UE = 192;                       // forward: (eta U)^T; reverse: dU^T
constexpr uint32_t T_PO = 256;                       // reverse: (P^T dO)^T
constexpr uint32_t T_OG = 320;                       // reverse: (gam dO~)^T
constexpr uint32_t T_D = 384;

// Sequences of min_chunks chunks run in segments, of which those between the
// first and the last count SEG_OTHER and these two SEG_END.  The first launch
// has, per value head, the forward chain's first segment and the reverse chain's
// last in full, and for each segment between them the state that either chain
// reaches from zero and the transition M (M^T for the reverse chain), which leave
// nothing else.  join_launch makes the start states, the second launch runs the
// other segments.  With fwd_parts the forward chain instead goes in two parts one
// after the other, FWD_FIRST % of it in the first launch.
enum Pass { WHOLE, FIRST, SECOND };
constexpr int SEG_END = 8, SEG_OTHER = 10, FWD_FIRST = 50;

struct Args {
    Seqs seqs;
    const uint8_t* rec;
    const float* h0;
    const float* dhT;
    float* dh0;
    // forward, reverse: as JoinSet, first the state (gradient) at the end of what the first launch runs in full
    float *first[2], *before_last[2], *M[2], *N[2], *start[2];
    int pass, segments, min_chunks, n_long;
    bool fwd_parts;
    uint8_t* S0;            // per (slot, value head): the chunk's start state, two planes
    uint8_t* dS1;           // and its end state's gradient
    uint8_t* u;             // U, two planes
    uint8_t* dv;            // dV, two planes
    int HK, HV;
    uint64_t wait_ns;
};

// What a CTA runs: chunks [c0, c1) of a sequence's head, from a state (gradient)
// (null: zero, or the identity for the transition, where V counts as zero) to
// one (null: not kept), and for the transition also its transpose.
struct Piece {
    int n, hv, c0, c1;
    bool rev, full, transition;
    const float* from;
    float *to, *to_t;
};

// False if there is nothing to run.
__device__ __forceinline__ bool find_piece(const Args& p, Piece& pc)
{
    const int between = p.segments - 2, fwd_others = p.fwd_parts ? 1 : between + 1;
    const int tasks = p.pass == WHOLE ? 0 : p.pass == FIRST ? 2 + between * (p.fwd_parts ? 2 : 3) : between + 1 + fwd_others;
    const int64_t in_segments = (int64_t)p.n_long * p.HV * tasks, at = (int64_t)blockIdx.x - in_segments;
    pc.full = true;
    pc.transition = false;
    pc.to = pc.to_t = nullptr;
    if (at >= 0) {                                   // the two chains of a head next to one another: they share loads
        pc.rev = (at & 1) != 0;
        pc.hv = (int)((at >> 1) % p.HV);
        pc.n = (int)((at >> 1) / p.HV);
        pc.c0 = 0;
        pc.c1 = chunk_count(p.seqs, pc.n);
        const int64_t head = ((int64_t)pc.n * p.HV + pc.hv) * D * D;
        pc.from = pc.rev ? (p.dhT ? p.dhT + head : nullptr) : p.h0 ? p.h0 + head : nullptr;
        if (pc.rev && p.dh0) pc.to = p.dh0 + head;
        return p.pass == WHOLE || pc.c1 < p.min_chunks;
    }
    const int task = (int)(blockIdx.x / p.HV) % tasks, l = (int)(blockIdx.x / p.HV) / tasks;
    pc.hv = (int)(blockIdx.x % p.HV);
    pc.n = long_sequence(p.seqs, p.min_chunks, l);
    if (pc.n < 0) return false;
    const int chunks = chunk_count(p.seqs, pc.n);
    const int64_t head = ((int64_t)pc.n * p.HV + pc.hv) * D * D, kept = ((int64_t)l * p.HV + pc.hv) * D * D;
    auto bound = [&](int x) {
        return x == 0 ? 0 : x == p.segments ? chunks
                          : (int)((int64_t)chunks * (SEG_END + SEG_OTHER * (x - 1)) / (2 * SEG_END + SEG_OTHER * between));
    };
    // segment x between the ends, as the forward (0) and the reverse chain (1) count it
    auto mid = [&](int dir, int x) { return (((int64_t)l * between + (dir ? between - x : x - 1)) * p.HV + pc.hv) * D * D; };
    int seg;
    if (p.pass == FIRST) {
        const int kinds = p.fwd_parts ? 2 : 3;
        const int kind = task < 2 ? task : (task - 2) % kinds;           // 0 reverse, 1 forward or transition, 2 forward
        seg = task == 0 ? p.segments - 1 : task == 1 ? 0 : 1 + (task - 2) / kinds;
        pc.rev = kind == 0;
        if (task < 2) {
            const float* h = pc.rev ? p.dhT : p.h0;
            pc.from = h ? h + head : nullptr;
            pc.to = p.first[pc.rev] + kept;
        } else {
            pc.full = false;
            pc.from = nullptr;
            pc.transition = kind == 1;
            pc.to = pc.transition ? (p.fwd_parts ? nullptr : p.M[0] + mid(0, seg)) : p.N[pc.rev] + mid(pc.rev, seg);
            if (pc.transition) pc.to_t = p.M[1] + mid(1, seg);
        }
    } else {
        pc.rev = task <= between;
        seg = pc.rev ? task : p.fwd_parts ? 1 : task - between;
        const bool is_mid = seg >= 1 && seg <= between;
        pc.from = !pc.rev && p.fwd_parts ? p.first[0] + kept
               : is_mid ? p.start[pc.rev] + mid(pc.rev, seg) : p.before_last[pc.rev] + kept;
        if (pc.rev && seg == 0 && p.dh0) pc.to = p.dh0 + head;
    }
    pc.c0 = bound(seg);
    pc.c1 = bound(seg + 1);
    if (!pc.rev && pc.full && p.fwd_parts) {
        const int half = (int)((int64_t)chunks * FWD_FIRST / 100);
        pc.c0 = p.pass == FIRST ? 0 : half;
        pc.c1 = p.pass == FIRST ? half : chunks;
    }
    return true;
}

template <bool REV>
__device__ __forceinline__ void chain(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& p,
                                      uint8_t* sm, uint64_t* bars, volatile int* s_abort, const Piece& pc)
{
    using namespace tc;
    constexpr uint32_t tm = 0;                       // all of tensor memory is this CTA's
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = pc.hv, hk = hv / (p.HV / p.HK), chunks = pc.c1 - pc.c0;
    int begin, end;
    seq_range(p.seqs, pc.n, begin, end);
    const int64_t slot0 = (int64_t)(begin / C) + pc.n + pc.c0;
    end = min(end, begin + pc.c1 * C);
    begin += pc.c0 * C;
    const bool full = pc.full, transition = !REV && pc.transition;
    auto bar = [&](int b) { return smem_u32(&bars[b]); };
    auto chunk_at = [&](int c) { return REV ? chunks - 1 - c : c; };
    auto u_cols = [](int c) { return REV || (c & 1) == 0 ? T_U : T_U2; };
    const Waits wait = {s_abort, &g_back_status, p.wait_ns};

    if (warp < N_CHAIN) {
        const int sp = warp & 3, part = warp >> 2, j = 32 * sp + lane;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
        float S[2][16];                              // S[b][i]: d_k = 64 b + 16 part + i
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int dk = 64 * b + 16 * part + i;
                S[b][i] = pc.from ? pc.from[dk * D + j] : transition && dk == j ? 1.f : 0.f;
            }
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        auto give = [&](int b) {
            wait_st();
            fence_before_sync();
            arrive(b);
        };
        auto give_state = [&](int b) {               // the state's half b: operand of the next chunk
            float w[16];
            tmem_put16(t + T_S + 64 * b + 16 * part, S[b], w);
            give(B_S + b);
        };
        // The same words for the local kernel.  An SM stores about 32 bytes a cycle, so that a chunk's 64 KB take as
        // long as half its chain: each half goes out where the chain would wait for a product, read back from the
        // operand, which this warp replaces itself.
        uint8_t* dst0 = (REV ? p.dS1 : p.S0) + (slot0 * p.HV + hv) * (2 * (int64_t)PLANE) + (j / 64) * HALF + 2 * part * ST_SBO + (j % 64) * 16;
        auto store_state = [&](int b, int c) {
            float w[16];
            tmem_ld16(t + T_S + 64 * b + 16 * part, w);
            wait_ld();
            uint8_t* dst = dst0 + chunk_at(c) * (int64_t)p.HV * (2 * (int64_t)PLANE) + 8 * b * ST_SBO;
            *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<float4*>(dst + ST_SBO) = make_float4(w[4], w[5], w[6], w[7]);
            *reinterpret_cast<float4*>(dst + PLANE) = make_float4(w[8], w[9], w[10], w[11]);
            *reinterpret_cast<float4*>(dst + PLANE + ST_SBO) = make_float4(w[12], w[13], w[14], w[15]);
        };
        if (chunks > 0) {
            give_state(0);
            give_state(1);
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const float* gates = reinterpret_cast<const float*>(sm + s * STAGE + S_REC + REC_NGAM);
            wait(bar(B_FULL + s), (c >> 1) & 1);
            const float last = -gates[C - 1];
            float4 eta[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) eta[i] = reinterpret_cast<const float4*>(gates + C + 16 * part)[i];
            float x[16];
            if constexpr (REV) {                     // gam dO~ as an operand, while K dS1 is computed
                const uint8_t* box = sm + s * STAGE + S_V + (j / 64) * BOX + (j % 8) * 2;
                const int piece = (j % 64) / 8, left = end - begin - chunk_at(c) * C - 16 * part;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float d = to_f32(*reinterpret_cast<const __nv_bfloat16*>(box + (16 * part + i) * 128 + ((piece ^ (i & 7)) * 16)));
                    x[i] = i < left ? gates[2 * C + 16 * part + i] * d : 0.f;
                }
                float w[16];
                tmem_put16(t + T_OG + 16 * part, x, w);
                give(B_DO);
            }
            if (full) store_state(0, c);
            wait(bar(B_MU), c & 1);                  // U, or K dS1 and P^T dO
            fence_after_sync();
            tmem_ld16(t + u_cols(c) + 16 * part, x);
            if constexpr (REV) {
                float y[16];
                tmem_ld16(t + T_PO + 16 * part, y);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = fma2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(eta[i].x, eta[i].y), make_float2(y[4 * i], y[4 * i + 1]));
                    const float2 b = fma2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(eta[i].z, eta[i].w), make_float2(y[4 * i + 2], y[4 * i + 3]));
                    x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
                }
            } else {
                wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = mul2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(eta[i].x, eta[i].y));
                    const float2 b = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(eta[i].z, eta[i].w));
                    x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
                }
            }
            {
                float w[16];
                tmem_put16(t + T_UE + 16 * part, x, w);
            }
            give(B_U);
            if (full) store_state(1, c);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                wait(bar(B_MD + b), c & 1);
                fence_after_sync();
                tmem_ld16(t + T_D + 64 * b + 16 * part, x);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 y = fma2(make_float2(last, last), make_float2(S[b][i], S[b][i + 1]), make_float2(x[i], x[i + 1]));
                    S[b][i] = y.x;
                    S[b][i + 1] = y.y;
                }
                if (c + 1 < chunks) give_state(b);
            }
        }
        if (pc.to)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) pc.to[(64 * b + 16 * part + i) * D + j] = S[b][i];
        if (transition)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(pc.to_t + j * D + 64 * b + 16 * part + i) = make_float4(S[b][i], S[b][i + 1], S[b][i + 2], S[b][i + 3]);
    } else if (warp < W_MMA) {
        const int sp = warp & 3, j = 32 * sp + lane;
        const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
#pragma unroll 1
        for (int c = 0; c < chunks && full; ++c) {
            const int s = c & 1;
            wait(bar(B_MV + s), (c >> 1) & 1);
            fence_after_sync();
            uint8_t* out = (REV ? p.dv : p.u) + ((slot0 + chunk_at(c)) * p.HV + hv) * (2 * (int64_t)UPLANE) + j * 16;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                float x[32];
                tmem_ld32(t + u_cols(c) + 32 * q, x);
                wait_ld();
                if (q == 1) {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_OFREE + s));
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split_bf16(x[i + 2 * e], x[i + 2 * e + 1], hi[e], lo[e]);
                    *reinterpret_cast<float4*>(out) = make_float4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<float4*>(out + UPLANE) = make_float4(lo[0], lo[1], lo[2], lo[3]);
                    out += U_SBO;
                }
            }
        }
    } else if (warp == W_MMA) {
        const uint32_t id_n64 = idesc_bf16(128, 64), id_bmn = idesc_bf16(128, 64, false, true);
        const uint32_t id_v = idesc_bf16(128, 64, true, REV);
        auto ok = [&](int b, uint32_t parity) {       // every lane sees the same outcome
            const bool w = wait(bar(b), parity);
            return __all_sync(0xffffffffu, w) != 0;
        };
        // chunk c is there: its rows behind the sequence count as zero, whatever they hold; what needs no state
        auto begin_chunk = [&](int c) {
            const int s = c & 1;
            if (!ok(B_FULL + s, (c >> 1) & 1)) return false;
            uint8_t* st = sm + s * STAGE;
            const int nv = min(C, end - (begin + chunk_at(c) * C));
            if (nv < C) {
                for (int e = lane; e < (C - nv) * 6 * 8; e += 32) {
                    const int piece = e & 7, box = (e >> 3) % 6, r = nv + (e >> 3) / 6;
                    *reinterpret_cast<uint4*>(st + box * BOX + r * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_smem_to_async();
                __syncwarp();
            }
            const uint32_t base = smem_u32(st);
            const uint64_t vd = (sdesc_sw128(base + S_V) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(BOX >> 4) << 16);
            if constexpr (REV) {                     // (P^T dO)^T = dO^T P
                if (!ok(B_P, c & 1)) return false;
                const uint64_t ph = sdesc(smem_u32(sm + S_P), 1024, 128);
                mma4_ss<128, 128>(tm + T_PO, vd, ph, id_v, 0u);
                mma4_ss<128, 128>(tm + T_PO, vd, ph + (uint64_t)(BOX >> 4), id_v, 1u);
            } else {                                 // U^T = V^T T^T
                if (transition) return true;
                if (full && c > 1 && !ok(B_OFREE + (c & 1), ((c >> 1) - 1) & 1)) return false;     // chunk c - 2's U has been read
                fence_after_sync();
                mma4_ss<128, 16>(tm + u_cols(c), vd, sdesc(base + S_REC + REC_TH, 128, 1024), id_v, 0u);
                mma4_ss<128, 16>(tm + u_cols(c), vd, sdesc(base + S_REC + REC_TL, 128, 1024), id_v, 1u);
            }
            return true;
        };
        if (chunks > 0) begin_chunk(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t base = smem_u32(sm + (c & 1) * STAGE);
            const uint64_t kq = sdesc_sw128(base), wd = sdesc_sw128(base + S_REC + REC_WH);
            constexpr uint64_t LO = 2 * BOX >> 4;
            // forward: -(W S)^T; reverse: (K dS1)^T; half b of d_k
            auto s_product = [&](int b) {
                const uint64_t h = REV ? kq + (uint64_t)(2 * b * (BOX >> 4)) : wd + (uint64_t)(b * (BOX >> 4));
                const uint32_t u = tm + u_cols(c);
                mma4_ts<2>(u, tm + T_S + 64 * b, h, id_n64, (REV || transition) && b == 0 ? 0u : 1u);
                mma4_ts<2>(u, tm + T_S + 64 * b + LOWER, h, id_n64, 1u);
                if (!REV) mma4_ts<2>(u, tm + T_S + 64 * b, h + LO, id_n64, 1u);
            };
            if (REV && full && c > 0 && !ok(B_OFREE + ((c - 1) & 1), ((c - 1) >> 1) & 1)) break;
            if (!ok(B_S, c & 1)) break;
            fence_after_sync();
            s_product(0);
            if (!ok(B_S + 1, c & 1)) break;
            fence_after_sync();
            s_product(1);
            mma_commit_w(bar(B_MU));
            if (!REV) mma_commit_w(bar(B_MV + (c & 1)));
            if constexpr (REV) {
                if (!ok(B_DO, c & 1)) break;
                fence_after_sync();
#pragma unroll
                for (int b = 0; b < 2; ++b) {        // Q^T (gam dO~), while the chain computes dU
                    const uint64_t qd = kq + (uint64_t)((2 * b + 1) * (BOX >> 4));
                    mma4_ts<128>(tm + T_D + 64 * b, tm + T_OG, qd, id_bmn, 0u);
                    mma4_ts<128>(tm + T_D + 64 * b, tm + T_OG + LOWER, qd, id_bmn, 1u);
                }
            }
            if (!ok(B_U, c & 1)) break;
            fence_after_sync();
#pragma unroll
            for (int b = 0; b < 2; ++b) {            // forward: (K^T eta U)^T; reverse: -(W^T dU)^T; half b of d_k
                const uint64_t h = REV ? wd + (uint64_t)(b * (BOX >> 4)) : kq + (uint64_t)(2 * b * (BOX >> 4));
                mma4_ts<128>(tm + T_D + 64 * b, tm + T_UE, h, id_bmn, REV ? 1u : 0u);
                mma4_ts<128>(tm + T_D + 64 * b, tm + T_UE + LOWER, h, id_bmn, 1u);
                if (REV) mma4_ts<128>(tm + T_D + 64 * b, tm + T_UE, h + LO, id_bmn, 1u);
                mma_commit_w(bar(B_MD + b));
            }
            if (REV && full) {                       // dV^T = dU^T T
                const uint64_t th = sdesc(base + S_REC + REC_TH, 1024, 128), tl = th + (uint64_t)(BOX >> 4);
                mma4_ts<128>(tm + T_U, tm + T_UE, th, id_bmn, 0u);
                mma4_ts<128>(tm + T_U, tm + T_UE + LOWER, th, id_bmn, 1u);
                mma4_ts<128>(tm + T_U, tm + T_UE, tl, id_bmn, 1u);
                mma_commit_w(bar(B_MV + (c & 1)));
            }
            mma_commit_w(bar(B_FREE + (c & 1)));
            if (c + 1 < chunks && !begin_chunk(c + 1)) break;
        }
        if (chunks > 0) {                             // what was issued ends before its memory goes
            mma_commit_w(bar(B_DRAIN));
            mbar_wait(bar(B_DRAIN), 0, DRAIN_NS);
        }
    } else if (lane == 0) {
        const uint32_t bytes = REV ? STAGE : (transition ? 2 : 4) * BOX + REC_W_BYTES;
        int loaded = 0, loaded_p = 0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            // chunk c - 2's last product is complete: it is done with the stage (who reads the gates or dO does so
            // before a product that this one waits for)
            if (c >= 2 && !wait(bar(B_FREE + s), ((c >> 1) - 1) & 1)) break;
            if (*s_abort) break;
            const uint32_t base = smem_u32(sm + s * STAGE), landed = bar(B_FULL + s);
            const int y = begin + chunk_at(c) * C;
            const uint8_t* rec = p.rec + ((slot0 + chunk_at(c)) * p.HV + hv) * REC_BYTES;
            mbar_arrive_expect_tx(landed, bytes);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tma_load_2d(base + 2 * b * BOX, &mk, hk * D + 64 * b, y, landed);
                if (REV) tma_load_2d(base + (2 * b + 1) * BOX, &mq, hk * D + 64 * b, y, landed);
                if (!transition) tma_load_2d(base + S_V + b * BOX, &mv, hv * D + 64 * b, y, landed);
            }
            bulk_load(base + S_REC, rec, REC_W_BYTES, landed);
            loaded = c + 1;
            if (c + 2 < chunks) {                     // on its way to L2
                const int yn = begin + chunk_at(c + 2) * C;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tma_prefetch_2d(&mk, hk * D + 64 * b, yn);
                    if (REV) tma_prefetch_2d(&mq, hk * D + 64 * b, yn);
                    if (!transition) tma_prefetch_2d(&mv, hv * D + 64 * b, yn);
                }
                bulk_prefetch(p.rec + ((slot0 + chunk_at(c + 2)) * p.HV + hv) * REC_BYTES, REV ? REC_BYTES : REC_W_BYTES);
            }
            if (REV) {                                // P's buffer has been read when chunk c - 1's first products are there
                if (c >= 1 && !wait(bar(B_MU), (c - 1) & 1)) break;
                mbar_arrive_expect_tx(bar(B_P), P_BYTES);
                bulk_load(smem_u32(sm + S_P), rec + REC_PH, P_BYTES, bar(B_P));
                loaded_p = c + 1;
            }
        }
        for (int c = max(0, loaded - STAGES); c < loaded; ++c)
            mbar_wait(bar(B_FULL + (c & 1)), (c >> 1) & 1, DRAIN_NS);
        if (loaded_p > 0) mbar_wait(bar(B_P), (loaded_p - 1) & 1, DRAIN_NS);
    }
}

__global__ void __launch_bounds__(NT, 1)
chains_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const __grid_constant__ Args p)
{
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[N_BAR];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5;
    Piece pc;
    if (!find_piece(p, pc)) return;
    if (tid == 0) {
        for (int b = 0; b < N_BAR; ++b) {
            const int count = b == B_S || b == B_S + 1 || b == B_U || b == B_DO ? N_CHAIN
                            : b == B_OFREE || b == B_OFREE + 1 ? N_OUT : 1;
            mbar_init(smem_u32(&bars[b]), count);
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
    if (pc.rev) chain<true>(mq, mk, mdo, p, sm, bars, &s_abort, pc);
    else chain<false>(mq, mk, mv, p, sm, bars, &s_abort, pc);
    fence_before_sync();
    __syncthreads();
    if (warp == W_MMA) {
        fence_after_sync();
        tmem_dealloc(tm, 512);
    }
    if (*(volatile int*)&s_abort) {                  // a wait expired: no partial result passes for a real one
        const int64_t first = first_slot(p.seqs, pc.n);
        uint8_t* out = pc.rev ? p.dv : p.u;           // the local kernel reads both: its gradients become NaN
        for (int c = pc.c0; c < pc.c1 && pc.full; ++c)
            for (int e = tid; e < (int)UPLANE / 4; e += NT)
                reinterpret_cast<uint32_t*>(out + ((first + c) * p.HV + pc.hv) * (2 * (int64_t)UPLANE))[e] = 0x7fc07fc0u;
        float* to[2] = {pc.to, pc.to_t};
        for (int i = 0; i < 2; ++i)
            if (to[i])
                for (int e = tid; e < D * D; e += NT) to[i][e] = __int_as_float(0x7fc00000);
    }
}

// ------------------------------------------------------------------- local --

namespace lo {
constexpr int LNT = 256, LALL = LNT + 128;            // threads that compute; and a warpgroup whose first warp loads and issues
// registers per thread of the two kinds: 168 at launch, 256 x 216 + 128 x 72 = 384 x 168
constexpr int REGS_COMPUTE = 216, REGS_ISSUE = 72;
// dV and U (two planes each), then boxes of 64 tokens x 64 channels: dO0 dO1 K0 Q0 K1 Q1
constexpr uint32_t O_V = 0, O_U = 2 * UPLANE, O_X = 4 * UPLANE;
constexpr int X_DO = 0, X_K = 2, X_Q = 3, BOXES = 6;
// halves (64 of d_v) of S0 and dS1, two planes each
constexpr uint32_t O_ST = O_X + BOXES * BOX;
// the pair gradients [dkk; dqk] (128 rows of 64, swizzled as a box), two planes; the gates
constexpr uint32_t O_L = O_ST + 4 * HALF, O_G = O_L + 4 * BOX;
constexpr uint32_t SMEM = O_G + 2 * 1024 + 1024;     // two sets of gates
constexpr uint32_t O_OUT = 0;                        // dk and dq [64][128] bf16, at the end
// tensor memory: S0 [dV; dO]^T, dS1 U^T, [dkk; dqk] with K and the rest of dk, dV U^T (lanes 0-63), dO U^T (lanes
// 64-127), [K; Q] K^T
constexpr uint32_t T_A = 0, T_B = 128, T_C = 192, T_G = 320, T_G2 = 384, T_KK = 448;

// Sum over the warp's lanes of each of N values: lane l gets that of x[l % N].
template <int N>
__device__ __forceinline__ float lane_sums(float (&x)[N], int lane)
{
#pragma unroll
    for (int w = N / 2; w > 0; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = up ? x[i] : x[i + w], keep = up ? x[i + w] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    return N == 32 ? x[0] : x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

enum { L_FULL, L_FULL2, L_PAIRS, L_HALF, L_ALL, L_DRAIN, L_ROWS, L_DOT, L_GRADS, L_READ, L_FREE, NBARS };
__device__ __forceinline__ void computing_sync() { asm volatile("bar.sync 1, %0;" :: "n"(LNT) : "memory"); }
}  // namespace lo

struct LocalArgs {
    Seqs seqs;
    const void* g;
    const uint8_t* rec;
    const uint8_t* S0;
    const uint8_t* dS1;
    const uint8_t* u;
    const uint8_t* dvp;
    __nv_bfloat16 *dq, *dk, *dv, *dg, *dbeta;
    float scale;
    int HK, HV;
    int f32_gates;
    uint64_t wait_ns;
};
struct LocalMaps {
    CUtensorMap q, k, dO;
};

__global__ void __launch_bounds__(lo::LALL, 1)
local_kernel(const __grid_constant__ LocalMaps maps, const __grid_constant__ LocalArgs p)
{
    using namespace lo;
    using namespace tc;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[NBARS];
    __shared__ __align__(16) float sGh[C], sGl[C];
    __shared__ float sDB[C], sA[4][C], sB[4][C], sW[4][C], sTot[2 * C], sDot[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x / p.HK;
    const int hk = (int)(blockIdx.x % p.HK), group = p.HV / p.HK;
    int n, chunk, begin, end;
    if (!slot_chunk(p.seqs, slot, n, chunk, begin, end)) return;
    const int t0 = begin + chunk * C, nv = min(C, end - t0);
    const uint32_t base = smem_u32(sm);
    // From the loads and products: L_FULL and L_FULL2 a value head's operands and its states' second halves are here;
    // L_PAIRS, L_HALF, L_ALL the products of the pairs, of the states' first halves, and all are done.  From the
    // computing warps: L_ROWS rows behind the sequence are zero, L_DOT the states' first halves have been read, L_GRADS
    // the pair gradients are in place, L_READ the second halves and dV have been read, L_FREE the sums of all products.
    auto bar = [&](int b) { return smem_u32(&bars[b]); };
    if (tid == 0) {
        for (int b = 0; b < NBARS; ++b) mbar_init(bar(b), b < L_ROWS ? 1 : LNT / 32);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    const Waits waits = {&s_abort, &g_back_status, p.wait_ns};
    auto wait = [&](uint32_t b, uint32_t parity) { return waits.inlined(b, parity); };
    // this thread in tensor memory: lane 32 sp + lane, and the first or second half of the columns
    const int sp = warp & 3, half = warp >> 2, row = 32 * sp + lane;
    const uint32_t t = tm + ((uint32_t)(32 * sp) << 16);
    // dk, dq at channel `row`, 32 tokens, over the group: what comes from the states
    float ak[32], aq[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) ak[i] = aq[i] = 0.f;
    auto xb = [&](int b) { return sdesc_sw128(base + O_X + b * BOX); };
    auto xb_mn = [&](int b) {                        // 128 channels as M or N: the next 64 are two boxes on
        return (sdesc_sw128(base + O_X + b * BOX) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(2 * BOX >> 4) << 16);
    };
    // a plane of dV or U, half h of d_v
    auto up = [&](uint32_t off, int h) { return sdesc(base + off + h * 1024, U_LBO, U_SBO); };
    // the states' half h: S0 and dS1, upper and lower plane
    auto load_states = [&](int64_t unit, int h, uint32_t b) {
        for (int x = 0; x < 2; ++x)
            for (int pl = 0; pl < 2; ++pl)
                bulk_load(base + O_ST + (2 * x + pl) * HALF, (x ? p.dS1 : p.S0) + unit * (2 * (int64_t)PLANE) + pl * PLANE + h * HALF, HALF, b);
    };
    // everything of value head m but the states' second halves; K and Q stay for the group
    auto load_head = [&](int m) {
        const int hv = hk * group + m;
        const int64_t unit = slot * p.HV + hv;
        mbar_arrive_expect_tx(bar(L_FULL), (m == 0 ? 6 : 2) * BOX + 4 * UPLANE + 4 * HALF + 1024);
        bulk_load(base + O_V, p.dvp + unit * (2 * (int64_t)UPLANE), 2 * UPLANE, bar(L_FULL));
        bulk_load(base + O_U, p.u + unit * (2 * (int64_t)UPLANE), 2 * UPLANE, bar(L_FULL));
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            const int x = hv * D + 64 * b, y = hk * D + 64 * b;
            tma_load_2d(base + O_X + (X_DO + b) * BOX, &maps.dO, x, t0, bar(L_FULL));
            if (m == 0) {
                tma_load_2d(base + O_X + (X_K + 2 * b) * BOX, &maps.k, y, t0, bar(L_FULL));
                tma_load_2d(base + O_X + (X_Q + 2 * b) * BOX, &maps.q, y, t0, bar(L_FULL));
            }
        }
        bulk_load(base + O_G + 1024 * (m & 1), p.rec + unit * REC_BYTES + REC_NGAM, 1024, bar(L_FULL));
        load_states(unit, 0, bar(L_FULL));
    };
    // products with the states' half in shared memory: S0 [dV; dO]^T and dS1 U^T (d_k as M)
    auto state_products = [&](int h) {
        const uint32_t idk = idesc_bf16(128, 64, true, false), idm = idesc_bf16(128, 64, true, true);
        const uint64_t s0 = sdesc(base + O_ST, ST_LBO, ST_SBO), s0l = sdesc(base + O_ST + HALF, ST_LBO, ST_SBO);
        const uint64_t ds = sdesc(base + O_ST + 2 * HALF, ST_LBO, ST_SBO), dsl = sdesc(base + O_ST + 3 * HALF, ST_LBO, ST_SBO);
        const uint32_t more = h > 0 ? 1u : 0u;
        mma4_ss<16, 16>(tm + T_A, s0, up(O_V, h), idm, more);
        mma4_ss<16, 16>(tm + T_A, s0l, up(O_V, h), idm, 1u);
        mma4_ss<16, 16>(tm + T_A, s0, up(O_V + UPLANE, h), idm, 1u);
        mma4_ss<16, 2>(tm + T_A + 64, s0, xb(X_DO + h), idk, more);
        mma4_ss<16, 2>(tm + T_A + 64, s0l, xb(X_DO + h), idk, 1u);
        mma4_ss<16, 16>(tm + T_B, ds, up(O_U, h), idm, more);
        mma4_ss<16, 16>(tm + T_B, dsl, up(O_U, h), idm, 1u);
        mma4_ss<16, 16>(tm + T_B, ds, up(O_U + UPLANE, h), idm, 1u);
    };
    // <dS1, S0> over the half in shared memory
    auto state_dot = [&]() {
        float dot = 0.f;
#pragma unroll 2
        for (int e = tid; e < (int)(HALF / 16); e += LNT) {
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = *reinterpret_cast<const uint4*>(sm + O_ST + x * HALF + 16 * e);
            const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = __uint_as_float(u[i] << 16) + __uint_as_float(u[4 + i] << 16);
                const float a1 = __uint_as_float(u[i] & 0xffff0000u) + __uint_as_float(u[4 + i] & 0xffff0000u);
                const float b0 = __uint_as_float(u[8 + i] << 16) + __uint_as_float(u[12 + i] << 16);
                const float b1 = __uint_as_float(u[8 + i] & 0xffff0000u) + __uint_as_float(u[12 + i] & 0xffff0000u);
                dot = fmaf(a0, b0, fmaf(a1, b1, dot));
            }
        }
        return dot;
    };

    if (warp >= LNT / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS_ISSUE));
        if (warp > LNT / 32) {
            __syncthreads();
            return;
        }
        auto ok = [&](int b, int m) {
            const bool r = wait(bar(b), m & 1);
            fence_after_sync();
            return __all_sync(0xffffffffu, r && *(volatile int*)&s_abort == 0);
        };
        bool loaded2 = false;
        int m = 0;
        if (lane == 0) load_head(0);
        __syncwarp();
#pragma unroll 1
        for (; m < group; ++m) {
            loaded2 = false;
            if (!ok(nv < C ? L_ROWS : L_FULL, m)) break;
            // an operand of 64 rows is taken as 128 with its neighbours in shared memory, whose results are not read
            const uint32_t id = idesc_bf16(128, 64), idm = idesc_bf16(128, 64, true, true), idb = idesc_bf16(128, 64, false, true);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint32_t more = h > 0 ? 1u : 0u;
                if (m == 0) mma4_ss<2, 2>(tm + T_KK, xb(X_K + 2 * h), xb(X_K + 2 * h), id, more);
                mma4_ss<16, 16>(tm + T_G, up(O_V, h), up(O_U, h), idm, more);
                mma4_ss<16, 16>(tm + T_G, up(O_V, h), up(O_U + UPLANE, h), idm, 1u);
                mma4_ss<16, 16>(tm + T_G, up(O_V + UPLANE, h), up(O_U, h), idm, 1u);
                mma4_ss<2, 16>(tm + T_G2, xb(X_DO + h - 1), up(O_U, h), idb, more);
                mma4_ss<2, 16>(tm + T_G2, xb(X_DO + h - 1), up(O_U + UPLANE, h), idb, 1u);
            }
            mma_commit_w(bar(L_PAIRS));
            if (m > 0 && !ok(L_FREE, m - 1)) break;
            state_products(0);
            mma_commit_w(bar(L_HALF));
            if (!ok(L_HALF, m) || !ok(L_DOT, m)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(L_FULL2), 4 * HALF);
                load_states(slot * p.HV + hk * group + m, 1, bar(L_FULL2));
            }
            __syncwarp();
            loaded2 = true;
            if (!ok(L_FULL2, m)) break;
            state_products(1);
            if (!ok(L_GRADS, m)) break;
            const uint32_t id128 = idesc_bf16(128, 128, true, false), idmn = idesc_bf16(128, 64, true, true);
            const uint64_t l = sdesc_sw128(base + O_L), k = xb_mn(X_K), q = xb_mn(X_Q);
            constexpr uint64_t LO = 2 * BOX >> 4, Q_ROWS = BOX >> 4;
            // K^T [dkk; dqk]^T, then the columns of dk: K^T dkk + Q^T dqk; summed over the group
            mma4_ss<128, 2>(tm + T_C, k, l, id128, m > 0 ? 1u : 0u);
            mma4_ss<128, 2>(tm + T_C, k, l + LO, id128, 1u);
            mma4_ss<128, 128>(tm + T_C, k, l, idmn, 1u);
            mma4_ss<128, 128>(tm + T_C, k, l + LO, idmn, 1u);
            mma4_ss<128, 128>(tm + T_C, q, l + Q_ROWS, idmn, 1u);
            mma4_ss<128, 128>(tm + T_C, q, l + LO + Q_ROWS, idmn, 1u);
            mma_commit_w(bar(L_ALL));
            if (!ok(L_ALL, m) || !ok(L_READ, m)) break;
            if (m + 1 < group && lane == 0) load_head(m + 1);
            __syncwarp();
        }
        if (m < group) {                              // gave up: what is in flight ends before its space is used again
            mbar_wait(bar(L_FULL), m & 1, DRAIN_NS);
            if (loaded2) mbar_wait(bar(L_FULL2), m & 1, DRAIN_NS);
            mma_commit_w(bar(L_DRAIN));
            mbar_wait(bar(L_DRAIN), 0, DRAIN_NS);
        }
        __syncthreads();
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS_COMPUTE));
#pragma unroll 1
    for (int m = 0; m < group; ++m) {
        const int hv = hk * group + m;
        auto give = [&](int b) {                      // this warp's part of what the issuer waits for
            fence_smem_to_async();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        if (warp == 2) {                              // the running sum of g in units of log 2
            double x[2];
            for (int i = 0; i < 2; ++i) {
                const int rr = 2 * lane + i;
                x[i] = rr < nv ? (double)cut_decay(gate(p.g, (int64_t)(t0 + rr) * p.HV + hv, p.f32_gates & G_F32)) : 0.0;
            }
            double sum = x[0] + x[1];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += y;
            }
            for (int i = 0; i < 2; ++i) {
                const double G = (i == 0 ? sum - x[1] : sum) * 1.4426950408889634;
                sGh[2 * lane + i] = (float)G;
                sGl[2 * lane + i] = (float)(G - (double)(float)G);
            }
        }
        wait(bar(L_FULL), m & 1);
        if (nv < C) {                                 // rows behind the sequence (U's and dV's are zero)
            const int boxes = m == 0 ? BOXES : 2;
            for (int e = tid; e < (C - nv) * boxes * 8; e += LNT) {
                const int piece = e & 7, box = (e >> 3) % boxes, rr = nv + (e >> 3) / boxes;
                *reinterpret_cast<uint4*>(sm + O_X + box * BOX + rr * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            give(L_ROWS);
        }
        computing_sync();
        float dot = state_dot();
        give(L_DOT);
        wait(bar(L_PAIRS), m & 1);
        fence_after_sync();
        {   // pair gradients: dkk_ri = -D_ri dV_r . U_i (i < r), dqk_ri = scale D_ri dO_r . U_i (i <= r)
            float x[32], y[32];
            const int r = row % C;
            const bool is_q = row >= C;
            tmem_ld32(t + (is_q ? T_G2 : T_G) + 32 * half, x);  // is_q is warp-uniform
            tmem_ld32(t + T_KK + 32 * half, y);
            wait_ld();
            const float gh = sGh[r], gl = sGl[r], f = is_q ? p.scale : -1.f;
            const int last = is_q ? r : r - 1;
            float pre = 0.f;                          // of w over the columns before
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 ch = *reinterpret_cast<const float4*>(sGh + 32 * half + i), cl = *reinterpret_cast<const float4*>(sGl + 32 * half + i);
                const float dh[4] = {ch.x, ch.y, ch.z, ch.w}, dl[4] = {cl.x, cl.y, cl.z, cl.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 32 * half + i + e;
                    if (!is_q && c == r) sDB[r] = x[i + e];
                    x[i + e] = c <= last ? f * exp2_fast((gh - dh[e]) + (gl - dl[e])) * x[i + e] : 0.f;
                    pre = fmaf(x[i + e], c < r ? y[i + e] : 0.f, pre);
                    y[i + e] = c + 1 <= r ? pre : 0.f;           // token t = c + 1: this row's part of sum_{i < t <= r} w_ri
                }
            }
            if (half == 0) sTot[row] = pre;
            const float ws = lane_sums(y, lane);
            sW[sp][32 * half + lane] = ws;            // for token 32 half + lane + 1, columns of this half only
#pragma unroll
            for (int pc = 0; pc < 4; ++pc) {
                float hi[4], lw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_bf16(x[8 * pc + 2 * e], x[8 * pc + 2 * e + 1], hi[e], lw[e]);
                uint8_t* dst = sm + O_L + row * 128 + (((4 * half + pc) ^ (row & 7)) * 16);
                *reinterpret_cast<float4*>(dst) = make_float4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<float4*>(dst + 2 * BOX) = make_float4(lw[0], lw[1], lw[2], lw[3]);
            }
        }
        give(L_GRADS);
        wait(bar(L_FULL2), m & 1);
        dot += state_dot();
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) sDot[warp] = dot;
        {   // dv: dV's upper plane, token by token
            const int tok = tid / 4, q = tid & 3, j0 = 32 * q;
            const uint8_t* src = sm + O_V + (tok / 8) * U_SBO + (tok % 8) * 2;
            __nv_bfloat16* out = p.dv + ((int64_t)(t0 + tok) * p.HV + hv) * D + j0;
            if (tok < nv)
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {     // pair (e + q) & 3: neighbouring threads in different banks
                        const uint8_t* a = src + (j0 + i + 2 * ((e + q) & 3)) * 16;
                        w[e] = *reinterpret_cast<const uint16_t*>(a) | ((uint32_t)*reinterpret_cast<const uint16_t*>(a + 16) << 16);
                    }
                    const uint4 x = q & 1 ? make_uint4(w[3], w[0], w[1], w[2]) : make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(out + i) = q & 2 ? make_uint4(x.z, x.w, x.x, x.y) : x;
                }
        }
        give(L_READ);
        wait(bar(L_ALL), m & 1);
        fence_after_sync();
        const float* gates = reinterpret_cast<const float*>(sm + O_G + 1024 * (m & 1));       // -gam, eta, scale gam, beta: 64 each
        {   // channel `row`, tokens 32 half .. + 31 in two parts
            const uint8_t* kp = sm + O_X + (X_K + 2 * (row / 64)) * BOX + (row % 8) * 2;
            const int piece = (row % 64) / 8;
            auto at = [&](const uint8_t* x, int i) {
                return to_f32(*reinterpret_cast<const __nv_bfloat16*>(x + i * 128 + ((piece ^ (i & 7)) * 16)));
            };
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const int tok0 = 32 * half + 16 * part;
                const uint8_t* kt = kp + tok0 * 128;
                float a[16], b[16], c[16], pa[16];
                auto gate4 = [&](int which, int i) { return *reinterpret_cast<const float4*>(gates + which * C + tok0 + i); };
                tmem_ld16(t + T_A + tok0, a);         // dV S0^T
                tmem_ld16(t + T_A + 64 + tok0, b);    // dO S0^T
                tmem_ld16(t + T_B + tok0, c);         // U dS1^T
                wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 g4 = gate4(0, i), h4 = gate4(1, i), q4 = gate4(2, i);
                    const float fa[4] = {g4.x, g4.y, g4.z, g4.w}, fb[4] = {q4.x, q4.y, q4.z, q4.w}, fc[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = at(kt, i + e), y = at(kt + BOX, i + e);
                        const float za = fa[e] * a[i + e], zb = fb[e] * b[i + e], zc = fc[e] * c[i + e];
                        pa[i + e] = fmaf(za, x, zb * y);
                        c[i + e] = zc * x;
                        ak[16 * part + i + e] += za + zc;
                        aq[16 * part + i + e] += zb;
                    }
                }
                const float as = lane_sums(pa, lane), bs = lane_sums(c, lane);
                if (lane < 16) {
                    sA[sp][tok0 + lane] = as;
                    sB[sp][tok0 + lane] = bs;
                }
            }
        }
        give(L_FREE);
        computing_sync();
        if (warp == LNT / 32 - 1) {                   // dg and dbeta, two tokens per lane
            float a[2], b[2], w[2], tot[2], dd = lane < 8 ? sDot[lane] : 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                a[i] = (sA[0][r] + sA[1][r]) + (sA[2][r] + sA[3][r]);
                b[i] = (sB[0][r] + sB[1][r]) + (sB[2][r] + sB[3][r]);
                w[i] = r > 0 ? (sW[0][r - 1] + sW[1][r - 1]) + (sW[2][r - 1] + sW[3][r - 1]) : 0.f;
                tot[i] = sTot[r] + sTot[C + r];       // row r's first 32 columns
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, off);
            float sa = a[0] + a[1], sb = b[0] + b[1], st = tot[0] + tot[1];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float x = __shfl_down_sync(0xffffffffu, sa, off), y = __shfl_up_sync(0xffffffffu, sb, off);
                const float z = __shfl_down_sync(0xffffffffu, st, off);
                if (lane + off < 32) sa += x, st += z;
                if (lane >= off) sb += y;
            }
            // sa, st: from token 2 lane on; sb: up to token 2 lane + 1
            const float before = __shfl_up_sync(0xffffffffu, sb, 1);
            const float from0[2] = {sa, sa - a[0]}, tot0[2] = {st, st - tot[0]};
            const float b0 = lane > 0 ? before : 0.f, upto[2] = {b0, b0 + b[0]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                if (r < nv) {
                    const int64_t o = (int64_t)(t0 + r) * p.HV + hv;
                    const float beta = gates[3 * C + r];
                    const float pairs = w[i] + (r > 32 ? tot0[i] : 0.f);
                    p.dg[o] = __float2bfloat16_rn(fmaf(-gates[C - 1], dd, from0[i] + upto[i] + pairs));
                    p.dbeta[o] = __float2bfloat16_rn(sDB[r] / beta / beta);
                }
            }
        }
    }
    __syncthreads();                                  // no load is in flight
    {   // dk, dq: channel-major in registers, token-major in memory
        __nv_bfloat16* so = reinterpret_cast<__nv_bfloat16*>(sm + O_OUT);
        const bool bad = *(volatile int*)&s_abort != 0;
        float x[32], y[32];
        tmem_ld32(t + T_C + 32 * half, x);
        tmem_ld32(t + T_C + 64 + 32 * half, y);
        wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int tok = 32 * half + i;
            so[tok * D + row] = __float2bfloat16_rn(bad ? __int_as_float(0x7fc00000) : ak[i] + x[i]);
            so[(C + tok) * D + row] = __float2bfloat16_rn(bad ? __int_as_float(0x7fc00000) : aq[i] + y[i]);
        }
        computing_sync();
#pragma unroll 4
        for (int e = tid; e < 2 * C * D / 8; e += LNT) {
            const int r = (e / (D / 8)) % C, c8 = e % (D / 8);
            if (r < nv)
                *reinterpret_cast<uint4*>((e >= C * D / 8 ? p.dq : p.dk) + ((int64_t)(t0 + r) * p.HK + hk) * D + 8 * c8) =
                    *reinterpret_cast<const uint4*>(so + 8 * e);
        }
    }
    fence_before_sync();
    computing_sync();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tm, 512);
    }
    if (*(volatile int*)&s_abort) {
        const __nv_bfloat16 nan = __float2bfloat16_rn(__int_as_float(0x7fc00000));
        for (int e = tid; e < nv * group; e += LNT) {
            const int64_t at = (int64_t)(t0 + e / group) * p.HV + hk * group + e % group;
            p.dg[at] = nan;
            p.dbeta[at] = nan;
        }
        for (int e = tid; e < nv * group * D; e += LNT)
            p.dv[((int64_t)(t0 + e / (group * D)) * p.HV + hk * group) * D + e % (group * D)] = nan;
    }
}

// Tokens before the first sequence and behind the last belong to none: their
// gradients are zero.
struct Outside {
    __nv_bfloat16* p[5];
    int64_t row[5];
};
__global__ void outside_kernel(const Outside z, const int* __restrict__ cu, int n_seq, int64_t tokens)
{
    const int lane = (int)(threadIdx.x & 31);         // fewer than 32 sequences: in any order; else in order
    const int most = __reduce_max_sync(0xffffffffu, n_seq >= 32 ? cu[n_seq] : lane <= n_seq ? cu[lane] : 0);
    const int64_t a = min((int64_t)max(cu[0], 0), tokens), b = min(max((int64_t)most, a), tokens);
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int i = 0; i < 5; ++i) {
        for (int64_t e = at; e < a * z.row[i]; e += step) z.p[i][e] = __float2bfloat16_rn(0.f);
        for (int64_t e = b * z.row[i] + at; e < tokens * z.row[i]; e += step) z.p[i][e] = __float2bfloat16_rn(0.f);
    }
}

}  // namespace bk

static DeviceFlags g_back_attr_done;

// Segments of a call's long sequences, as in the forward: the first launch has
// 3 segments - 4 CTAs per sequence and value head, or 4 for three segments with
// the forward chain in two parts.  Whole call, one sequence, in one piece and so,
// us: 8192 tokens 1009 -> 850 at 32 heads (in parts), 861 -> 724 at 24, 644 ->
// 334 at 8, 534 -> 186 at 1 (6 segments 234, 8 203, 16 183, 24 205); 2560 tokens
// 357 -> 339 at 32 heads; 2048 tokens 274 -> 279 at 32 heads, 255 -> 242 at 24,
// 182 -> 138 at 8; 1024 tokens 159 -> 172, 159 -> 169 and 111 -> 109: in one piece
// below 32 chunks on average, one sequence of 30 heads and more below 40.  Several
// with cu_seqlens go in parts from 32 on, though only the device has their
// lengths: sequences of 16 heads with 4000 + 96 tokens 439 -> 368, 3000 + 1096
// 367 -> 324, 2500 + 2100 343 -> 314, 2048 + 2048 298 -> 287, but 2300 + 1796 317
// -> 347, and of 10 heads with 2000 + 1900 + 2244 298 -> 346: one a little
// below 32 chunks runs in one piece, and what is left of the long one after it.
static void choose_segments(bk::Args& a, int64_t heads, bool ragged)
{
    if (heads == 0) return;
    const int64_t chunks = a.seqs.tokens / C / a.seqs.n_seq, per_head = current_sm_count() / heads;
    a.fwd_parts = per_head < 5;
    const int64_t least = a.fwd_parts && !(ragged && a.seqs.n_seq > 1) ? MIN_CHUNKS + 8 : MIN_CHUNKS;
    if (chunks < least || per_head < 4) return;
    a.segments = (int)std::max<int64_t>(3, std::min((per_head + 4) / 3, (int64_t)std::sqrt((double)chunks)));
    a.min_chunks = MIN_CHUNKS;
    a.n_long = ragged ? (int)std::min<int64_t>(a.seqs.n_seq, a.seqs.tokens / ((MIN_CHUNKS - 1) * C + 1)) : a.seqs.n_seq;
}

}  // namespace gdn

cudaError_t act8_launch(int count, const void* const* src, void* const* dst, void* const* scales, const int64_t* rows,
                        const int64_t* cols, const int64_t* strides, bool pack, cudaStream_t stream);

// scales: null (q, k, v bf16 with the given strides) or the scales of q, k, v
// in 8 bits (dense), which are expanded into the workspace first.
cudaError_t gdn_backward_launch(const void* q, const void* k, const void* v, const void* const* scales, const void* g,
                                const void* beta, const float* h0, const void* dO, const float* dhT, void* dq, void* dk,
                                void* dv, void* dg, void* dbeta, float* dh0, const int* cu, float scale, int N, int T,
                                int HK, int HV, int64_t q_stride, int64_t k_stride, int64_t v_stride, int f32_gates,
                                cudaStream_t stream)
{
    using namespace gdn;
    using namespace bk;
    Args a = {};
    a.seqs.cu = cu;
    a.seqs.n_seq = N;
    a.seqs.n_slots = N;
    a.seqs.len = T;
    a.seqs.tokens = cu ? T : (int64_t)N * T;
    const int64_t tokens = a.seqs.tokens;
    const size_t state = (size_t)N * HV * D * D * sizeof(float);
    if (tokens == 0) {       // no token: the start states' gradient is the last states'
        if (!dh0) return cudaSuccess;
        return dhT ? cudaMemcpyAsync(dh0, dhT, state, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(dh0, 0, state, stream);
    }
    cudaError_t e = once_per_device(g_back_attr_done, [](int) {
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        const cudaError_t r = cudaFuncSetAttribute(chains_kernel, at, (int)SMEM);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(local_kernel, at, (int)lo::SMEM);
    });
    if (e != cudaSuccess) return e;
    const size_t units = (size_t)slot_count(a.seqs) * HV;
    const size_t u_bytes = (size_t)tokens * HV * D * 2, qk_bytes = (size_t)tokens * HK * D * 2;
    choose_segments(a, (int64_t)N * HV, cu != nullptr);
    const int64_t heads = (int64_t)a.n_long * HV, between = a.segments - 2;
    const size_t kept = (size_t)heads * D * D, mids = kept * (heads > 0 ? between : 0);
    size_t bytes = units * (REC_BYTES + 4 * (size_t)PLANE + 4 * (size_t)UPLANE) + (4 * kept + (a.fwd_parts ? 3 : 6) * mids) * sizeof(float);
    if (scales) bytes += 2 * qk_bytes + u_bytes;
    if (cu) bytes += ((size_t)N + 1) * sizeof(int);
    uint8_t* ws = nullptr;
    keep_pool_memory();
    e = cudaMallocAsync(reinterpret_cast<void**>(&ws), bytes, stream);
    if (e != cudaSuccess) return e;
    uint8_t* at = ws;
    auto take = [&](size_t b) { uint8_t* r = at; at += b; return r; };
    a.rec = take(units * REC_BYTES);
    a.S0 = take(units * 2 * PLANE);
    a.dS1 = take(units * 2 * PLANE);
    a.u = take(units * 2 * UPLANE);
    a.dv = take(units * 2 * UPLANE);
    for (int r = 0; r < 2 && heads > 0; ++r) {
        auto floats = [&](size_t n) { return reinterpret_cast<float*>(take(n * sizeof(float))); };
        a.first[r] = floats(kept);
        a.before_last[r] = floats(kept);
        if (r == 0 && a.fwd_parts) continue;
        a.M[r] = floats(mids);
        a.N[r] = floats(mids);
        a.start[r] = floats(mids);
    }
    if (scales) {
        void* out[3] = {take(qk_bytes), take(qk_bytes), take(u_bytes)};
        const void* src[3] = {q, k, v};
        void* sc[3] = {const_cast<void*>(scales[0]), const_cast<void*>(scales[1]), const_cast<void*>(scales[2])};
        const int64_t rows[3] = {tokens, tokens, tokens}, cols[3] = {(int64_t)HK * D, (int64_t)HK * D, (int64_t)HV * D};
        e = act8_launch(3, src, out, sc, rows, cols, nullptr, false, stream);
        q = out[0], k = out[1], v = out[2];
        q_stride = k_stride = (int64_t)HK * D;
        v_stride = (int64_t)HV * D;
    }
    Seqs given = a.seqs;
    int* offsets = cu && N > 0 ? reinterpret_cast<int*>(take(((size_t)N + 1) * sizeof(int))) : nullptr;
    if (offsets) a.seqs.cu = offsets;
    a.h0 = h0;
    a.dhT = dhT;
    a.dh0 = dh0;
    a.HK = HK;
    a.HV = HV;
    a.wait_ns = bounded_wait_limit_ns();
    LocalArgs l = {};
    l.seqs = a.seqs;
    l.g = g;
    l.rec = a.rec;
    l.S0 = a.S0;
    l.dS1 = a.dS1;
    l.u = a.u;
    l.dvp = a.dv;
    l.dv = (__nv_bfloat16*)dv;
    l.dq = (__nv_bfloat16*)dq;
    l.dk = (__nv_bfloat16*)dk;
    l.dg = (__nv_bfloat16*)dg;
    l.dbeta = (__nv_bfloat16*)dbeta;
    l.scale = scale;
    l.HK = HK;
    l.HV = HV;
    l.f32_gates = f32_gates;
    l.wait_ns = a.wait_ns;
    LocalMaps maps;
    CUtensorMap mv;
    const int64_t row = (int64_t)HV * D;
    if (e == cudaSuccess &&
        (!make_token_map(&maps.q, q, tokens, (int64_t)HK * D, q_stride) || !make_token_map(&maps.k, k, tokens, (int64_t)HK * D, k_stride) ||
         !make_token_map(&mv, v, tokens, row, v_stride) || !make_token_map(&maps.dO, dO, tokens, row, row)))
        e = cudaErrorInvalidValue;
    if (e == cudaSuccess && offsets) e = order_launch(given, offsets, stream);
    if (e == cudaSuccess && cu) {
        const int64_t rows[5] = {(int64_t)HK * D, (int64_t)HK * D, (int64_t)HV * D, HV, HV};
        Outside z = {};
        void* out[5] = {dq, dk, dv, dg, dbeta};
        for (int i = 0; i < 5; ++i) z.p[i] = (__nv_bfloat16*)out[i], z.row[i] = rows[i];
        outside_kernel<<<64, 256, 0, stream>>>(z, given.cu, N, tokens);
        note_launches(1);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && N > 0)
        e = prep_launch(maps.q, maps.k, g, beta, given, offsets, const_cast<uint8_t*>(a.rec),
                        scale, HK, HV, f32_gates, true, stream);
    auto chains = [&](int pass, int64_t blocks) {
        a.pass = pass;
        chains_kernel<<<(unsigned)blocks, NT, SMEM, stream>>>(maps.q, maps.k, mv, maps.dO, a);
        note_launches(1);
        return cudaGetLastError();
    };
    if (e == cudaSuccess && N > 0 && heads == 0) {
        e = chains(WHOLE, 2 * (int64_t)N * HV);
    } else if (e == cudaSuccess && N > 0) {
        e = chains(FIRST, heads * (2 + between * (a.fwd_parts ? 2 : 3)) + (cu ? 2 * (int64_t)N * HV : 0));
        JoinArgs j = {a.seqs, {}, HV, (int)between, a.min_chunks};
        int sets = 0;
        for (int r = a.fwd_parts ? 1 : 0; r < 2; ++r) j.set[sets++] = {a.M[r], a.N[r], a.first[r], a.start[r], a.before_last[r]};
        if (e == cudaSuccess) e = join_launch(j, sets, heads, stream);
        if (e == cudaSuccess) e = chains(SECOND, heads * (between + 1 + (a.fwd_parts ? 1 : between + 1)));
    }
    if (e == cudaSuccess && N > 0) {
        note_launches(1);
        local_kernel<<<(unsigned)(slot_count(a.seqs) * HK), lo::LALL, lo::SMEM, stream>>>(maps, l);
        e = cudaGetLastError();
    }
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    return e == cudaSuccess ? ef : e;
}

int gdn_backward_status(cudaStream_t stream)
{
    int st = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&st, gdn::g_back_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(gdn::g_back_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return KDA_ERR_CUDA;
    return st;
}

}  // namespace kda
