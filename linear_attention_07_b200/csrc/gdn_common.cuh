// Shared pieces of the gated delta rule with one decay per head (the gdn_*
// kernels):
//     S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t
// with HV value heads (v, g, beta, o, S) of which HV / HK share a query/key
// head.  No method arithmetic here: arguments, sequences, gates.
#pragma once
#include "kda_common.cuh"

namespace kda {
namespace gdn {

// What a chunked call addresses.  Tokens are rows of q, k, v (row strides in
// elements: the three may be slices of one projection's output); sequence n
// has tokens [begin, end) of [0, tokens).
struct Seqs {
    const int* cu;          // [n_seq + 1] or null: sequences of `len` tokens each
    const int* slots;       // [n_seq] rows of the state arrays, or null: row n
    int n_seq, n_slots, len;
    int64_t tokens;
};

// The caller's offsets may hold anything.  Offset n counts as the largest of
// cu[0 .. n], cut to [0, tokens]: ranges neither overlap nor go back, whatever
// the array holds.  prep_launch leaves the offsets so for the kernels behind
// it.
__device__ __forceinline__ int cut_offset(const Seqs& s, int v)
{
    return v < 0 ? 0 : v > s.tokens ? (int)s.tokens : v;
}

// Token range of sequence n, by offsets that are in order.
__device__ __forceinline__ void seq_range(const Seqs& s, int n, int& begin, int& end)
{
    if (s.cu) {
        begin = cut_offset(s, s.cu[n]);
        end = max(begin, cut_offset(s, s.cu[n + 1]));
    } else {
        begin = n * s.len;
        end = begin + s.len;
    }
}

// Row of sequence n in the state arrays, or -1 (no state read, none kept).
__device__ __forceinline__ int state_row(const Seqs& s, int n)
{
    if (!s.slots) return n;
    const int r = s.slots[n];
    return r >= 0 && r < s.n_slots ? r : -1;
}

// Gates are fp32 or bf16; which of them are fp32 goes by these bits.
constexpr int G_F32 = 1, BETA_F32 = 2;
__device__ __forceinline__ float gate(const void* p, int64_t i, bool f32)
{
    return f32 ? reinterpret_cast<const float*>(p)[i]
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// Log-decays are cut at -104, where exp is zero in fp32 already: -inf (a
// reset of the state) then leaves the differences of running sums finite.
// NaN stays NaN.
__device__ __forceinline__ float cut_decay(float g) { return g < -104.f ? -104.f : g; }

}  // namespace gdn
}  // namespace kda
