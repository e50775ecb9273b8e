// The gated delta rule token by token on fp32 states (stq_recurrent_step).
//
// Per (request, head) and token, with the state S (d_k x d_v):
//   D = diag(a) S;  w = D^T k;  p = D^T q;  u = beta (v - w);
//   o = p + (q.k) u  (= (D + k u^T)^T q);   S = D + k u^T.
// Reading p from the decayed state lets both sums over the key rows be formed
// in one pass and reduced together, so a token costs one chain of cross-lane
// adds instead of two.
//
// Columns of S are independent of each other, so a wave owns 32 of them for all
// d_k key rows and runs every token without LDS or a barrier: lane l holds
// columns 4 (l % 8) .. +3 of the d_k/8 rows of group l / 8 (64 registers at
// d_k = 128), and the sums over the 8 groups are three cross-lane steps.  The
// bound is the state's one read and one write; the loads of a whole wave's
// slab are in flight at once.  Measured, bf16, d 128, 32 heads, MI355X: 512 requests of a token 426 us
// (2169 MB: 5.1 TB/s, what a large copy reaches), 96 of six tokens 85 us (422 MB: 5.0 TB/s), one
// of a token 4.9 us.
#include "stq_seq.h"

namespace stq {
namespace {

// Sum over the lanes l, l ^ 8, l ^ 16, l ^ 32 and their combinations.
__device__ inline float sum_groups(float x) {
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128 /* row_ror:8 */, 0xf, 0xf, true));
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

template <int DK, int DV, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__(2 * DV) k_recurrent(const RecurrentArgs A) {
    constexpr int R = DK / 8;  // key rows of a lane
    const int b = blockIdx.x / A.s.H, h = blockIdx.x % A.s.H;
    const int lane = threadIdx.x & 63, rg = lane >> 3;
    const int col = (threadIdx.x >> 6) * 32 + (lane & 7) * 4;
    const int H = A.s.H;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    if (t0 == t1) return;
    const int slot = A.slot_ids ? A.slot_ids[b] : b;
    if (slot < 0 || slot >= A.slots) {
        for (int t = t0; t < t1; ++t)
            if (rg == 0) {
                const float x = __int_as_float(0x7fc00000);
                *reinterpret_cast<float4 *>(A.o + ((size_t)t * H + h) * DV + col) = make_float4(x, x, x, x);
            }
        return;
    }
    const int commit = A.commit ? min(max(A.commit[b], 0), t1 - t0) : t1 - t0;
    float *sp = A.state + (((size_t)slot * H + h) * DK + rg * R) * DV + col;
    float4 S[R];
#pragma unroll
    for (int r = 0; r < R; ++r) S[r] = *reinterpret_cast<const float4 *>(sp + (size_t)r * DV);

    for (int t = t0; t < t1; ++t) {
        const size_t u0 = (size_t)t * H + h;
        float k[R], q[R], v[4], a[KEYVEC ? R : 1];
        load_row<BF16>(A.s.k, u0 * DK + rg * R, k);
        load_row<BF16>(A.s.q, u0 * DK + rg * R, q);
        load_row<BF16>(A.s.v, u0 * DV + col, v);
        if constexpr (KEYVEC) load_f32(A.s.a + u0 * DK + rg * R, a);
        else a[0] = A.s.a[u0];
        const float beta = A.s.beta[u0];
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f), p = w;
        float kq = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float g = a[KEYVEC ? r : 0];
            S[r].x *= g;
            S[r].y *= g;
            S[r].z *= g;
            S[r].w *= g;
            w.x = __builtin_fmaf(S[r].x, k[r], w.x);
            w.y = __builtin_fmaf(S[r].y, k[r], w.y);
            w.z = __builtin_fmaf(S[r].z, k[r], w.z);
            w.w = __builtin_fmaf(S[r].w, k[r], w.w);
            p.x = __builtin_fmaf(S[r].x, q[r], p.x);
            p.y = __builtin_fmaf(S[r].y, q[r], p.y);
            p.z = __builtin_fmaf(S[r].z, q[r], p.z);
            p.w = __builtin_fmaf(S[r].w, q[r], p.w);
            kq = __builtin_fmaf(k[r], q[r], kq);
        }
        kq = sum_groups(kq);
        const float4 u = make_float4(beta * (v[0] - sum_groups(w.x)), beta * (v[1] - sum_groups(w.y)),
                                     beta * (v[2] - sum_groups(w.z)), beta * (v[3] - sum_groups(w.w)));
        const float4 o = make_float4(
            __builtin_fmaf(kq, u.x, sum_groups(p.x)), __builtin_fmaf(kq, u.y, sum_groups(p.y)),
            __builtin_fmaf(kq, u.z, sum_groups(p.z)), __builtin_fmaf(kq, u.w, sum_groups(p.w)));
        if (rg == 0) *reinterpret_cast<float4 *>(A.o + u0 * DV + col) = o;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            S[r].x = __builtin_fmaf(k[r], u.x, S[r].x);
            S[r].y = __builtin_fmaf(k[r], u.y, S[r].y);
            S[r].z = __builtin_fmaf(k[r], u.z, S[r].z);
            S[r].w = __builtin_fmaf(k[r], u.w, S[r].w);
        }
        if (t - t0 + 1 == commit) {
#pragma unroll
            for (int r = 0; r < R; ++r) *reinterpret_cast<float4 *>(sp + (size_t)r * DV) = S[r];
        }
    }
}

template <int DK, int DV>
void go(const RecurrentArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)a.s.B * (unsigned)a.s.H), block(2 * DV);
    if (keyvec && bf16) k_recurrent<DK, DV, true, true><<<grid, block, 0, s>>>(a);
    else if (keyvec) k_recurrent<DK, DV, true, false><<<grid, block, 0, s>>>(a);
    else if (bf16) k_recurrent<DK, DV, false, true><<<grid, block, 0, s>>>(a);
    else k_recurrent<DK, DV, false, false><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_recurrent(const RecurrentArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && dv == 64) go<64, 64>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, 128>(a, keyvec, bf16, s);
    else if (dv == 64) go<128, 64>(a, keyvec, bf16, s);
    else go<128, 128>(a, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
