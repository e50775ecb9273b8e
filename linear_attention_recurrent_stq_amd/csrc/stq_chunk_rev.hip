// The pass of the state's gradient through the chunks of a sequence, from the last to the
// first (the middle part of stq_chunk_backward).
//
// Per chunk, with dS the gradient of the state behind it and E_i = G_64/G_i:
//   du = (K E) dS + P^T dO;   y = N^T du;   dV = beta y;
//   dS = diag(G_64) dS + (Q G)^T dO - (K G)^T (beta y).
// The gradient behind each chunk and y are kept for the chunk's own gradients.
//
// Laid out as the pass of the state (stq_chunk_fwd.hip).  The chain from one dS to the next is du,
// y, dS; the helping waves form what does not depend on it, P^T dO and (Q G)^T dO, and hand it
// over as result tiles in LDS.
//
// Measured, bf16, d_k = d_v = 128, 16 heads, MI355X: scalar gates, 8 ragged sequences of 16384 tokens 426 us,
// as long as the longest sequence's chain (about 7 us a step; the stores of dS, y and dV are 2 of
// them); key-vector gates, 4 x 2048 tokens 171 us.

#include "stq_chunk_pass.h"

namespace stq {
namespace {

// An upper triangular left operand (fragments at t in the order rows 0 (k steps 0, 1), 1 (0, 1),
// 2 (1), 3 (1); lo parts kTri further) times a column block; `undo` takes the block's scale
// away.  RLO: the block has a lo part (a block of bf16 values has none).
template <bool RLO>
__device__ inline void upper(lds_half t, const floatx4 (&X)[4], floatx4 (&Y)[4], float &undo) {
    const float s = scale_to(column_max(X), 13, undo);
    half8 hi, lo, f[4], f2[4];
    auto load = [&](half8 (&x)[4], int from) {       // of k step 1
        x[0] = frag(t + (from + 1) * kFrag);
        x[1] = frag(t + (from + 3) * kFrag);
        x[2] = frag(t + (from + 4) * kFrag);
        x[3] = frag(t + (from + 5) * kFrag);
    };
    auto mul2 = [&](half8 (&x)[4], half8 b) {        // of k step 0: rows 0 and 1
        Y[0] = mfma16(x[0], b, Y[0]);
        Y[1] = mfma16(x[1], b, Y[1]);
    };
    load(f, 0);
    right(X[2], X[3], s, hi, lo);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) Y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
    __builtin_amdgcn_sched_barrier(0);
    load(f2, kTri);
    mul4(f, hi, Y);
    if constexpr (RLO) mul4(f, lo, Y);
    __builtin_amdgcn_sched_barrier(0);
    f[0] = frag(t);
    f[1] = frag(t + 2 * kFrag);
    mul4(f2, hi, Y);
    right(X[0], X[1], s, hi, lo);
    __builtin_amdgcn_sched_barrier(0);
    f2[0] = frag(t + kTri * kFrag);
    f2[1] = frag(t + (kTri + 2) * kFrag);
    mul2(f, hi);
    if constexpr (RLO) mul2(f, lo);
    mul2(f2, hi);
    __builtin_amdgcn_sched_barrier(0);
}

template <int DK, int DV, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__((64 * 2 * PassShared<DK, KEYVEC, BF16, kReverse>::NW + 4 * DK))
    k_chunk_rev(const ChunkArgs A) {
    typedef PassShared<DK, KEYVEC, BF16, kReverse> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ, NW = Shared::NW;
    constexpr int parts = DV / (16 * NW);  // workgroups of a (sequence, head)
    __shared__ Shared sh;
    const int H = A.s.H;
    uint32_t seq, at_seq;
    xcd_place(blockIdx.x, H * parts, seq, at_seq);
    const int b = A.order ? A.order[seq] : seq, h = at_seq / parts, part = at_seq % parts;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    const int nc = (t1 - t0 + kC - 1) / kC;
    const size_t entry0 = (size_t)(t0 / kC + b) * H + h;
    const int wave = wave_index();

    if (wave >= 2 * NW) {
        if (nc == 0) return;
        Producer<DK, KEYVEC, BF16, kReverse> p;
        p.tid = threadIdx.x - 64 * 2 * NW;
        const uint32_t row_step = (uint32_t)(H * DV / 4);
        p.run(A, sh, h, t0, t1, nc, entry0,
              Shared::OUT ? static_cast<raw *>(A.dv) + (size_t)t0 * row_step + (size_t)h * (DV / 4) + part * Shared::GC
                          : nullptr,
              row_step);
        return;
    }

    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4, mine = wave < NW ? wave : wave - NW;
    const int col0 = (part * NW + mine) * 16;
    // lane (g, c16) reads and writes columns 4 (c16 / 4) .. + 3 of rows 16 rt + 4 g + c16 % 4
    const int row0 = 4 * g + (c16 & 3), out0 = slab_at<Shared::GC>(row0, 4 * mine + (c16 >> 2));
    const uint32_t row_step = (uint32_t)(H * DV / 4);    // in groups of four columns
    const size_t col4 = (size_t)h * (DV / 4) + col0 / 4;
    const uint32_t lane4 = c16 >> 2;     // (offsets of a lane stay 32 bits, bases in scalar registers)
    half8 f[4], f2[4];
    // The lane's numbers, formed anew in every step: what depends on them alone would be kept in
    // registers over the loop.
    auto anew = [](int x) {
        asm volatile("" : "+v"(x));
        return x;
    };

    if (wave >= NW) {                    // what dO gives to 16 columns
        if (nc == 0) return;
        raw v[4];                        // dO of the next chunk
        auto load_v = [&](int c) {
            const raw *base = static_cast<const raw *>(A.dout) + (size_t)(t0 + c * kC) * row_step + col4;
            const int n = t1 - t0 - c * kC, at = anew(row0);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) v[rt] = base[(uint32_t)min(16 * rt + at, n - 1) * row_step + lane4];
        };
        load_v(nc - 1);
        for (int i = 0; i < nc; ++i) {
            const int c = nc - 1 - i, n = t1 - t0 - c * kC, r16 = anew(c16);
            floatx4 D[4], y[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                float x[4];
                widen(v[rt], x);
                const bool on = 16 * rt + row0 < n;  // past the last token: 0
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = on ? x[r] : 0.f;
                quad_transpose(x);
#pragma unroll
                for (int r = 0; r < 4; ++r) D[rt][r] = x[r];
            }
            if (c > 0) load_v(c - 1);
            lds_barrier();
            const lds_float m = float_at(&sh.m[i & 1], 4 * g);
            float undo;
            upper<!BF16>(half_at(&sh.P, lane * 8), D, y, undo);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const floatx4 x = row_factors(m + factors(offsetof(ChunkMeta, rpt), rt)),
                              rq = row_factors(m + factors(offsetof(ChunkMeta, rq), rt));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    y[rt][r] = (y[rt][r] * x[r]) * undo;
                    D[rt][r] *= rq[r];
                }
                sh.pd[mine][rt][lane] = y[rt];
            }
            const float sd = scale_to(column_max(D), 13, undo);
            half8 dh[2], dl[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) right(D[2 * ks], D[2 * ks + 1], sd, dh[ks], dl[ks]);
            lds_half vb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) vb[j] = half_at(&sh.V, place_w(r16, g, j));
            auto load_c = [&](half8 (&x)[4], int l, int c0, int ks) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = frag(vb[j] + ((l * CT + c0 + j) * 2 + ks) * kFrag);
            };
            load_c(f, 0, 0, 0);
            columns_times<CT, NQ>(load_c, dh, dl, f, f2, [&](int ct, floatx4 z) { sh.zd[mine][ct][lane] = z * undo; });
            lds_barrier();
        }
        if constexpr (Shared::OUT) lds_barrier();
        return;
    }

    __builtin_amdgcn_s_setprio(3);       // the chain goes first where waves of a SIMD could both issue
    floatx4 S[CT];
    const size_t state0 = ((size_t)b * H + h) * DK * DV + col0;
    uint32_t at0 = 4 * g * DV + c16;     // of the lane's first value in the state
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[ct][r] = A.dlast ? (A.dlast + state0 + (16 * ct + r) * DV)[at0] : 0.f;
    asm volatile("" : "+v"(at0));

    for (int i = 0; i < nc; ++i) {
        const int c = nc - 1 - i, n = t1 - t0 - c * kC, r16 = anew(c16), at = anew(row0);
        const size_t entry = entry0 + (size_t)c * H;
        store_tiles(A.dS + entry * (DK * DV) + col0 * DK, S, CT);
        floatx4 R[4], y[4];
        float undo;
        const float s = scale_to(column_max(S), 13, undo);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
        lds_barrier();
        const lds_float m = float_at(&sh.m[i & 1], 4 * g);
        rows_times<KS, NK>([&](int ks) { return half_at(&sh.K, place_k(r16, g, ks)) + ks * kFrag; },
                           [&](int ks, half8 &hi, half8 &lo) { right(S[2 * ks], S[2 * ks + 1], s, hi, lo); }, R, f, f2);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rw = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) R[rt][r] = (R[rt][r] * rw[r]) * undo;
        }
        lds_barrier();
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] += sh.pd[mine][rt][lane];
        upper<true>(half_at(&sh.T, lane * 8), R, y, undo);
        raw *dv = static_cast<raw *>(A.dv) + (size_t)(t0 + c * kC) * row_step + col4;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rn = row_factors(m + factors(offsetof(ChunkMeta, rn), rt)),
                          be = row_factors(m + factors(offsetof(ChunkMeta, be), rt)),
                          rk = row_factors(m + factors(offsetof(ChunkMeta, rk), rt));
            float z[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[rt][r] = (y[rt][r] * rn[r]) * undo;
                z[r] = be[r] * y[rt][r];
                R[rt][r] = -z[r] * rk[r];
            }
            quad_transpose(z);
            raw out;
            narrow(z, out);
            if constexpr (Shared::OUT) sh.out[out0 + 16 * Shared::GC * rt] = out;
            else if (16 * rt + at < n) dv[(uint32_t)(16 * rt + at) * row_step + lane4] = out;
        }
        store_tiles(A.y + entry * (kC * DV) + col0 * kC, y, 4);
        const float su = scale_to(column_max(R), 13, undo);
        half8 kh[2], kl[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) right(R[2 * ks], R[2 * ks + 1], su, kh[ks], kl[ks]);
        lds_half wb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) wb[j] = half_at(&sh.W, place_w(r16, g, j));
        auto load_w = [&](half8 (&x)[4], int l, int c0, int ks) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = frag(wb[j] + ((l * CT + c0 + j) * 2 + ks) * kFrag);
        };
        load_w(f, 0, 0, 0);
        columns_times<CT, NK>(load_w, kh, kl, f, f2, [&](int ct, floatx4 z) {
            const floatx4 d = row_factors(m + factors(offsetof(ChunkMeta, dec), ct)), q = sh.zd[mine][ct][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) S[ct][r] = __builtin_fmaf(z[r], undo, __builtin_fmaf(S[ct][r], d[r], q[r]));
        });
    }
    if (Shared::OUT && nc) lds_barrier();  // the last rows are stored
    if (!A.dinitial) return;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) (A.dinitial + state0 + (16 * ct + r) * DV)[at0] = S[ct][r];
}

template <int DK, int DV, bool KEYVEC, bool BF16>
void go(const ChunkArgs &a, hipStream_t s) {
    constexpr int NW = PassShared<DK, KEYVEC, BF16, kReverse>::NW;
    const dim3 grid((unsigned)(DV / (16 * NW)) * (unsigned)a.s.H * (unsigned)a.s.B);
    k_chunk_rev<DK, DV, KEYVEC, BF16><<<grid, 64 * 2 * NW + 4 * DK, 0, s>>>(a);
}

template <int DK, int DV>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    if (keyvec && bf16) go<DK, DV, true, true>(a, s);
    else if (keyvec) go<DK, DV, true, false>(a, s);
    else if (bf16) go<DK, DV, false, true>(a, s);
    else go<DK, DV, false, false>(a, s);
}

}  // namespace

hipError_t launch_chunk_reverse(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && dv == 64) go<64, 64>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, 128>(a, keyvec, bf16, s);
    else if (dv == 64) go<128, 64>(a, keyvec, bf16, s);
    else go<128, 128>(a, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
