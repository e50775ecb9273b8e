// The pass of the state through the chunks of a sequence (stq_chunk_forward).
//
// Per chunk, from T, P and the factors that k_chunk_prep left (stq_chunk.h):
//   R = V - (K G) S;   u = T R;   O = (Q G) S + P u;   S = diag(G_64) S + (K G_64/G)^T u.
//
// Columns of S are independent, so a wave owns 16 of them for the whole
// sequence: S stays in its registers, and no wave waits for another's values.
// A result tile of the matrix instructions holds column l % 16 in lane l, which
// is where a right operand wants it, so S, R and u go from one product into the
// next without leaving the registers; only the order of a left operand's columns
// is permuted to match (4 g + e and 16 + 4 g + e in lane group g).
//
// The left operands K, Q, T, P and K^T are the same for every wave.  Four
// waves more (4 d_k threads) turn the next chunk's rows into scaled fp16 fragments in LDS
// while the others multiply.  The fragments need no second buffer: K and Q are
// read in the first half of a chunk, T, P and K^T in the second, and each half's are
// replaced while the other half runs (two barriers a chunk, which wait for
// LDS only).
//
// A workgroup takes 64 columns with four multiplying waves, so that the twelve waves of a
// head of 128 keep 168 registers each; two workgroups take a head of 128
// columns and find its rows in the same XCD's L2.  Longest sequences start first.
//
// v and o are read and written four columns of a row a lane, and turned within
// quads of lanes.
#include <type_traits>

#include "stq_chunk_pass.h"

namespace stq {
namespace {

// PASS: kForward, or kSave, which leaves every chunk's first state and delta errors
// w = R - A u (u = beta w) instead of the outputs.
template <int DK, int DV, bool KEYVEC, bool BF16, Pass PASS>
__global__ void __launch_bounds__(256 + 4 * DK) k_chunk_fwd(const ChunkArgs A) {
    typedef PassShared<DK, KEYVEC, BF16, PASS> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ;
    constexpr bool FWD = PASS == kForward;
    constexpr int parts = DV / 64;       // workgroups of a (sequence, head)
    __shared__ Shared sh;
    const int H = A.s.H;
    uint32_t seq, at_seq;
    xcd_place(blockIdx.x, H * parts, seq, at_seq);
    const int b = A.order ? A.order[seq] : seq, h = at_seq / parts, part = at_seq % parts;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    const int nc = (t1 - t0 + kC - 1) / kC;

    if (threadIdx.x >= 256) {
        if (nc == 0) return;
        Producer<DK, KEYVEC, BF16, PASS> p;
        p.tid = threadIdx.x - 256;
        p.run(A, sh, h, t0, t1, nc, (size_t)(t0 / kC + b) * H + h);
        return;
    }

    const int lane = threadIdx.x & 63, wave = wave_index(), c16 = lane & 15, g = lane >> 4;
    const int col0 = (part * 4 + wave) * 16;
    floatx4 S[CT];
    const size_t state0 = ((size_t)b * H + h) * DK * DV + col0;
    uint32_t at0 = 4 * g * DV + c16;     // of the lane's first value in the state
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[ct][r] = A.initial ? (A.initial + state0 + (16 * ct + r) * DV)[at0] : 0.f;
    asm volatile("" : "+v"(at0));        // (what is formed from it for the last states is formed there)

    // lane (g, c16) reads and writes columns 4 (c16 / 4) .. + 3 of rows 16 rt + 4 g + c16 % 4
    const int row0 = 4 * g + (c16 & 3);
    const uint32_t row_step = (uint32_t)(H * DV / 4);    // in groups of four columns
    const size_t col4 = (size_t)h * (DV / 4) + col0 / 4 + (c16 >> 2);
    raw v[4];                            // of the next chunk; past the last token its row again
    auto load_v = [&](int c) {
        const raw *base = static_cast<const raw *>(A.s.v) + (size_t)(t0 + c * kC) * row_step + col4;
        const int n = t1 - t0 - c * kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) v[rt] = base[(uint32_t)min(16 * rt + row0, n - 1) * row_step];
    };
    if (nc) load_v(0);

    for (int c = 0; c < nc; ++c) {
        const size_t entry = (size_t)(t0 / kC + b + c) * H + h;
        if constexpr (!FWD) {
            float *to = A.S + entry * (DK * DV) + col0;
            uint32_t at = 4 * g * DV + c16;
            asm volatile("" : "+v"(at));
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int r = 0; r < 4; ++r) (to + (16 * ct + r) * DV)[at] = S[ct][r];
        }
        floatx4 R[4], O[4];
        float undo;
        const float s = scale_to(column_max(S), 13, undo);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = O[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
        half8 hi, lo, f[4], f2[4];
        right(S[0], S[1], s, hi, lo);
        lds_barrier();
        const lds_float m = float_at(&sh.m[c & 1], 4 * g);
        auto place = [&](int ks) { return half_at(&sh.K, place_k(c16, g, ks)) + ks * kFrag; };
        lds_half kq = place(0);
        constexpr int row = KS * kFrag, q_at = 4 * row * NK;  // steps to the next row tile, to Q
        load4(f, kq, row);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // K hi, Q hi, K lo, Q lo (as far as there are), each on its way while the one before multiplies
            constexpr int blocks = FWD ? NK + NQ : NK;
            const lds_half now = kq;
            auto ahead = [&](int block, half8 (&x)[4]) {  // block of this k step, or the next one's first
                if (block == blocks) {
                    if (ks + 1 < KS) {
                        kq = place(ks + 1);
                        load4(x, kq, row);
                    }
                } else if (FWD) {
                    load4(x, now + (block == 1 ? q_at : block == 3 ? q_at + 4 * row : NK == 2 ? 4 * row : q_at + 4 * row),
                          row);
                } else {
                    load4(x, now + 4 * row, row);
                }
            };
            constexpr bool flip = blocks & 1;  // the first block of odd k steps is then in f2
            half8(&x0)[4] = flip && (ks & 1) ? f2 : f;
            half8(&x1)[4] = flip && (ks & 1) ? f : f2;
            __builtin_amdgcn_sched_barrier(0);
            ahead(1, x1);
            mul4(x0, hi, R);
            mul4(x0, lo, R);
            if constexpr (blocks > 1) {
                __builtin_amdgcn_sched_barrier(0);
                ahead(2, x0);
                if constexpr (FWD) {
                    mul4(x1, hi, O);
                    if constexpr (NQ == 2) mul4(x1, lo, O);
                } else {
                    mul4(x1, hi, R);
                }
            }
            if constexpr (blocks > 2) {
                __builtin_amdgcn_sched_barrier(0);
                ahead(3, x1);
                mul4(x0, hi, R);
            }
            if constexpr (blocks > 3) {
                __builtin_amdgcn_sched_barrier(0);
                ahead(4, x0);
                mul4(x1, hi, O);
            }
            if (ks + 1 < KS) right(S[2 * ks + 2], S[2 * ks + 3], s, hi, lo);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rk = row_factors(m + factors(offsetof(ChunkMeta, rk), rt)),
                          rq = FWD ? row_factors(m + factors(offsetof(ChunkMeta, rq), rt)) : rk;
            float x[4];
            widen(v[rt], x);
            quad_transpose(x);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // (one factor after the other: their product may underflow where the value does not)
                R[rt][r] = __builtin_fmaf(-(R[rt][r] * rk[r]), undo, x[r]);
                if constexpr (FWD) O[rt][r] = (O[rt][r] * rq[r]) * undo;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (c + 1 < nc) load_v(c + 1);
        lds_barrier();
        floatx4 u[4], y[4];
        const lds_half t = half_at(&sh.tp, lane * 8), p = t + 2 * kTri * kFrag;
        f[0] = frag(t);
        f[1] = frag(t + kFrag);
        f[2] = frag(t + 2 * kFrag);
        f[3] = frag(t + 4 * kFrag);
        lower<true>(t, R, u, undo, f, f2, [&] {
            f[0] = frag(p);
            f[1] = frag(p + kFrag);
            f[2] = frag(p + 2 * kFrag);
            f[3] = frag(p + 4 * kFrag);
        });
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 x = row_factors(m + factors(offsetof(ChunkMeta, rt), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = (u[rt][r] * x[r]) * undo;
        }
        lds_half wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[i] = half_at(&sh.W, place_w(c16, g, i));
        auto load_w = [&](half8 (&x)[4], int l, int c0, int ks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = frag(wb[i] + ((l * CT + c0 + i) * 2 + ks) * kFrag);
        };
        lower<!FWD || NQ == 2>(p, u, y, undo, f, f2, [&] { load_w(f, 0, 0, 0); });
        __builtin_amdgcn_sched_barrier(0);
        typedef typename std::conditional<FWD, raw, float4>::type out_t;
        out_t *out = FWD ? static_cast<out_t *>(A.o) + (size_t)(t0 + c * kC) * row_step + col4
                         : reinterpret_cast<out_t *>(A.w) + entry * (kC * DV / 4) + col0 / 4 + (c16 >> 2);
        const uint32_t out_step = FWD ? row_step : DV / 4;
        const int n = FWD ? t1 - t0 - c * kC : kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 pf = row_factors(m + factors(offsetof(ChunkMeta, rp), rt)),
                          wf = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = __builtin_fmaf(FWD ? y[rt][r] * pf[r] : -(y[rt][r] * pf[r]), undo, FWD ? O[rt][r] : R[rt][r]);
                u[rt][r] *= wf[r];
            }
            quad_transpose(x);
            out_t z;
            narrow(x, z);
            if (16 * rt + row0 < n) out[(uint32_t)(16 * rt + row0) * out_step] = z;
            __builtin_amdgcn_sched_barrier(0);
        }
        const float su = scale_to(column_max(u), 13, undo);
        half8 uh[2], ul[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) right(u[2 * ks], u[2 * ks + 1], su, uh[ks], ul[ks]);
#pragma unroll
        for (int c0 = 0; c0 < CT; c0 += 4) {
            floatx4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                __builtin_amdgcn_sched_barrier(0);
                const bool more = ks == 0 || c0 + 4 < CT;
                const int nc0 = ks ? c0 + 4 : c0, nks = ks ? 0 : 1;
                if constexpr (NK == 2) {
                    load_w(f2, 1, c0, ks);
                    mul4(f, uh[ks], z);
                    mul4(f, ul[ks], z);
                    __builtin_amdgcn_sched_barrier(0);
                    if (more) load_w(f, 0, nc0, nks);
                    mul4(f2, uh[ks], z);
                } else {
                    if (more) load_w(ks ? f : f2, 0, nc0, nks);
                    mul4(ks ? f2 : f, uh[ks], z);
                    mul4(ks ? f2 : f, ul[ks], z);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const floatx4 d = row_factors(m + factors(offsetof(ChunkMeta, dec), c0 + i));
#pragma unroll
                for (int r = 0; r < 4; ++r) S[c0 + i][r] = __builtin_fmaf(z[i][r], undo, S[c0 + i][r] * d[r]);
            }
        }
    }
    if (!A.last) return;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) (A.last + state0 + (16 * ct + r) * DV)[at0] = S[ct][r];
}

template <int DK, int DV, Pass PASS>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)(DV / 64) * (unsigned)a.s.H * (unsigned)a.s.B);
    constexpr int block = 256 + 4 * DK;
    if (keyvec && bf16) k_chunk_fwd<DK, DV, true, true, PASS><<<grid, block, 0, s>>>(a);
    else if (keyvec) k_chunk_fwd<DK, DV, true, false, PASS><<<grid, block, 0, s>>>(a);
    else if (bf16) k_chunk_fwd<DK, DV, false, true, PASS><<<grid, block, 0, s>>>(a);
    else k_chunk_fwd<DK, DV, false, false, PASS><<<grid, block, 0, s>>>(a);
}

template <Pass PASS>
void go(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && dv == 64) go<64, 64, PASS>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, 128, PASS>(a, keyvec, bf16, s);
    else if (dv == 64) go<128, 64, PASS>(a, keyvec, bf16, s);
    else go<128, 128, PASS>(a, keyvec, bf16, s);
}

}  // namespace

hipError_t launch_chunk_forward(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (a.back) go<kSave>(a, dk, dv, keyvec, bf16, s);
    else go<kForward>(a, dk, dv, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
