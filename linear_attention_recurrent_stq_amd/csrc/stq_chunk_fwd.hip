// The pass of the state through the chunks of a sequence (stq_chunk_forward; the first part
// of stq_chunk_backward).
//
// Per chunk, from T, P and the factors that the preparation left (stq_chunk.h):
//   R = V - (K G) S;   u = T R;   O = (Q G) S + P u;   S = diag(G_64) S + (K G_64/G)^T u.
//
// Columns of S are independent, so a wave carries 16 of them through the whole
// sequence: S stays in its registers, and no wave waits for another's columns.
// A result tile of the matrix instructions holds column l % 16 in lane l, which
// is where a right operand wants it, so S, R and u go from one product into the
// next without leaving the registers; only the order of a left operand's columns
// is permuted to match (4 g + e and 16 + 4 g + e in lane group g).
//
// What bounds it is the chain from one state to the next, R, u, S, or with enough sequences the
// reading of the left operands from LDS.  So the chain is all that a carrying wave does: a second
// wave forms the outputs of its columns, from S and u as fp16 fragments in LDS, (Q G) S beside
// R and P u a step later; and 4 d_k threads turn the next chunk's rows into the left operands,
// scaled fp16 fragments in LDS, the same for every column.  There is no second buffer: K and Q are read in
// the first half of a step, T, P and K^T in the second, and each half's are replaced while
// the other half runs (two barriers a step, which wait for LDS only).  Fragments are on
// their way while the ones before multiply.
//
// A workgroup takes 64 columns (32 where the fragments of fp32 rows leave no room); the others of
// a head find its rows in the same XCD's L2.  Longest sequences start first.  v and
// o are read and written four columns of a row a lane, and turned within quads of lanes.
#include <type_traits>

#include "stq_chunk_pass.h"

namespace stq {
namespace {

template <int DK, int DV, bool KEYVEC, bool BF16, Pass PASS>
__global__ void __launch_bounds__((64 * (PassShared<DK, KEYVEC, BF16, PASS>::NW + PassShared<DK, KEYVEC, BF16, PASS>::NH) +
                                   4 * DK)) k_chunk_fwd(const ChunkArgs A) {
    typedef PassShared<DK, KEYVEC, BF16, PASS> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ, NW = Shared::NW, NH = Shared::NH;
    constexpr bool FWD = PASS == kForward;
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

    if (wave >= NW + NH) {
        if (nc == 0) return;
        Producer<DK, KEYVEC, BF16, PASS> p;
        p.tid = threadIdx.x - 64 * (NW + NH);
        p.run(A, sh, h, t0, t1, nc, entry0);
        return;
    }

    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4, mine = wave < NW ? wave : wave - NW;
    const int col0 = (part * NW + mine) * 16;
    // lane (g, c16) reads and writes columns 4 (c16 / 4) .. + 3 of rows 16 rt + 4 g + c16 % 4
    const int row0 = 4 * g + (c16 & 3);
    const uint32_t row_step = (uint32_t)(H * DV / 4);    // in groups of four columns
    const size_t col4 = (size_t)h * (DV / 4) + col0 / 4 + (c16 >> 2);
    half8 f[4], f2[4];

    if constexpr (FWD) {
        if (wave >= NW) {                // the outputs of 16 columns
            if (nc == 0) return;
            floatx4 old[4], O[4], y[4];
            half8 uh[2], ul[2];
            float undo_u = 0.f;
            int which = 0, last = 0;
            for (int i = 0; i <= nc; ++i) {
                lds_barrier();
                const lds_float m = float_at(&sh.m[which], 4 * g);
                if (i > 0) {             // u of the step before
                    const lds_half p = half_at(&sh.uf, mine * (2 * kFrag) + lane * 8);
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        uh[ks] = frag(p + ks * kFrag);
                        if constexpr (NQ == 2) ul[ks] = frag(p + (NW * 2 + ks) * kFrag);
                    }
                    undo_u = sh.uu[mine][c16];
                }
                if (i < nc) {
                    const float undo = sh.us[mine][c16];
                    const lds_half sp = half_at(&sh.sf, mine * (KS * kFrag) + lane * 8);
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) O[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
                    auto place = [&](int ks) { return half_at(&sh.Q, place_k(c16, g, ks)) + ks * kFrag; };
                    if constexpr (NQ == 2) {
                        rows_times<KS, 2>(place, [&](int ks, half8 &hi, half8 &lo) {
                            hi = frag(sp + ks * kFrag);
                            lo = frag(sp + (NW * KS + ks) * kFrag);
                        }, O, f, f2);
                    } else {
                        half8 s[2];
                        s[0] = frag(sp);
                        load4(f, place(0), KS * kFrag);
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            __builtin_amdgcn_sched_barrier(0);
                            if (ks + 1 < KS) {
                                s[(ks + 1) & 1] = frag(sp + (ks + 1) * kFrag);
                                load4(ks & 1 ? f : f2, place(ks + 1), KS * kFrag);
                            }
                            mul4(ks & 1 ? f2 : f, s[ks & 1], O);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) {
                        const floatx4 rq = row_factors(m + factors(offsetof(ChunkMeta, rq), rt));
#pragma unroll
                        // (one factor after the other: their product may underflow where the value does not)
                        for (int r = 0; r < 4; ++r) O[rt][r] = (O[rt][r] * rq[r]) * undo;
                    }
                }
                lds_barrier();
                if (i > 0) {
                    const lds_half p = half_at(&sh.P, lane * 8);
                    const lds_float mp = float_at(&sh.m[last], 4 * g);
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int l = 0; l < NQ; ++l) {
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int rt = 2 * ks; rt < 4; ++rt) {
                                const half8 x = frag(p + (l * kTri + tri(rt, ks)) * kFrag);
                                y[rt] = mfma16(x, uh[ks], y[rt]);
                                if constexpr (NQ == 2)
                                    if (l == 0) y[rt] = mfma16(x, ul[ks], y[rt]);
                            }
                    }
                    raw *out = static_cast<raw *>(A.o) + (size_t)(t0 + (i - 1) * kC) * row_step + col4;
                    const int n = t1 - t0 - (i - 1) * kC;
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) {
                        const floatx4 pf = row_factors(mp + factors(offsetof(ChunkMeta, rp), rt));
                        float x[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(y[rt][r] * pf[r], undo_u, old[rt][r]);
                        quad_transpose(x);
                        raw z;
                        narrow(x, z);
                        if (16 * rt + row0 < n) out[(uint32_t)(16 * rt + row0) * row_step] = z;
                    }
                }
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) old[rt] = O[rt];
                last = which;
                which = which == 2 ? 0 : which + 1;
            }
            return;
        }
    }

    floatx4 S[CT];
    const size_t state0 = ((size_t)b * H + h) * DK * DV + col0;
    uint32_t at0 = 4 * g * DV + c16;     // of the lane's first value in the state
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[ct][r] = A.initial ? (A.initial + state0 + (16 * ct + r) * DV)[at0] : 0.f;
    asm volatile("" : "+v"(at0));        // (what is formed from it for the last states is formed there)

    raw v[4];                            // of the next chunk; past the last token its row again
    auto load_v = [&](int c) {
        const raw *base = static_cast<const raw *>(A.s.v) + (size_t)(t0 + c * kC) * row_step + col4;
        const int n = t1 - t0 - c * kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) v[rt] = base[(uint32_t)min(16 * rt + row0, n - 1) * row_step];
    };
    if (nc) load_v(0);
    float s, undo_s;                     // the state's scale
    auto publish = [&] {                 // the state as the helper's right operand
        s = scale_to(column_max(S), 13, undo_s);
        if constexpr (FWD) {
            _Float16 *to = &sh.sf[0][mine][0][lane * 8];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                half8 hi, lo;
                right(S[2 * ks], S[2 * ks + 1], s, hi, lo);
                *reinterpret_cast<half8 *>(to + ks * kFrag) = hi;
                if constexpr (NQ == 2) *reinterpret_cast<half8 *>(to + (NW * KS + ks) * kFrag) = lo;
            }
            if (g == 0) sh.us[mine][c16] = undo_s;
        }
    };
    publish();

    int which = 0;
    for (int c = 0; c < nc; ++c) {
        const size_t entry = entry0 + (size_t)c * H;
        if constexpr (!FWD) store_tiles(A.S + entry * (DK * DV) + col0 * DK, S, CT);
        floatx4 R[4], u[4];
        float undo;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
        lds_barrier();
        const lds_float m = float_at(&sh.m[which], 4 * g);
        rows_times<KS, NK>([&](int ks) { return half_at(&sh.K, place_k(c16, g, ks)) + ks * kFrag; },
                           [&](int ks, half8 &hi, half8 &lo) { right(S[2 * ks], S[2 * ks + 1], s, hi, lo); }, R, f, f2);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rk = row_factors(m + factors(offsetof(ChunkMeta, rk), rt));
            float x[4];
            widen(v[rt], x);
            quad_transpose(x);
#pragma unroll
            for (int r = 0; r < 4; ++r) R[rt][r] = __builtin_fmaf(-(R[rt][r] * rk[r]), undo_s, x[r]);
        }
        if (c + 1 < nc) load_v(c + 1);
        lds_barrier();
        const lds_half t = half_at(&sh.T, lane * 8);
        f[0] = frag(t);
        f[1] = frag(t + kFrag);
        f[2] = frag(t + 2 * kFrag);
        f[3] = frag(t + 4 * kFrag);
        lds_half wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[i] = half_at(&sh.W, place_w(c16, g, i));
        auto load_w = [&](half8 (&x)[4], int l, int c0, int ks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = frag(wb[i] + ((l * CT + c0 + i) * 2 + ks) * kFrag);
        };
        lower<true>(t, R, u, undo, f, f2, [&] { load_w(f, 0, 0, 0); });
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 x = row_factors(m + factors(offsetof(ChunkMeta, rt), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = (u[rt][r] * x[r]) * undo;
        }
        if constexpr (FWD) {             // u as the helper's right operand
            const float su = scale_to(column_max(u), 13, undo);
            _Float16 *to = &sh.uf[0][mine][0][lane * 8];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                half8 hi, lo;
                right(u[2 * ks], u[2 * ks + 1], su, hi, lo);
                *reinterpret_cast<half8 *>(to + ks * kFrag) = hi;
                if constexpr (NQ == 2) *reinterpret_cast<half8 *>(to + (NW * 2 + ks) * kFrag) = lo;
            }
            if (g == 0) sh.uu[mine][c16] = undo;
        } else {
            store_tiles(A.w + entry * (kC * DV) + col0 * kC, u, 4);
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 wf = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
            floatx4 be = wf;
            if constexpr (!FWD) be = row_factors(m + factors(offsetof(ChunkMeta, be), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = FWD ? u[rt][r] * wf[r] : (u[rt][r] * be[r]) * wf[r];
        }
        const float su = scale_to(column_max(u), 13, undo);
        half8 uh[2], ul[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) right(u[2 * ks], u[2 * ks + 1], su, uh[ks], ul[ks]);
        columns_times<CT, NK>(load_w, uh, ul, f, f2, [&](int ct, floatx4 z) {
            const floatx4 d = row_factors(m + factors(offsetof(ChunkMeta, dec), ct));
#pragma unroll
            for (int r = 0; r < 4; ++r) S[ct][r] = __builtin_fmaf(z[r], undo, S[ct][r] * d[r]);
        });
        publish();
        which = which == 2 ? 0 : which + 1;
    }
    if (FWD && nc) {                     // the helper's last step
        lds_barrier();
        lds_barrier();
    }
    if (!A.last) return;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) (A.last + state0 + (16 * ct + r) * DV)[at0] = S[ct][r];
}

template <int DK, int DV, bool KEYVEC, bool BF16, Pass PASS>
void go(const ChunkArgs &a, hipStream_t s) {
    typedef PassShared<DK, KEYVEC, BF16, PASS> Shared;
    const dim3 grid((unsigned)(DV / (16 * Shared::NW)) * (unsigned)a.s.H * (unsigned)a.s.B);
    k_chunk_fwd<DK, DV, KEYVEC, BF16, PASS><<<grid, 64 * (Shared::NW + Shared::NH) + 4 * DK, 0, s>>>(a);
}

template <int DK, int DV, Pass PASS>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    if (keyvec && bf16) go<DK, DV, true, true, PASS>(a, s);
    else if (keyvec) go<DK, DV, true, false, PASS>(a, s);
    else if (bf16) go<DK, DV, false, true, PASS>(a, s);
    else go<DK, DV, false, false, PASS>(a, s);
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
