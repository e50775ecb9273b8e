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
// What bounds it is the chain from one state to the next, R, u, S, in a step of about 4 us
// (d_k = d_v = 128), so nothing else stands in it: 4 d_k other threads turn the next chunk's rows
// into the left operands, scaled fp16 fragments in LDS, the same for every column.  There is no
// second buffer: K and Q are read in the first half of a step, T, P and K^T in the second, and each
// half's are replaced while the other half runs (two barriers a step, which wait for LDS only).
// Fragments are on their way while the ones before multiply.  (A second wave for the outputs,
// as the reverse pass has, was measured: scalar gates 485 against 483 us, key-vector gates, where the
// threads that fold the gates in then have too few registers, 407 against 468.)
//
// A workgroup takes 64 columns; the others of a head find its rows in the same XCD's L2.
// Longest sequences start first.  v and o are read and written four columns of a row a lane (bf16
// outputs by way of LDS), and turned within quads of lanes.
//
// Measured, bf16, d_k = d_v = 128, MI355X: scalar gates, 24 ragged sequences of 24000 tokens, 32
// heads 461 us; key-vector gates, 40 of 16001 tokens, 32 heads 408 us.  One sequence of 16384
// tokens, 16 heads, key-vector gates: 1063 us in one go (32 workgroups); in 5 segments 217 us for
// the segments' states and matrices, 14 us to join them, 259 us for the outputs.

#include "stq_chunk_pass.h"

namespace stq {
namespace {

// Chunks first .. last - 1 of a sequence of nc are its segment j of segs.
__device__ inline void segment(int nc, int segs, int j, int &first, int &last) {
    const int each = max((nc + segs - 1) / segs, kSegment);
    first = min(j * each, nc);
    last = min(first + each, nc);
}

// PASS: kForward; kCarry, which leaves what a segment makes of no state (the first segment: of the
// initial one) and of each unit vector; or kSave.
template <int DK, int DV, bool KEYVEC, bool BF16, Pass PASS>
__global__ void __launch_bounds__(256 + 4 * DK) k_chunk_fwd(const ChunkArgs A) {
    typedef PassShared<DK, KEYVEC, BF16, PASS> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ;
    constexpr bool FWD = PASS == kForward, SAVE = PASS == kSave, CARRY = PASS == kCarry;
    constexpr int parts = (CARRY ? DV + DK : DV) / 64;   // workgroups of a (sequence, head)
    __shared__ Shared sh;
    const int H = A.s.H, segs = SAVE ? 1 : A.segs, runs = CARRY ? segs - 1 : segs;
    uint32_t seq, at_seq;
    xcd_place(blockIdx.x, H * parts * runs, seq, at_seq);
    const int b = A.order ? A.order[seq] : seq, h = at_seq / parts % H, part = at_seq % parts, j = at_seq / (parts * H);
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    int nc = (t1 - t0 + kC - 1) / kC;
    size_t entry0 = (size_t)(t0 / kC + b) * H + h;
    bool ends = true;                    // with the sequence's last chunk
    if (!SAVE && segs > 1) {
        int first, last;
        segment(nc, segs, j, first, last);
        ends = last == nc && (j == 0 || first < nc);
        // nothing is left for the segment; or it is the last, or its part of a matrix that is not used
        if (CARRY ? ends || first == last || (j == 0 && part >= DV / 64) : j > 0 && first == nc) return;
        nc = last - first;
        entry0 += (size_t)first * H;
        t0 += first * kC;
        t1 = min(t1, t0 + nc * kC);
    }

    if (threadIdx.x >= 256) {
        if (nc == 0) return;
        Producer<DK, KEYVEC, BF16, PASS> p;
        p.tid = threadIdx.x - 256;
        const uint32_t row_step = (uint32_t)(H * DV / 4);
        p.run(A, sh, h, t0, t1, nc, entry0,
              Shared::OUT ? static_cast<raw *>(A.o) + (size_t)t0 * row_step + (size_t)h * (DV / 4) + part * Shared::GC
                          : nullptr,
              row_step);
        return;
    }

    const int lane = threadIdx.x & 63, wave = wave_index(), c16 = lane & 15, g = lane >> 4;
    const int col0 = (part * 4 + wave) * 16;
    const bool unit = CARRY && col0 >= DV;       // a column of the segment's matrix: no v
    const size_t head = (size_t)b * H + h;
    const float *from = A.initial ? A.initial + head * DK * DV : nullptr;
    if (FWD && segs > 1) from = A.starts + (head * segs + j) * (DK * DV);
    if (CARRY && j > 0) from = nullptr;
    floatx4 S[CT];
    uint32_t at0 = 4 * g * DV + c16;     // of the lane's first value in the state
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            S[ct][r] = from && !unit ? (from + col0 + (16 * ct + r) * DV)[at0] : 0.f;
            if (CARRY && unit) S[ct][r] = 16 * ct + 4 * g + r == col0 - DV + c16 ? 1.f : 0.f;
        }
    asm volatile("" : "+v"(at0));        // (what is formed from it for the last states is formed there)

    // lane (g, c16) reads and writes columns 4 (c16 / 4) .. + 3 of rows 16 rt + 4 g + c16 % 4
    const int row0 = 4 * g + (c16 & 3), out0 = slab_at<Shared::GC>(row0, 4 * wave + (c16 >> 2));
    const uint32_t row_step = (uint32_t)(H * DV / 4);    // in groups of four columns
    const size_t col4 = (size_t)h * (DV / 4) + col0 / 4 + (c16 >> 2);
    raw v[4];                            // of the next chunk; past the last token its row again
    auto load_v = [&](int c) {
        const raw *base = static_cast<const raw *>(A.s.v) + (size_t)(t0 + c * kC) * row_step + col4;
        const int n = t1 - t0 - c * kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) v[rt] = base[(uint32_t)min(16 * rt + row0, n - 1) * row_step];
    };
    if (nc && !unit) load_v(0);

    for (int c = 0; c < nc; ++c) {
        const size_t entry = entry0 + (size_t)c * H;
        if constexpr (SAVE) store_tiles(A.S + entry * (DK * DV) + col0 * DK, S, CT);
        floatx4 R[4], O[FWD ? 4 : 1];
        float undo;
        const float s = scale_to(column_max(S), 13, undo);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = O[FWD ? rt : 0] = floatx4{0.f, 0.f, 0.f, 0.f};
        half8 f[4], f2[4];
        lds_barrier();
        const lds_float m = float_at(&sh.m[c & 1], 4 * g);
        auto place = [&](int ks) { return half_at(&sh.K, place_k(c16, g, ks)) + ks * kFrag; };
        if constexpr (FWD) {
            half8 hi, lo;
            right(S[0], S[1], s, hi, lo);
            lds_half kq = place(0);
            constexpr int row = KS * kFrag, q_at = 4 * row * NK;  // steps to the next row tile, to Q
            load4(f, kq, row);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                // K hi, Q hi, K lo, Q lo (as far as there are), each on its way while the one before multiplies
                constexpr int blocks = NK + NQ;
                const lds_half now = kq;
                auto ahead = [&](int block, half8 (&x)[4]) {  // block of this k step, or the next one's first
                    if (block == blocks) {
                        if (ks + 1 < KS) {
                            kq = place(ks + 1);
                            load4(x, kq, row);
                        }
                    } else {
                        load4(x, now + (block == 1   ? q_at
                                        : block == 3 ? q_at + 4 * row
                                        : NK == 2    ? 4 * row
                                                     : q_at + 4 * row),
                              row);
                    }
                };
                constexpr bool flip = blocks & 1;  // the first block of odd k steps is then in f2
                half8(&x0)[4] = flip && (ks & 1) ? f2 : f;
                half8(&x1)[4] = flip && (ks & 1) ? f : f2;
                __builtin_amdgcn_sched_barrier(0);
                ahead(1, x1);
                mul4(x0, hi, R);
                mul4(x0, lo, R);
                __builtin_amdgcn_sched_barrier(0);
                ahead(2, x0);
                mul4(x1, hi, O);
                if constexpr (NQ == 2) mul4(x1, lo, O);
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
        } else {
            rows_times<KS, NK>(place, [&](int ks, half8 &hi, half8 &lo) { right(S[2 * ks], S[2 * ks + 1], s, hi, lo); },
                               R, f, f2);
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rk = row_factors(m + factors(offsetof(ChunkMeta, rk), rt)),
                          rq = FWD ? row_factors(m + factors(offsetof(ChunkMeta, rq), rt)) : rk;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (!unit) {
                widen(v[rt], x);
                quad_transpose(x);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // (one factor after the other: their product may underflow where the value does not)
                R[rt][r] = __builtin_fmaf(-(R[rt][r] * rk[r]), undo, x[r]);
                if constexpr (FWD) O[rt][r] = (O[rt][r] * rq[r]) * undo;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (c + 1 < nc && !unit) load_v(c + 1);
        lds_barrier();
        floatx4 u[4];
        const lds_half t = half_at(&sh.T, lane * 8), p = half_at(&sh.P, lane * 8);
        f[0] = frag(t);
        f[1] = frag(t + kFrag);
        f[2] = frag(t + 2 * kFrag);
        f[3] = frag(t + 4 * kFrag);
        lds_half wb[4];
        auto load_w = [&](half8 (&x)[4], int l, int c0, int ks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = frag(wb[i] + ((l * CT + c0 + i) * 2 + ks) * kFrag);
        };
        auto place_wb = [&] {
#pragma unroll
            for (int i = 0; i < 4; ++i) wb[i] = half_at(&sh.W, place_w(c16, g, i));
        };
        if constexpr (!FWD) place_wb();
        lower<true>(t, R, u, undo, f, f2, [&] {
            if constexpr (FWD) {
                f[0] = frag(p);
                f[1] = frag(p + kFrag);
                f[2] = frag(p + 2 * kFrag);
                f[3] = frag(p + 4 * kFrag);
            } else {
                load_w(f, 0, 0, 0);
            }
        });
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 x = row_factors(m + factors(offsetof(ChunkMeta, rt), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = (u[rt][r] * x[r]) * undo;
        }
        if constexpr (SAVE) store_tiles(A.w + entry * (kC * DV) + col0 * kC, u, 4);
        if constexpr (FWD) {
            floatx4 y[4];
            place_wb();
            lower<NQ == 2>(p, u, y, undo, f, f2, [&] { load_w(f, 0, 0, 0); });
            __builtin_amdgcn_sched_barrier(0);
            raw *out = static_cast<raw *>(A.o) + (size_t)(t0 + c * kC) * row_step + col4;
            const int n = t1 - t0 - c * kC;
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const floatx4 pf = row_factors(m + factors(offsetof(ChunkMeta, rp), rt));
                float x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(y[rt][r] * pf[r], undo, O[rt][r]);
                quad_transpose(x);
                raw z;
                narrow(x, z);
                if constexpr (Shared::OUT) sh.out[out0 + 16 * Shared::GC * rt] = z;
                else if (16 * rt + row0 < n) out[(uint32_t)(16 * rt + row0) * row_step] = z;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 wf = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
            floatx4 be = wf;
            if constexpr (SAVE) be = row_factors(m + factors(offsetof(ChunkMeta, be), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = SAVE ? (u[rt][r] * be[r]) * wf[r] : u[rt][r] * wf[r];
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
    }
    if (Shared::OUT && nc) lds_barrier();  // the last rows are stored
    if constexpr (CARRY) {
        float *to = A.steps + (head * runs + j) * (DK * (DV + DK)) + col0;
        uint32_t at = 4 * g * (DV + DK) + c16;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r) (to + (16 * ct + r) * (DV + DK))[at] = S[ct][r];
        return;
    }
    if (!A.last || !ends) return;
    float *to = A.last + head * DK * DV + col0;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) (to + (16 * ct + r) * DV)[at0] = S[ct][r];
}

// The states before a sequence's segments, S_j+1 = M_j S_j + L_j, by fp32 matrix instructions (16x16x4).  A
// workgroup of four waves takes 16 columns, a wave d_k / 4 of their rows; a lane reads four
// neighbours of a row of M, which belong to four instructions, so it takes S's rows in that order.
// The state before the first segment is written too: the passes may write the last states
// over the initial ones.
template <int DK, int DV>
__global__ void __launch_bounds__(256) k_chunk_join(const ChunkArgs A) {
    constexpr int CT = DK / 16, RT = CT / 4;
    __shared__ float cur[2][DK][17];
    const int H = A.s.H, segs = A.segs, part = blockIdx.x % (DV / 16);
    const int head = blockIdx.x / (DV / 16), b = head / H;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    const int nc = (t1 - t0 + kC - 1) / kC;
    const int lane = threadIdx.x & 63, wave = wave_index(), c16 = lane & 15, g = lane >> 4;
    const float *from = A.initial ? A.initial + (size_t)head * DK * DV : nullptr;
    floatx4 S[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = from ? from[(16 * (wave * RT + i) + 4 * g + r) * DV + 16 * part + c16] : 0.f;
    for (int j = 0;; ++j) {
        float *to = A.starts + ((size_t)head * segs + j) * (DK * DV);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * (wave * RT + i) + 4 * g + r;
                to[row * DV + 16 * part + c16] = S[i][r];
                cur[j & 1][row][c16] = S[i][r];
            }
        int first, last;
        segment(nc, segs, j, first, last);
        if (last >= nc) return;          // (all waves of the workgroup)
        __syncthreads();
        const float *step = A.steps + ((size_t)head * (segs - 1) + j) * (DK * (DV + DK));
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int rt = wave * RT + i;
            floatx4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = step[(16 * rt + 4 * g + r) * (DV + DK) + 16 * part + c16];
            if (j > 0) {                 // the first segment began with the initial state itself
                const float *row = step + (16 * rt + c16) * (DV + DK) + DV + 4 * g;
                floatx4 a[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) a[ct] = *reinterpret_cast<const floatx4 *>(row + 16 * ct);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x = __builtin_amdgcn_mfma_f32_16x16x4f32(a[ct][r], cur[j & 1][16 * ct + 4 * g + r][c16], x, 0, 0, 0);
            }
            S[i] = x;
        }
    }
}

template <int DK, int DV, bool KEYVEC, bool BF16, Pass PASS>
void run(const ChunkArgs &a, hipStream_t s) {
    const unsigned parts = (PASS == kCarry ? DV + DK : DV) / 64, runs = PASS == kCarry ? a.segs - 1 : PASS == kSave ? 1 : a.segs;
    k_chunk_fwd<DK, DV, KEYVEC, BF16, PASS><<<parts * runs * (unsigned)a.s.H * (unsigned)a.s.B, 256 + 4 * DK, 0, s>>>(a);
}

template <int DK, int DV, bool KEYVEC, bool BF16>
void go(const ChunkArgs &a, hipStream_t s) {
    if (a.back) {
        run<DK, DV, KEYVEC, BF16, kSave>(a, s);
        return;
    }
    if (a.segs > 1) {
        run<DK, DV, KEYVEC, BF16, kCarry>(a, s);
        k_chunk_join<DK, DV><<<(unsigned)(DV / 16) * (unsigned)a.s.H * (unsigned)a.s.B, 256, 0, s>>>(a);
    }
    run<DK, DV, KEYVEC, BF16, kForward>(a, s);
}

template <int DK, int DV>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    if (keyvec && bf16) go<DK, DV, true, true>(a, s);
    else if (keyvec) go<DK, DV, true, false>(a, s);
    else if (bf16) go<DK, DV, false, true>(a, s);
    else go<DK, DV, false, false>(a, s);
}

}  // namespace

hipError_t launch_chunk_forward(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && dv == 64) go<64, 64>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, 128>(a, keyvec, bf16, s);
    else if (dv == 64) go<128, 64>(a, keyvec, bf16, s);
    else go<128, 128>(a, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
