// The passes of the state, or its gradient, through the chunks of a sequence: the producing
// waves, and what the multiplying waves share.  Device code only.
#pragma once

#include "stq_chunk.h"

namespace stq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMeta = sizeof(ChunkMeta) / 16;  // 16-byte pieces
constexpr int kPart = kTri * kFrag * 2 / 16;   // of a triangular matrix's hi or lo part

// Where lane (row, g)'s eight halves stand in a fragment: rows are permuted so
// that the producers' writes (fixed row, all g and k steps) and the readers'
// (fixed k step, all rows) both spread over the banks.
__device__ inline int place_k(int row16, int g, int ks) { return (g * 16 + (row16 ^ ((4 * g + ks) & 15))) * 8; }
__device__ inline int place_w(int ch16, int g, int ct) { return (g * 16 + (ch16 ^ (ct & 3))) * 8; }

// Four elements as they are in memory.
template <bool BF16> struct Raw4;
template <> struct Raw4<true> { typedef uint2 type; };
template <> struct Raw4<false> { typedef float4 type; };

__device__ inline void widen(uint2 w, float (&x)[4]) {
    x[0] = bf16_lo(w.x);
    x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y);
    x[3] = bf16_hi(w.y);
}
__device__ inline void widen(float4 w, float (&x)[4]) {
    x[0] = w.x;
    x[1] = w.y;
    x[2] = w.z;
    x[3] = w.w;
}
__device__ inline void narrow(const float (&x)[4], uint2 &w) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    union { bf16x2 v; uint32_t u; } a, b;
    a.v = bf16x2{(__bf16)x[0], (__bf16)x[1]};
    b.v = bf16x2{(__bf16)x[2], (__bf16)x[3]};
    w = make_uint2(a.u, b.u);
}
__device__ inline void narrow(const float (&x)[4], float4 &w) { w = make_float4(x[0], x[1], x[2], x[3]); }

// The passes over a sequence's chunks.  Every chunk (step i) has two halves, A and B, parted by
// barriers; what one half reads is replaced while the other half runs:
//   forward: A reads K, Q [token x channel] times the gates up to a token (before);
//            B reads K^T [channel x token] times those after it, T and P
//   carry:   A K before; B K^T after, T.  The state alone, no outputs
//   save:    as carry, N' in T's place.  Leaves each chunk's first state and delta errors w, which
//            the backward pass starts from
//   reverse: A K after, Q^T before, P^T; B K^T before, N^T.  The state's gradient, last chunk first
enum Pass { kForward, kCarry, kSave, kReverse };

// What a rule's operands carry.  All that a state or its gradient depends on keeps 22 bits:
// K (and Q^T) in the hi part alone where the rows are bf16 and not folded with gates.  Q and P of
// the forward pass reach the outputs only; for bf16 outputs (half a step: 2^-9) their hi
// parts, and those of what they multiply, are enough (2^-12).
//
// NW: columns of 16 of a workgroup, each with a wave that carries the state and (reverse) one that
// helps it: four, or two where what the helpers hand over leaves no room for four in LDS.
template <int DK, bool KEYVEC, bool BF16, Pass PASS>
struct PassShared {
    // (Every array on a 128-byte line: a wave's fragment that straddles one takes more cycles.  16 bytes off, the
    // carrying pass took 363 in place of 217 us.)
    static constexpr int NK = KEYVEC || !BF16 ? 2 : 1, KS = DK / 32, CT = DK / 16;
    static constexpr int NQ = PASS == kForward ? (BF16 ? 1 : 2) : NK;  // parts of Q
    static constexpr int NP = PASS == kForward ? NQ : 2;               // parts of P (P^T)
    static constexpr bool FWD = PASS == kForward, REV = PASS == kReverse;
    static constexpr int NW = DK == 128 && REV && NK == 2 ? 2 : 4;
    static constexpr int GC = 4 * NW;            // groups of four columns
    static constexpr bool OUT = BF16 && (FWD || REV);  // (see slab_at)
    alignas(128) _Float16 K[NK][4][KS][kFrag];
    alignas(128) _Float16 Q[FWD ? NQ : 1][FWD ? 4 : 1][FWD ? KS : 1][kFrag];
    alignas(128) u32x4 T[2 * kPart];                          // T, N' or N^T
    alignas(128) u32x4 P[FWD || REV ? NP * kPart : 1];        // P or P^T
    alignas(128) ChunkMeta m[2];                              // of even and of odd steps
    alignas(128) _Float16 W[NK][CT][2][kFrag];                // K^T
    alignas(128) _Float16 V[REV ? NQ : 1][REV ? CT : 1][REV ? 2 : 1][kFrag];  // Q^T
    // reverse, helper to carrier: P^T dO and (Q before)^T dO, as result tiles
    alignas(128) floatx4 pd[REV ? NW : 1][4][REV ? 64 : 1], zd[REV ? NW : 1][REV ? CT : 1][REV ? 64 : 1];
    alignas(128) typename Raw4<BF16>::type out[OUT ? kC * GC : 1];  // o or dv, on their way out
};

// COUNT pieces of 16 bytes, PT threads.
template <int COUNT, int PT>
struct Pieces {
    static constexpr int n = (COUNT + PT - 1) / PT;
    u32x4 x[n];
    __device__ inline void load(const void *from, int tid) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if ((i + 1) * PT <= COUNT || i * PT + tid < COUNT) x[i] = static_cast<const u32x4 *>(from)[i * PT + tid];
    }
    __device__ inline void store(u32x4 *to, int tid) const {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if ((i + 1) * PT <= COUNT || i * PT + tid < COUNT) to[i * PT + tid] = x[i];
    }
};

// bf16 outputs go through LDS: a lane has four columns of a row, and the producing threads store whole
// rows of the workgroup's columns, 16 bytes each.  (A wave's own 16 columns are 32 bytes of a row; stored
// from there they held up the chain for 3000 to 4000 of a step's 10000 cycles.  Measured: scalar gates, forward of 24000
// tokens 708 -> 684 us, backward of 16384 1238 -> 1208 us; key-vector gates the same.  Of fp32 rows they are
// 64 bytes, and it loses: backward of 700 tokens 95 -> 103 us.)  Groups of four columns are
// exchanged in pairs, so that 16 rows of one group spread over the banks.
template <int GC>
__device__ inline int slab_at(int row, int group) {
    return row * GC + (group ^ (2 * row & (GC - 1)));
}

// The producing waves: 4 DK threads; a thread takes 4 tokens x 4 channels.
template <int DK, bool KEYVEC, bool BF16, Pass PASS>
struct Producer {
    typedef PassShared<DK, KEYVEC, BF16, PASS> Shared;
    typedef typename Raw4<BF16>::type raw;
    static constexpr int NK = Shared::NK, NQ = Shared::NQ;
    static constexpr int PT = 4 * DK, CG = DK / 4;           // threads; channel groups
    static constexpr bool FWD = PASS == kForward, REV = PASS == kReverse, kQ = FWD || REV;
    raw k[4], q[kQ ? 4 : 1];
    float4 a[KEYVEC ? 4 : 1], pre, suf, sk, sq;
    Pieces<2 * kPart, PT> tm;        // T, N' or N^T
    Pieces<Shared::NP * kPart, PT> pm;  // P or P^T
    u32x4 meta;
    half4 w[NK][4];                  // K^T of the chunk whose A half is written
    int n;                           // tokens of the chunk in k, q and a
    int tid, cg, tg;

    // The workgroup's columns of the first `count` rows of a chunk, row_step groups of four apart.
    __device__ inline void store_out(const Shared &sh, raw *rows, uint32_t row_step, int count) {
        constexpr int per = BF16 ? 2 : 1, GC = Shared::GC, pieces = kC * GC / per;  // groups in 16 bytes
        constexpr int each = (pieces + PT - 1) / PT;
        u32x4 x[each];
#pragma unroll
        for (int i = 0; i < each; ++i) {
            const int p = i * PT + tid, row = p / (GC / per), group = p % (GC / per) * per;
            if ((i + 1) * PT <= pieces || p < pieces) x[i] = *reinterpret_cast<const u32x4 *>(&sh.out[slab_at<GC>(row, group)]);
        }
#pragma unroll
        for (int i = 0; i < each; ++i) {
            const int p = i * PT + tid, row = p / (GC / per), group = p % (GC / per) * per;
            if (p < pieces && row < count) *reinterpret_cast<u32x4 *>(rows + (uint32_t)row * row_step + group) = x[i];
        }
    }

    __device__ inline void fetch(const ChunkArgs &A, int h, int first, int n_, size_t entry) {
        n = n_;
        const ChunkPrep *e = A.prep + entry;
        const size_t base = ((size_t)first * A.s.H + h) * CG;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // past the last token its row again: T (N', N^T) and u have zeros there, so whatever
            // finite values stand there add nothing
            const uint32_t at = (uint32_t)min(4 * tg + i, n - 1) * (uint32_t)(A.s.H * CG) + cg;
            k[i] = (static_cast<const raw *>(A.s.k) + base)[at];
            if constexpr (kQ) q[i] = (static_cast<const raw *>(A.s.q) + base)[at];
            if constexpr (KEYVEC) a[i] = (reinterpret_cast<const float4 *>(A.s.a) + base)[at];
        }
        if constexpr (KEYVEC) {
            pre = *reinterpret_cast<const float4 *>(&A.gates[entry].pre[tg][4 * cg]);
            suf = *reinterpret_cast<const float4 *>(&A.gates[entry].suf[tg][4 * cg]);
        }
        sk = *reinterpret_cast<const float4 *>(&e->m.sk[4 * tg]);
        if constexpr (kQ) sq = *reinterpret_cast<const float4 *>(&e->m.sq[4 * tg]);
        if (tid < kMeta) meta = reinterpret_cast<const u32x4 *>(&e->m)[tid];
        if constexpr (REV) pm.load(A.back[entry].P, tid);
    }

    // Gate of the thread's token i: 1 past the last token.
    __device__ inline void gate(int i, float (&x)[4]) const {
        widen(a[KEYVEC ? i : 0], x);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = 4 * tg + i < n ? x[c] : 1.f;
    }

    // Where column c of the thread stands among the columns' fragments.
    __device__ inline int column(int c, int &ct) const {
        const int ch = 4 * cg + c;
        ct = ch >> 4;
        return place_w(ch & 15, tg & 3, ct) + ((tg >> 2) & 1) * 4;
    }

    // The chunk's A half into LDS, its K^T into w.
    __device__ inline void write_a(Shared &sh, int which) {
        float before[4], after[4][4];  // gate products up to and past a token
        if constexpr (KEYVEC) {
            widen(pre, before);
            float s[4];
            widen(suf, s);
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                float x[4];
                gate(i, x);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    after[i][c] = s[c];
                    s[c] *= x[c];
                }
            }
        }
        const int g = cg & 3, ks = cg >> 3, eh = ((cg >> 2) & 1) * 4, rt = tg >> 2;
        const float ek[4] = {sk.x, sk.y, sk.z, sk.w}, eq[4] = {sq.x, sq.y, sq.z, sq.w};
        half4 v[REV ? NQ : 1][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float kx[4], qx[4];
            widen(k[i], kx);
            if constexpr (kQ) widen(q[kQ ? i : 0], qx);
            if constexpr (KEYVEC) {
                float x[4];              // (of a token past the last one too: its row is not used)
                widen(a[i], x);
#pragma unroll
                for (int c = 0; c < 4; ++c) before[c] *= x[c];
            }
            half4 kh, kl, qh, ql;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                _Float16 hi, lo;
                if constexpr (NK == 2) {
                    // (ek is a power of two; the reverse pass, short of registers, spills where it comes first)
                    const float s = REV ? kx[c] : kx[c] * ek[i];
                    const float b = KEYVEC ? s * before[c] : s, f = KEYVEC ? s * after[i][c] : s;
                    if constexpr (REV) split(f, ek[i], hi, lo);
                    else split(b, hi, lo);
                    kh[c] = hi;
                    kl[c] = lo;
                    if constexpr (KEYVEC && REV) split(b, ek[i], hi, lo);
                    else if constexpr (KEYVEC) split(f, hi, lo);
                    w[0][c][i] = hi;
                    w[NK - 1][c][i] = lo;
                } else {
                    kh[c] = w[0][c][i] = (_Float16)(kx[c] * ek[i]);
                }
                if constexpr (kQ) {
                    split(KEYVEC ? qx[c] * before[c] : qx[c], eq[i], hi, lo);
                    qh[c] = hi;
                    ql[c] = lo;
                    if constexpr (REV) {
                        v[0][c][i] = hi;
                        if constexpr (NQ == 2) v[NQ - 1][c][i] = lo;
                    }
                }
            }
            const int at = place_k(4 * (tg & 3) + i, g, ks) + eh;
            *reinterpret_cast<half4 *>(&sh.K[0][rt][ks][at]) = kh;
            if constexpr (NK == 2) *reinterpret_cast<half4 *>(&sh.K[NK - 1][rt][ks][at]) = kl;
            if constexpr (FWD) {
                *reinterpret_cast<half4 *>(&sh.Q[0][rt][ks][at]) = qh;
                if constexpr (NQ == 2) *reinterpret_cast<half4 *>(&sh.Q[NQ - 1][rt][ks][at]) = ql;
            }
        }
        if constexpr (REV) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                int ct;
                const int at = column(c, ct);
#pragma unroll
                for (int l = 0; l < NQ; ++l) *reinterpret_cast<half4 *>(&sh.V[l][ct][tg >> 3][at]) = v[l][c];
            }
            pm.store(sh.P, tid);
        }
        if (tid < kMeta) reinterpret_cast<u32x4 *>(&sh.m[which])[tid] = meta;
    }

    __device__ inline void write_b(Shared &sh) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            int ct;
            const int at = column(c, ct);
#pragma unroll
            for (int l = 0; l < NK; ++l) *reinterpret_cast<half4 *>(&sh.W[l][ct][tg >> 3][at]) = w[l][c];
        }
        tm.store(sh.T, tid);
        if constexpr (FWD) pm.store(sh.P, tid);
    }

    // All of a producing thread's work on a sequence of nc chunks: step i is chunk i, or nc - 1 - i
    // in the reverse pass.  out: o (dv) from the first token and the workgroup's first column on, where it goes
    // through LDS.
    __device__ inline void run(const ChunkArgs &A, Shared &sh, int h, int t0, int t1, int nc, size_t entry0, raw *out,
                               uint32_t row_step) {
        cg = tid % CG;
        tg = tid / CG;
        auto chunk = [&](int i) { return REV ? nc - 1 - i : i; };
        auto entry = [&](int i) { return entry0 + (size_t)chunk(i) * A.s.H; };
        auto get = [&](int i) {
            const int c = chunk(i);
            fetch(A, h, t0 + c * kC, min(t1 - t0 - c * kC, kC), entry(i));
        };
        auto put = [&](int i) {
            const int c = chunk(i);
            store_out(sh, out + (size_t)c * kC * row_step, row_step, t1 - t0 - c * kC);
        };
        auto get_t = [&](int i) {
            if constexpr (REV) tm.load(A.back[entry(i)].N, tid);
            else tm.load(A.prep[entry(i)].T, tid);
            if constexpr (FWD) pm.load(A.prep[entry(i)].P, tid);
        };
        get(0);
        get_t(0);
        write_a(sh, 0);
        if (nc > 1) get(1);
        for (int i = 0; i < nc; ++i) {
            lds_barrier();               // half A of i stands; half B of i - 1 is done with
            write_b(sh);
            if (i + 1 < nc) get_t(i + 1);
            if constexpr (Shared::OUT)
                if (i > 0) put(i - 1);
            lds_barrier();               // half B of i stands; half A of i is done with
            if (i + 1 < nc) write_a(sh, (i + 1) & 1);
            if (i + 2 < nc) get(i + 2);
        }
        if constexpr (Shared::OUT) {
            lds_barrier();               // the last rows stand
            put(nc - 1);
        }
    }
};

// Places in LDS whose constant offsets go into the reading instructions.  They are
// formed anew where they are used: the compiler would otherwise keep the sums of place
// and offset, dozens of registers, over the whole loop.
typedef __attribute__((address_space(3))) const _Float16 *lds_half;
typedef __attribute__((address_space(3))) const float *lds_float;

__device__ inline lds_half half_at(const void *p, int at) {
    lds_half q = (lds_half)p + at;
    asm volatile("" : "+v"(q));
    return q;
}
__device__ inline lds_float float_at(const void *p, int at) {
    lds_float q = (lds_float)p + at;
    asm volatile("" : "+v"(q));
    return q;
}
__device__ inline half8 frag(lds_half p) { return *(__attribute__((address_space(3))) const half8 *)p; }

// Two result tiles (rows 16 m.. and 16 m + 16..) times s as a right operand.
__device__ inline void right(const floatx4 &x, const floatx4 &y, float s, half8 &hi, half8 &lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        _Float16 a, b;
        split(x[e], s, a, b);
        hi[e] = a;
        lo[e] = b;
        split(y[e], s, a, b);
        hi[4 + e] = a;
        lo[4 + e] = b;
    }
}

template <int n>
__device__ inline float column_max(const floatx4 (&x)[n]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(x[i][r]));
    return max_groups(m);
}

__device__ inline floatx4 row_factors(lds_float p) {
    return *(__attribute__((address_space(3))) const floatx4 *)p;
}
// Of the factors at `member` of ChunkMeta, those of row tile rt.
constexpr int factors(size_t member, int rt) { return (int)(member / sizeof(float)) + 16 * rt; }

// Four left fragments p + at(i), then their products: while a block of four multiplies, the
// next one is on its way from LDS.
__device__ inline void load4(half8 (&f)[4], lds_half p, int step, int first = 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i >= first) f[i] = frag(p + i * step);
}
__device__ inline void mul4(const half8 (&f)[4], half8 x, floatx4 (&Y)[4], int first = 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i >= first) Y[i] = mfma16(f[i], x, Y[i]);
}

// Blocks of four row tiles through all k steps: Y += (K hi + K lo) (x hi + x lo), rows KS * kFrag apart,
// K lo 4 rows further.  `place` gives the fragments of a k step, `operand` the right
// operand.
template <int KS, int NK, class P, class O>
__device__ inline void rows_times(P place, O operand, floatx4 (&Y)[4], half8 (&f)[4], half8 (&f2)[4]) {
    constexpr int row = KS * kFrag;
    half8 hi, lo;
    operand(0, hi, lo);
    lds_half at = place(0);
    load4(f, at, row);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const lds_half now = at;
        half8(&x0)[4] = NK == 1 && (ks & 1) ? f2 : f;
        half8(&x1)[4] = NK == 1 && (ks & 1) ? f : f2;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (NK == 2) load4(x1, now + 4 * row, row);
        if (ks + 1 < KS) at = place(ks + 1);
        if constexpr (NK == 1)
            if (ks + 1 < KS) load4(x1, at, row);
        __builtin_amdgcn_sched_barrier(0);
        mul4(x0, hi, Y);
        mul4(x0, lo, Y);
        if constexpr (NK == 2) {
            __builtin_amdgcn_sched_barrier(0);
            if (ks + 1 < KS) load4(x0, at, row);
            __builtin_amdgcn_sched_barrier(0);
            mul4(x1, hi, Y);
        }
        if (ks + 1 < KS) operand(ks + 1, hi, lo);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// A state's tile, or another's, as it stands in the registers: [tile][lane][4].
__device__ inline void store_tiles(float *to, const floatx4 *x, int n) {
    floatx4 *p = reinterpret_cast<floatx4 *>(to) + (threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < n; ++i) p[64 * i] = x[i];
}

// Columns of (K^T hi + K^T lo) (x hi + x lo): tile by tile, each given to `done`.  f: on entry
// the first block, on its way.
template <int CT, int NK, class L, class D>
__device__ inline void columns_times(L load, const half8 (&hi)[2], const half8 (&lo)[2], half8 (&f)[4], half8 (&f2)[4],
                                     D done) {
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
                load(f2, 1, c0, ks);
                __builtin_amdgcn_sched_barrier(0);
                mul4(f, hi[ks], z);
                mul4(f, lo[ks], z);
                __builtin_amdgcn_sched_barrier(0);
                if (more) load(f, 0, nc0, nks);
                __builtin_amdgcn_sched_barrier(0);
                mul4(f2, hi[ks], z);
            } else {
                if (more) load(ks ? f : f2, 0, nc0, nks);
                __builtin_amdgcn_sched_barrier(0);
                mul4(ks ? f2 : f, hi[ks], z);
                mul4(ks ? f2 : f, lo[ks], z);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) done(c0 + i, z[i]);
    }
}

// A lower triangular left operand (fragments at t, lo parts kTri further) times
// a column block; `undo` takes the block's scale away.  FULL: with the lo parts.
// f: the first block, on its way; `next` loads what comes after.
template <bool FULL, class F>
__device__ inline void lower(lds_half t, const floatx4 (&X)[4], floatx4 (&Y)[4], float &undo, half8 (&f)[4],
                             half8 (&f2)[4], F next) {
    const float s = scale_to(column_max(X), 13, undo);
    half8 hi, lo, hi1, lo1;
    right(X[0], X[1], s, hi, lo);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) Y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
    // fragments of k step 0: rows 0, 1 at 0, 1, rows 2, 3 at 2, 4; of k step 1: rows 2, 3 at 3, 5
    auto load = [&](half8 (&x)[4], int from) {
        x[0] = frag(t + from * kFrag);
        x[1] = frag(t + (from + 1) * kFrag);
        x[2] = frag(t + (from + 2) * kFrag);
        x[3] = frag(t + (from + 4) * kFrag);
    };
    auto load1 = [&](half8 (&x)[4], int from) {
        x[2] = frag(t + (from + 3) * kFrag);
        x[3] = frag(t + (from + 5) * kFrag);
    };
    if constexpr (FULL) {
        load(f2, kTri);
        __builtin_amdgcn_sched_barrier(0);
        mul4(f, hi, Y);
        mul4(f, lo, Y);
        __builtin_amdgcn_sched_barrier(0);
        load1(f, 0);
        __builtin_amdgcn_sched_barrier(0);
        right(X[2], X[3], s, hi1, lo1);
        mul4(f2, hi, Y);
        __builtin_amdgcn_sched_barrier(0);
        load1(f2, kTri);
        __builtin_amdgcn_sched_barrier(0);
        mul4(f, hi1, Y, 2);
        mul4(f, lo1, Y, 2);
        __builtin_amdgcn_sched_barrier(0);
        next();
        __builtin_amdgcn_sched_barrier(0);
        mul4(f2, hi1, Y, 2);
    } else {
        right(X[2], X[3], s, hi1, lo1);
        load1(f2, 0);
        mul4(f, hi, Y);
        next();
        mul4(f2, hi1, Y, 2);
    }
}

}  // namespace
}  // namespace stq
