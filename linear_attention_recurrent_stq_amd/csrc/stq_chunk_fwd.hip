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
#include "stq_chunk.h"

namespace stq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMeta = sizeof(ChunkMeta) / 16;  // 16-byte pieces
constexpr int kPart = kTri * kFrag * 2 / 16;   // of T's or P's hi or lo part

// What a rule's operands carry.  K and T, which the state depends on, always
// keep 22 bits: K in its hi part alone where it is bf16 and not folded with gates.  Q
// and P reach the outputs only; for bf16 outputs (half a step: 2^-9) their hi
// parts, and those of what they multiply, are enough (2^-12).
template <int DK, bool KEYVEC, bool BF16>
struct FwdShared {
    static constexpr int NK = KEYVEC || !BF16 ? 2 : 1, NQ = BF16 ? 1 : 2, KS = DK / 32, CT = DK / 16;
    static constexpr int TP = (2 + NQ) * kPart;  // 16-byte pieces of T hi, T lo, P hi (, P lo)
    _Float16 K[NK][4][KS][kFrag], Q[NQ][4][KS][kFrag];
    u32x4 tp[TP];
    ChunkMeta m[2];                  // of even and of odd chunks
    _Float16 W[NK][CT][2][kFrag];
};

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

// The producing waves: 4 DK threads; a thread takes 4 tokens x 4 channels.
template <int DK, bool KEYVEC, bool BF16>
struct Producer {
    typedef FwdShared<DK, KEYVEC, BF16> Shared;
    typedef typename Raw4<BF16>::type raw;
    static constexpr int NK = Shared::NK, NQ = Shared::NQ, TP = Shared::TP;
    static constexpr int PT = 4 * DK, CG = DK / 4;           // threads; channel groups
    raw k[4], q[4];
    float4 a[KEYVEC ? 4 : 1], pre, suf, sk, sq;
    u32x4 tp0, tp1, tp2, tp3, tp4, tp5, meta;
    half4 w[NK][4];                  // K^T fragments of the chunk whose K and Q are written
    int n;                           // tokens of the chunk in k, q and a
    int tid, cg, tg;

    __device__ inline void load(const ChunkArgs &A, int h, int first, int n_, size_t entry) {
        n = n_;
        const ChunkPrep *e = A.prep + entry;
        const size_t base = ((size_t)first * A.s.H + h) * CG;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // past the last token its row again: T has zeros in those columns and rows,
            // so whatever finite values stand there add nothing
            const uint32_t at = (uint32_t)min(4 * tg + i, n - 1) * (uint32_t)(A.s.H * CG) + cg;
            k[i] = (static_cast<const raw *>(A.s.k) + base)[at];
            q[i] = (static_cast<const raw *>(A.s.q) + base)[at];
            if constexpr (KEYVEC) a[i] = (reinterpret_cast<const float4 *>(A.s.a) + base)[at];
        }
        if constexpr (KEYVEC) {
            pre = *reinterpret_cast<const float4 *>(&A.gates[entry].pre[tg][4 * cg]);
            suf = *reinterpret_cast<const float4 *>(&A.gates[entry].suf[tg][4 * cg]);
        }
        sk = *reinterpret_cast<const float4 *>(&e->m.sk[4 * tg]);
        sq = *reinterpret_cast<const float4 *>(&e->m.sq[4 * tg]);
        if (tid < kMeta) meta = reinterpret_cast<const u32x4 *>(&e->m)[tid];
    }

    // f(piece, its number) over this thread's pieces of T and P
    template <class F>
    __device__ inline void pieces(F f) {
        f(tp0, tid);
        f(tp1, tid + PT);
        if (3 * PT <= TP || tid + 2 * PT < TP) f(tp2, tid + 2 * PT);
        if constexpr (3 * PT < TP) f(tp3, tid + 3 * PT);
        if constexpr (4 * PT < TP)
            if (5 * PT <= TP || tid + 4 * PT < TP) f(tp4, tid + 4 * PT);
        if constexpr (5 * PT < TP) f(tp5, tid + 5 * PT);
    }

    __device__ inline void load_tp(const ChunkPrep *e) {
        pieces([&](u32x4 &x, int i) { x = reinterpret_cast<const u32x4 *>(e)[i]; });
    }

    // Gate of the thread's token i: 1 past the last token.
    __device__ inline void gate(int i, float (&x)[4]) const {
        widen(a[KEYVEC ? i : 0], x);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = 4 * tg + i < n ? x[c] : 1.f;
    }

    // K and Q of the chunk into LDS, its K^T into w.
    __device__ inline void write_kq(Shared &sh, int which) {
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float kx[4], qx[4];
            widen(k[i], kx);
            widen(q[i], qx);
            if constexpr (KEYVEC) {
                float x[4];
                gate(i, x);
#pragma unroll
                for (int c = 0; c < 4; ++c) before[c] *= x[c];
            }
            half4 kh, kl, qh, ql;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                _Float16 hi, lo;
                if constexpr (NK == 2) {
                    split(KEYVEC ? kx[c] * before[c] : kx[c], ek[i], hi, lo);
                    kh[c] = hi;
                    kl[c] = lo;
                    if constexpr (KEYVEC) split(kx[c] * after[i][c], ek[i], hi, lo);
                    w[0][c][i] = hi;
                    w[NK - 1][c][i] = lo;
                } else {
                    kh[c] = w[0][c][i] = (_Float16)(kx[c] * ek[i]);
                }
                split(KEYVEC ? qx[c] * before[c] : qx[c], eq[i], hi, lo);
                qh[c] = hi;
                ql[c] = lo;
            }
            const int at = place_k(4 * (tg & 3) + i, g, ks) + eh;
            *reinterpret_cast<half4 *>(&sh.K[0][rt][ks][at]) = kh;
            *reinterpret_cast<half4 *>(&sh.Q[0][rt][ks][at]) = qh;
            if constexpr (NK == 2) *reinterpret_cast<half4 *>(&sh.K[NK - 1][rt][ks][at]) = kl;
            if constexpr (NQ == 2) *reinterpret_cast<half4 *>(&sh.Q[NQ - 1][rt][ks][at]) = ql;
        }
        if (tid < kMeta) reinterpret_cast<u32x4 *>(&sh.m[which])[tid] = meta;
    }

    __device__ inline void write_tpw(Shared &sh) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int ch = 4 * cg + c, ct = ch >> 4;
            const int at = place_w(ch & 15, tg & 3, ct) + ((tg >> 2) & 1) * 4;
#pragma unroll
            for (int l = 0; l < NK; ++l) *reinterpret_cast<half4 *>(&sh.W[l][ct][tg >> 3][at]) = w[l][c];
        }
        pieces([&](u32x4 &x, int i) { sh.tp[i] = x; });
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
        mul4(f, hi, Y);
        mul4(f, lo, Y);
        __builtin_amdgcn_sched_barrier(0);
        right(X[2], X[3], s, hi1, lo1);
        load1(f, 0);
        mul4(f2, hi, Y);
        __builtin_amdgcn_sched_barrier(0);
        load1(f2, kTri);
        mul4(f, hi1, Y, 2);
        mul4(f, lo1, Y, 2);
        next();
        mul4(f2, hi1, Y, 2);
    } else {
        right(X[2], X[3], s, hi1, lo1);
        load1(f2, 0);
        mul4(f, hi, Y);
        next();
        mul4(f2, hi1, Y, 2);
    }
}

template <int DK, int DV, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__((256 + Producer<DK, KEYVEC, BF16>::PT)) k_chunk_fwd(const ChunkArgs A) {
    typedef FwdShared<DK, KEYVEC, BF16> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ;
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
        const size_t entry = (size_t)(t0 / kC + b) * H + h;
        Producer<DK, KEYVEC, BF16> p;
        p.tid = threadIdx.x - 256;
        p.cg = p.tid % p.CG;
        p.tg = p.tid / p.CG;
        auto load = [&](int c) { p.load(A, h, t0 + c * kC, min(t1 - t0 - c * kC, kC), entry + (size_t)c * H); };
        load(0);
        p.load_tp(A.prep + entry);
        p.write_kq(sh, 0);
        if (nc > 1) load(1);
        for (int c = 0; c < nc; ++c) {
            lds_barrier();               // K and Q of c stand; T, P, K^T of c - 1 are done with
            p.write_tpw(sh);
            if (c + 1 < nc) p.load_tp(A.prep + entry + (size_t)(c + 1) * H);
            lds_barrier();               // T, P, K^T of c stand; K and Q of c are done with
            if (c + 1 < nc) p.write_kq(sh, (c + 1) & 1);
            if (c + 2 < nc) load(c + 2);
        }
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
            // K hi, Q hi, K lo, Q lo, each on its way while the one before multiplies
            __builtin_amdgcn_sched_barrier(0);
            load4(f2, kq + q_at, row);
            mul4(f, hi, R);
            mul4(f, lo, R);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (NK == 2) {
                load4(f, kq + 4 * row, row);
                mul4(f2, hi, O);
                if constexpr (NQ == 2) mul4(f2, lo, O);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (NQ == 2) load4(f2, kq + q_at + 4 * row, row);
                mul4(f, hi, R);
                if constexpr (NQ == 2) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (ks + 1 < KS) {
                        kq = place(ks + 1);
                        load4(f, kq, row);
                    }
                    mul4(f2, hi, O);
                } else if (ks + 1 < KS) {
                    __builtin_amdgcn_sched_barrier(0);
                    kq = place(ks + 1);
                    load4(f, kq, row);
                }
            } else {
                if (ks + 1 < KS) {
                    kq = place(ks + 1);
                    load4(f, kq, row);
                }
                mul4(f2, hi, O);
            }
            if (ks + 1 < KS) right(S[2 * ks + 2], S[2 * ks + 3], s, hi, lo);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rk = row_factors(m + factors(offsetof(ChunkMeta, rk), rt)),
                          rq = row_factors(m + factors(offsetof(ChunkMeta, rq), rt));
            float x[4];
            widen(v[rt], x);
            quad_transpose(x);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // (one factor after the other: their product may underflow where the value does not)
                R[rt][r] = __builtin_fmaf(-(R[rt][r] * rk[r]), undo, x[r]);
                O[rt][r] = (O[rt][r] * rq[r]) * undo;
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
        lower<NQ == 2>(p, u, y, undo, f, f2, [&] { load_w(f, 0, 0, 0); });
        __builtin_amdgcn_sched_barrier(0);
        raw *out = static_cast<raw *>(A.o) + (size_t)(t0 + c * kC) * row_step + col4;
        const int n = t1 - t0 - c * kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 pf = row_factors(m + factors(offsetof(ChunkMeta, rp), rt)),
                          wf = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = __builtin_fmaf(y[rt][r] * pf[r], undo, O[rt][r]);
                u[rt][r] *= wf[r];
            }
            quad_transpose(x);
            raw z;
            narrow(x, z);
            if (16 * rt + row0 < n) out[(uint32_t)(16 * rt + row0) * row_step] = z;
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

template <int DK, int DV>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)(DV / 64) * (unsigned)a.s.H * (unsigned)a.s.B);
    constexpr int block = 256 + 4 * DK;
    if (keyvec && bf16) k_chunk_fwd<DK, DV, true, true><<<grid, block, 0, s>>>(a);
    else if (keyvec) k_chunk_fwd<DK, DV, true, false><<<grid, block, 0, s>>>(a);
    else if (bf16) k_chunk_fwd<DK, DV, false, true><<<grid, block, 0, s>>>(a);
    else k_chunk_fwd<DK, DV, false, false><<<grid, block, 0, s>>>(a);
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
