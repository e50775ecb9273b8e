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
// producing waves turn the next chunk's rows into scaled fp16 fragments in LDS
// while the others multiply.  The fragments need no second buffer: K and Q are
// read in the first half of a chunk, T, P and K^T in the second, and each half's are
// replaced while the other half runs (two barriers a chunk, which wait for
// LDS only).
//
// Eight multiplying waves take the 128 columns of a (sequence, head), so that
// two share a SIMD and fill each other's waits; with fewer pairs than compute
// units, two workgroups of four waves take 64 each.
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

// The producing waves; a unit is 4 tokens x 4 channels.  Rules with lo parts of
// K take a thread a unit (with two, the raw rows and the K^T kept back spill).
template <int DK, bool KEYVEC, bool BF16>
struct Producer {
    typedef FwdShared<DK, KEYVEC, BF16> Shared;
    typedef typename Raw4<BF16>::type raw;
    static constexpr int NK = Shared::NK, NQ = Shared::NQ;
    static constexpr int PT = NK == 2 ? 4 * DK : 256;        // producing threads
    static constexpr int CG = DK / 4, U = 4 * DK / PT;       // channel groups; units of a thread
    raw k[U][4], q[U][4];
    float4 a[KEYVEC ? U : 1][4], pre[KEYVEC ? U : 1], suf[KEYVEC ? U : 1], sk[U], sq[U];
    u32x4 tp0, tp1, tp2, tp3, tp4, tp5, meta;
    half4 w[U][NK][4];               // K^T fragments of the chunk whose K and Q are written
    int n;                           // tokens of the chunk in k, q and a

    __device__ static inline int channels(int u, int tid) { return (tid + PT * u) % CG; }
    __device__ static inline int tokens(int u, int tid) { return (tid + PT * u) / CG; }

    __device__ inline void load(const ChunkArgs &A, int h, int first, int n_, size_t entry, int tid) {
        n = n_;
        const ChunkPrep *e = A.prep + entry;
        const size_t base = ((size_t)first * A.s.H + h) * CG;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cg = channels(u, tid), tg = tokens(u, tid);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // past the last token its row again: T has zeros in those columns and rows,
                // so whatever finite values stand there add nothing
                const uint32_t at = (uint32_t)min(4 * tg + i, n - 1) * (uint32_t)(A.s.H * CG) + cg;
                k[u][i] = (static_cast<const raw *>(A.s.k) + base)[at];
                q[u][i] = (static_cast<const raw *>(A.s.q) + base)[at];
                if constexpr (KEYVEC) a[u][i] = (reinterpret_cast<const float4 *>(A.s.a) + base)[at];
            }
            if constexpr (KEYVEC) {
                pre[u] = *reinterpret_cast<const float4 *>(&A.gates[entry].pre[tg][4 * cg]);
                suf[u] = *reinterpret_cast<const float4 *>(&A.gates[entry].suf[tg][4 * cg]);
            }
            sk[u] = *reinterpret_cast<const float4 *>(&e->m.sk[4 * tg]);
            sq[u] = *reinterpret_cast<const float4 *>(&e->m.sq[4 * tg]);
        }
        if (tid < kMeta) meta = reinterpret_cast<const u32x4 *>(&e->m)[tid];
    }

    // f(piece, its number) over this thread's pieces of T and P
    template <class F>
    __device__ inline void pieces(int tid, F f) {
        constexpr int TP = Shared::TP;
        f(tp0, tid);
        f(tp1, tid + PT);
        if (2 * PT + PT <= TP || tid + 2 * PT < TP) f(tp2, tid + 2 * PT);
        if constexpr (3 * PT < TP) f(tp3, tid + 3 * PT);
        if constexpr (4 * PT < TP)
            if (5 * PT <= TP || tid + 4 * PT < TP) f(tp4, tid + 4 * PT);
        if constexpr (5 * PT < TP) f(tp5, tid + 5 * PT);
    }

    __device__ inline void load_tp(const ChunkPrep *e, int tid) {
        pieces(tid, [&](u32x4 &x, int i) { x = reinterpret_cast<const u32x4 *>(e)[i]; });
    }

    // Gate of token t in a unit's channels: 1 past the last token.
    __device__ inline void gate(int u, int i, int t, float (&x)[4]) const {
        widen(a[u][i], x);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = t < n ? x[c] : 1.f;
    }

    // K and Q of the chunk into LDS, its K^T into w.
    __device__ inline void write_kq(Shared &sh, int which, int tid) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cg = channels(u, tid), tg = tokens(u, tid);
            float before[4], after[4][4];  // gate products up to and past a token
            if constexpr (KEYVEC) {
                widen(pre[u], before);
                float s[4];
                widen(suf[u], s);
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    float x[4];
                    gate(u, i, 4 * tg + i, x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        after[i][c] = s[c];
                        s[c] *= x[c];
                    }
                }
            }
            const int g = cg & 3, ks = cg >> 3, eh = ((cg >> 2) & 1) * 4, rt = tg >> 2;
            const float ek[4] = {sk[u].x, sk[u].y, sk[u].z, sk[u].w}, eq[4] = {sq[u].x, sq[u].y, sq[u].z, sq[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float kx[4], qx[4];
                widen(k[u][i], kx);
                widen(q[u][i], qx);
                if constexpr (KEYVEC) {
                    float x[4];
                    gate(u, i, 4 * tg + i, x);
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
                        w[u][0][c][i] = hi;
                        w[u][NK - 1][c][i] = lo;
                    } else {
                        kh[c] = w[u][0][c][i] = (_Float16)(kx[c] * ek[i]);
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
        }
        if (tid < kMeta) reinterpret_cast<u32x4 *>(&sh.m[which])[tid] = meta;
    }

    __device__ inline void write_tpw(Shared &sh, int tid) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cg = channels(u, tid), tg = tokens(u, tid);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int ch = 4 * cg + c, ct = ch >> 4;
                const int at = place_w(ch & 15, tg & 3, ct) + ((tg >> 2) & 1) * 4;
#pragma unroll
                for (int l = 0; l < NK; ++l) *reinterpret_cast<half4 *>(&sh.W[l][ct][tg >> 3][at]) = w[u][l][c];
            }
        }
        pieces(tid, [&](u32x4 &x, int i) { sh.tp[i] = x; });
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

// A lower triangular left operand (fragments at t, lo parts kTri further) times
// a column block; `undo` takes the block's scale away.  FULL: with the lo parts.
template <bool FULL>
__device__ inline void lower(lds_half t, const floatx4 (&X)[4], floatx4 (&Y)[4], float &undo) {
    const float s = scale_to(column_max(X), 13, undo);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) Y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        __builtin_amdgcn_sched_barrier(0);
        half8 hi, lo, th[4];
        right(X[2 * ks], X[2 * ks + 1], s, hi, lo);
#pragma unroll
        for (int rt = 2 * ks; rt < 4; ++rt) th[rt] = frag(t + tri(rt, ks) * kFrag);
#pragma unroll
        for (int rt = 2 * ks; rt < 4; ++rt) Y[rt] = mfma16(th[rt], hi, Y[rt]);
        if constexpr (FULL) {
#pragma unroll
            for (int rt = 2 * ks; rt < 4; ++rt) Y[rt] = mfma16(th[rt], lo, Y[rt]);
#pragma unroll
            for (int rt = 2 * ks; rt < 4; ++rt) th[rt] = frag(t + (kTri + tri(rt, ks)) * kFrag);
#pragma unroll
            for (int rt = 2 * ks; rt < 4; ++rt) Y[rt] = mfma16(th[rt], hi, Y[rt]);
        }
    }
}

template <int DK, int DV, int NW, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__((64 * NW + Producer<DK, KEYVEC, BF16>::PT)) k_chunk_fwd(const ChunkArgs A) {
    typedef FwdShared<DK, KEYVEC, BF16> Shared;
    typedef typename Raw4<BF16>::type raw;
    constexpr int KS = Shared::KS, CT = Shared::CT, NK = Shared::NK, NQ = Shared::NQ;
    __shared__ Shared sh;
    const int H = A.s.H, h = blockIdx.y, b = blockIdx.z;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    const int nc = (t1 - t0 + kC - 1) / kC;

    if (threadIdx.x >= 64 * NW) {
        if (nc == 0) return;
        const size_t entry = (size_t)(t0 / kC + b) * H + h;
        const int tid = threadIdx.x - 64 * NW;
        Producer<DK, KEYVEC, BF16> p;
        auto load = [&](int c) {
            p.load(A, h, t0 + c * kC, min(t1 - t0 - c * kC, kC), entry + (size_t)c * H, tid);
        };
        load(0);
        p.load_tp(A.prep + entry, tid);
        p.write_kq(sh, 0, tid);
        if (nc > 1) load(1);
        for (int c = 0; c < nc; ++c) {
            lds_barrier();               // K and Q of c stand; T, P, K^T of c - 1 are done with
            p.write_tpw(sh, tid);
            if (c + 1 < nc) p.load_tp(A.prep + entry + (size_t)(c + 1) * H, tid);
            lds_barrier();               // T, P, K^T of c stand; K and Q of c are done with
            if (c + 1 < nc) p.write_kq(sh, (c + 1) & 1, tid);
            if (c + 2 < nc) load(c + 2);
        }
        return;
    }

    const int lane = threadIdx.x & 63, wave = wave_index(), c16 = lane & 15, g = lane >> 4;
    const int col0 = (blockIdx.x * NW + wave) * 16;
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
        lds_barrier();
        const lds_float m = float_at(&sh.m[c & 1], 4 * g);
        floatx4 R[4], O[4];
        float undo;
        {
            const float s = scale_to(column_max(S), 13, undo);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) R[rt] = O[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                half8 hi, lo;
                right(S[2 * ks], S[2 * ks + 1], s, hi, lo);
                const lds_half kq = half_at(&sh.K, place_k(c16, g, ks));
                half8 f[4];
                // (an operand's four fragments at a time: more of them in flight spill)
                auto rows = [&](int from, floatx4 (&Y)[4], bool both) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) f[rt] = frag(kq + (from + rt * KS + ks) * kFrag);
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) Y[rt] = mfma16(f[rt], hi, Y[rt]);
                    if (both) {
#pragma unroll
                        for (int rt = 0; rt < 4; ++rt) Y[rt] = mfma16(f[rt], lo, Y[rt]);
                    }
                };
                rows(0, R, true);
                rows(4 * KS * NK, O, NQ == 2);
                if constexpr (NK == 2) rows(4 * KS, R, false);
                if constexpr (NQ == 2) rows(4 * KS * (NK + 1), O, false);
            }
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            __builtin_amdgcn_sched_barrier(0);
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
        }
        if (c + 1 < nc) load_v(c + 1);
        lds_barrier();
        floatx4 u[4], y[4];
        const lds_half t = half_at(&sh.tp, lane * 8);
        lower<true>(t, R, u, undo);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 f = row_factors(m + factors(offsetof(ChunkMeta, rt), rt));
#pragma unroll
            for (int r = 0; r < 4; ++r) u[rt][r] = (u[rt][r] * f[r]) * undo;
        }
        lower<NQ == 2>(t + 2 * kTri * kFrag, u, y, undo);
        raw *out = static_cast<raw *>(A.o) + (size_t)(t0 + c * kC) * row_step + col4;
        const int n = t1 - t0 - c * kC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            __builtin_amdgcn_sched_barrier(0);
            const floatx4 f = row_factors(m + factors(offsetof(ChunkMeta, rp), rt)),
                          w = row_factors(m + factors(offsetof(ChunkMeta, rw), rt));
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = __builtin_fmaf(y[rt][r] * f[r], undo, O[rt][r]);
                u[rt][r] *= w[r];
            }
            quad_transpose(x);
            raw z;
            narrow(x, z);
            if (16 * rt + row0 < n) out[(uint32_t)(16 * rt + row0) * row_step] = z;
        }
        __builtin_amdgcn_sched_barrier(0);
        const float s = scale_to(column_max(u), 13, undo);
        half8 hi[2], lo[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) right(u[2 * ks], u[2 * ks + 1], s, hi[ks], lo[ks]);
        lds_half wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[i] = half_at(&sh.W, place_w(c16, g, i));
#pragma unroll
        for (int c0 = 0; c0 < CT; c0 += 4) {
            __builtin_amdgcn_sched_barrier(0);
            floatx4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                half8 wf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) wf[i] = frag(wb[i] + ((c0 + i) * 2 + ks) * kFrag);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = mfma16(wf[i], hi[ks], z[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = mfma16(wf[i], lo[ks], z[i]);
                if constexpr (NK == 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        z[i] = mfma16(frag(wb[i] + ((CT + c0 + i) * 2 + ks) * kFrag), hi[ks], z[i]);
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

template <int DK, int DV, int NW>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid(DV / (16 * NW), (unsigned)a.s.H, (unsigned)a.s.B);
    constexpr int lo = 64 * NW + Producer<DK, true, true>::PT, plain = 64 * NW + Producer<DK, false, true>::PT;
    if (keyvec && bf16) k_chunk_fwd<DK, DV, NW, true, true><<<grid, lo, 0, s>>>(a);
    else if (keyvec) k_chunk_fwd<DK, DV, NW, true, false><<<grid, lo, 0, s>>>(a);
    else if (bf16) k_chunk_fwd<DK, DV, NW, false, true><<<grid, plain, 0, s>>>(a);
    else k_chunk_fwd<DK, DV, NW, false, false><<<grid, lo, 0, s>>>(a);
}

template <int DK>
void go_dv(const ChunkArgs &a, int dv, bool keyvec, bool bf16, hipStream_t s) {
    const bool few = (int64_t)a.s.B * a.s.H < 256;  // fewer pairs than compute units
    if (dv == 64) go<DK, 64, 4>(a, keyvec, bf16, s);
    else if (few) go<DK, 128, 4>(a, keyvec, bf16, s);
    else go<DK, 128, 8>(a, keyvec, bf16, s);
}

}  // namespace

hipError_t launch_chunk_forward(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64) go_dv<64>(a, dv, keyvec, bf16, s);
    else go_dv<128>(a, dv, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
