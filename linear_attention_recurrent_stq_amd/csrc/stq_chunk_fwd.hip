// The pass of the state through the chunks of a sequence (stq_chunk_forward).
//
// Per chunk, from T, P and the factors that k_chunk_prep left (stq_chunk.h):
//   R = V - (K G) S;   u = T R;   O = (Q G) S + P u;   S = diag(G_64) S + (K G_64/G)^T u.
//
// Columns of S are independent, so each of four waves owns 16 NT of them for
// the whole sequence: S stays in its registers, and no wave waits for another's
// values.  A result tile of the matrix instructions holds column l % 16 in lane
// l, which is where a right operand wants it, so S, R and u go from one product
// into the next without leaving the registers; only the order of a left
// operand's columns is permuted to match (4 g + e and 16 + 4 g + e in lane group
// g).  The left operands K, Q, K^T, T and P are the same for every wave: four
// more waves turn the next chunk's rows into scaled fp16 fragments in LDS
// while the first four multiply.
//
// Scalar bf16 rules need no lo parts of K and Q (exact in fp16) and fit two
// chunks of fragments in LDS: one barrier a chunk.  The others fold G into K and
// Q (key-vector gates) or carry fp32 rows, as hi + lo: one chunk fits, and the
// write of the next one stands between two barriers.
//
// NT = 2 (a workgroup takes 128 columns) halves the fragments read from LDS per
// matrix instruction; NT = 1 halves the time of a chunk and is taken when there
// are too few (sequence, head) pairs to fill the chip.
#include "stq_chunk.h"

namespace stq {
namespace {

constexpr int kMeta = sizeof(ChunkMeta) / 16;  // 16-byte pieces
constexpr int kTP = 2 * 2 * kTri * kFrag * 2 / 16;

template <int DK, bool LO>
struct FwdShared {
    static constexpr int NL = LO ? 2 : 1, NBUF = LO ? 1 : 2, KS = DK / 32, CT = DK / 16;
    struct Buf {
        _Float16 K[NL][4][KS][kFrag], Q[NL][4][KS][kFrag], W[NL][CT][2][kFrag];
        uint4 TP[kTP];               // T hi, T lo, P hi, P lo
        ChunkMeta m;
    } buf[NBUF];
    float gp[LO ? 16 : 1][DK];       // gate products of four tokens
};

// Where lane (row, g)'s eight halves stand in a fragment: rows are permuted so
// that the producers' writes (fixed row, all g and k steps) and the consumers'
// reads (fixed k step, all rows) both spread over the banks.
__device__ inline int place_k(int row16, int g, int ks) { return (g * 16 + (row16 ^ ((4 * g + ks) & 15))) * 8; }
__device__ inline int place_w(int ch16, int g, int ct) { return (g * 16 + (ch16 ^ (ct & 3))) * 8; }

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

// The producing waves: 256 threads; a unit is 4 tokens x 4 channels.
template <int DK, bool KEYVEC, bool BF16>
struct Producer {
    static constexpr bool LO = KEYVEC || !BF16;
    static constexpr int CG = DK / 4, U = DK / 64;  // channel groups; units of a thread
    typedef typename Raw4<BF16>::type raw;
    typedef FwdShared<DK, LO> Shared;
    raw k[U][4], q[U][4];
    float4 a[KEYVEC ? U : 1][4];
    uint4 tp[kTP / 256], meta;
    float sk[U][4], sq[U][4];

    __device__ inline void load(const ChunkArgs &A, int h, int first, int n, const ChunkPrep *e, int tid) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cg = (tid + 256 * u) % CG, tg = (tid + 256 * u) / CG;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * tg + i;
                k[u][i] = q[u][i] = raw{};
                if constexpr (KEYVEC) a[u][i] = make_float4(1.f, 1.f, 1.f, 1.f);
                if (t < n) {
                    const size_t at = (((size_t)(first + t) * A.s.H + h) * DK) / 4 + cg;
                    k[u][i] = static_cast<const raw *>(A.s.k)[at];
                    q[u][i] = static_cast<const raw *>(A.s.q)[at];
                    if constexpr (KEYVEC) a[u][i] = reinterpret_cast<const float4 *>(A.s.a)[at];
                }
                sk[u][i] = e->m.sk[t];
                sq[u][i] = e->m.sq[t];
            }
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(e);
#pragma unroll
        for (int i = 0; i < kTP / 256; ++i) tp[i] = src[tid + 256 * i];
        if (tid < kMeta) meta = src[kTP + tid];
    }

    // Key-vector gates: the product of the unit's four gates per channel.
    __device__ inline void groups(Shared &sh, int tid) {
        if constexpr (KEYVEC) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int cg = (tid + 256 * u) % CG, tg = (tid + 256 * u) / CG;
                float4 p = a[u][0];
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    p.x *= a[u][i].x;
                    p.y *= a[u][i].y;
                    p.z *= a[u][i].z;
                    p.w *= a[u][i].w;
                }
                *reinterpret_cast<float4 *>(&sh.gp[tg][4 * cg]) = p;
            }
        }
    }

    __device__ inline void write(Shared &sh, int which, int tid) {
        auto &B = sh.buf[which];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cg = (tid + 256 * u) % CG, tg = (tid + 256 * u) / CG;
            float pre[4] = {1.f, 1.f, 1.f, 1.f}, suf[4][4];
            if constexpr (KEYVEC) {
                float s[4] = {1.f, 1.f, 1.f, 1.f};
                for (int m = 0; m < 16; ++m) {
                    const float4 p = *reinterpret_cast<const float4 *>(&sh.gp[m][4 * cg]);
                    const float x[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        pre[c] *= m < tg ? x[c] : 1.f;
                        s[c] *= m > tg ? x[c] : 1.f;
                    }
                }
#pragma unroll
                for (int i = 3; i >= 0; --i) {  // products of the gates after token i
#pragma unroll
                    for (int c = 0; c < 4; ++c) suf[i][c] = s[c];
                    float x[4];
                    widen(a[u][i], x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[c] *= x[c];
                }
            }
            const int g = cg & 3, ks = cg >> 3, eh = ((cg >> 2) & 1) * 4, rt = tg >> 2;
            _Float16 wh[4][4], wl[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float kx[4], qx[4];
                widen(k[u][i], kx);
                widen(q[u][i], qx);
                if constexpr (KEYVEC) {
                    float x[4];
                    widen(a[u][i], x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) pre[c] *= x[c];
                }
                half4 kh, kl, qh, ql;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    _Float16 hi, lo;
                    if constexpr (LO) {
                        split(KEYVEC ? kx[c] * pre[c] : kx[c], sk[u][i], hi, lo);
                        kh[c] = hi;
                        kl[c] = lo;
                        if constexpr (KEYVEC) split(kx[c] * suf[i][c], sk[u][i], hi, lo);
                        wh[i][c] = hi;
                        wl[i][c] = lo;
                        split(KEYVEC ? qx[c] * pre[c] : qx[c], sq[u][i], hi, lo);
                        qh[c] = hi;
                        ql[c] = lo;
                    } else {
                        kh[c] = wh[i][c] = (_Float16)(kx[c] * sk[u][i]);
                        qh[c] = (_Float16)(qx[c] * sq[u][i]);
                    }
                }
                const int at = place_k(4 * (tg & 3) + i, g, ks) + eh;
                *reinterpret_cast<half4 *>(&B.K[0][rt][ks][at]) = kh;
                *reinterpret_cast<half4 *>(&B.Q[0][rt][ks][at]) = qh;
                if constexpr (LO) {
                    *reinterpret_cast<half4 *>(&B.K[1][rt][ks][at]) = kl;
                    *reinterpret_cast<half4 *>(&B.Q[1][rt][ks][at]) = ql;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int ch = 4 * cg + c, ct = ch >> 4;
                const int at = place_w(ch & 15, tg & 3, ct) + ((tg >> 2) & 1) * 4;
                half4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = wh[i][c];
                *reinterpret_cast<half4 *>(&B.W[0][ct][tg >> 3][at]) = w;
                if constexpr (LO) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = wl[i][c];
                    *reinterpret_cast<half4 *>(&B.W[1][ct][tg >> 3][at]) = w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kTP / 256; ++i) B.TP[tid + 256 * i] = tp[i];
        if (tid < kMeta) reinterpret_cast<uint4 *>(&B.m)[tid] = meta;
    }
};

__device__ inline half8 frag(const _Float16 *p) { return *reinterpret_cast<const half8 *>(p); }

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

__device__ inline floatx4 row_factors(const float *p) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    return floatx4{x.x, x.y, x.z, x.w};
}

template <int DK, int DV, int NT, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__(512) k_chunk_fwd(const ChunkArgs A) {
    constexpr bool LO = KEYVEC || !BF16;
    typedef FwdShared<DK, LO> Shared;
    constexpr int KS = Shared::KS, CT = Shared::CT, NBUF = Shared::NBUF;
    __shared__ Shared sh;
    const int H = A.s.H, h = blockIdx.y, b = blockIdx.z;
    int t0, t1;
    seq_range(A.s, b, t0, t1);
    const int nc = (t1 - t0 + kC - 1) / kC;
    const ChunkPrep *entry = A.prep + (size_t)(t0 / kC + b) * H + h;

    if (threadIdx.x >= 256) {
        const int tid = threadIdx.x - 256;
        Producer<DK, KEYVEC, BF16> p;
        auto load = [&](int c) {
            if (c < nc) p.load(A, h, t0 + c * kC, min(t1 - t0 - c * kC, kC), entry + (size_t)c * H, tid);
        };
        load(0);
        if constexpr (NBUF == 2) {
            if (nc) p.write(sh, 0, tid);
            load(1);
            for (int c = 0; c < nc; ++c) {
                __syncthreads();
                if (c + 1 < nc) p.write(sh, (c + 1) & 1, tid);
                load(c + 2);
            }
        } else {
            if (nc) p.groups(sh, tid);
            for (int c = 0; c < nc; ++c) {
                __syncthreads();
                p.write(sh, 0, tid);
                __syncthreads();
                load(c + 1);
                if (c + 1 < nc) p.groups(sh, tid);
            }
        }
        return;
    }

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    const int col = (blockIdx.x * 4 + wave) * 16 * NT + c16;  // of the first tile
    floatx4 S[NT][CT];
    const size_t state0 = ((size_t)b * H + h) * DK * DV;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[nt][ct][r] =
                    A.initial ? A.initial[state0 + (size_t)(16 * ct + 4 * g + r) * DV + col + 16 * nt] : 0.f;

    float v[NT][16];
    auto load_v = [&](int c) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = t0 + c * kC + 16 * (i >> 2) + 4 * g + (i & 3);
                v[nt][i] = 0.f;
                if (t < t1) {
                    const size_t at = ((size_t)t * H + h) * DV + col + 16 * nt;
                    if constexpr (BF16)
                        v[nt][i] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(A.s.v)[at] << 16);
                    else v[nt][i] = static_cast<const float *>(A.s.v)[at];
                }
            }
    };
    if (nc) load_v(0);

    for (int c = 0; c < nc; ++c) {
        __syncthreads();
        if constexpr (NBUF == 1) __syncthreads();
        const auto &B = sh.buf[NBUF == 2 ? c & 1 : 0];
        const _Float16 *tp = reinterpret_cast<const _Float16 *>(B.TP);
        floatx4 R[NT][4], O[NT][4];
        float inv[NT];
        {
            float s[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[nt] = scale_to(column_max(S[nt]), 13, inv[nt]);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) R[nt][rt] = O[nt][rt] = floatx4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                half8 hi[NT], lo[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) right(S[nt][2 * ks], S[nt][2 * ks + 1], s[nt], hi[nt], lo[nt]);
                const int at = place_k(c16, g, ks);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) {
                    const half8 kh = frag(&B.K[0][rt][ks][at]), qh = frag(&B.Q[0][rt][ks][at]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        R[nt][rt] = mfma16(kh, hi[nt], R[nt][rt]);
                        O[nt][rt] = mfma16(qh, hi[nt], O[nt][rt]);
                        R[nt][rt] = mfma16(kh, lo[nt], R[nt][rt]);
                        O[nt][rt] = mfma16(qh, lo[nt], O[nt][rt]);
                    }
                    if constexpr (LO) {
                        const half8 kl = frag(&B.K[1][rt][ks][at]), ql = frag(&B.Q[1][rt][ks][at]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            R[nt][rt] = mfma16(kl, hi[nt], R[nt][rt]);
                            O[nt][rt] = mfma16(ql, hi[nt], O[nt][rt]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const floatx4 rk = row_factors(&B.m.rk[16 * rt + 4 * g]), rq = row_factors(&B.m.rq[16 * rt + 4 * g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // (one factor after the other: their product may underflow where the value does not)
                    R[nt][rt][r] = __builtin_fmaf(-(R[nt][rt][r] * rk[r]), inv[nt], v[nt][4 * rt + r]);
                    O[nt][rt][r] = (O[nt][rt][r] * rq[r]) * inv[nt];
                }
        }
        if (c + 1 < nc) load_v(c + 1);
        // a lower triangular left operand (T at 0, P at 1) times a column block
        auto lower = [&](int which, const floatx4 (&X)[4], floatx4 (&Y)[4], float &undo) {
            const float s = scale_to(column_max(X), 13, undo);
            const _Float16 *t = tp + which * 2 * kTri * kFrag + lane * 8;
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) Y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                half8 hi, lo;
                right(X[2 * ks], X[2 * ks + 1], s, hi, lo);
#pragma unroll
                for (int rt = 2 * ks; rt < 4; ++rt) {
                    const half8 th = frag(t + tri(rt, ks) * kFrag), tl = frag(t + (kTri + tri(rt, ks)) * kFrag);
                    Y[rt] = mfma16(th, hi, Y[rt]);
                    Y[rt] = mfma16(th, lo, Y[rt]);
                    Y[rt] = mfma16(tl, hi, Y[rt]);
                }
            }
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            floatx4 u[4], y[4];
            float undo;
            lower(0, R[nt], u, undo);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const floatx4 f = row_factors(&B.m.rt[16 * rt + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) u[rt][r] = (u[rt][r] * f[r]) * undo;
            }
            lower(1, u, y, undo);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const floatx4 f = row_factors(&B.m.rp[16 * rt + 4 * g]);
                const floatx4 w = row_factors(&B.m.rw[16 * rt + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float o = __builtin_fmaf(y[rt][r] * f[r], undo, O[nt][rt][r]);
                    const int t = t0 + c * kC + 16 * rt + 4 * g + r;
                    if (t < t1) {
                        const size_t at = ((size_t)t * H + h) * DV + col + 16 * nt;
                        if constexpr (BF16) static_cast<__bf16 *>(A.o)[at] = (__bf16)o;
                        else static_cast<float *>(A.o)[at] = o;
                    }
                    u[rt][r] *= w[r];
                }
            }
            const float s = scale_to(column_max(u), 13, undo);
            half8 hi[2], lo[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) right(u[2 * ks], u[2 * ks + 1], s, hi[ks], lo[ks]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                floatx4 z = {0.f, 0.f, 0.f, 0.f};
                const int at = place_w(c16, g, ct);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const half8 wh = frag(&B.W[0][ct][ks][at]);
                    z = mfma16(wh, hi[ks], z);
                    z = mfma16(wh, lo[ks], z);
                    if constexpr (LO) z = mfma16(frag(&B.W[1][ct][ks][at]), hi[ks], z);
                }
                const floatx4 d = row_factors(&B.m.dec[16 * ct + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) S[nt][ct][r] = __builtin_fmaf(z[r], undo, S[nt][ct][r] * d[r]);
            }
        }
    }
    if (!A.last) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                A.last[state0 + (size_t)(16 * ct + 4 * g + r) * DV + col + 16 * nt] = S[nt][ct][r];
}

template <int DK, int DV, int NT>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid(DV / (64 * NT), (unsigned)a.s.H, (unsigned)a.s.B);
    if (keyvec && bf16) k_chunk_fwd<DK, DV, NT, true, true><<<grid, 512, 0, s>>>(a);
    else if (keyvec) k_chunk_fwd<DK, DV, NT, true, false><<<grid, 512, 0, s>>>(a);
    else if (bf16) k_chunk_fwd<DK, DV, NT, false, true><<<grid, 512, 0, s>>>(a);
    else k_chunk_fwd<DK, DV, NT, false, false><<<grid, 512, 0, s>>>(a);
}

template <int DK>
void go_dv(const ChunkArgs &a, int dv, bool keyvec, bool bf16, hipStream_t s) {
    const bool few = (int64_t)a.s.B * a.s.H < 256;  // fewer pairs than compute units
    if (dv == 64) go<DK, 64, 1>(a, keyvec, bf16, s);
    else if (few) go<DK, 128, 1>(a, keyvec, bf16, s);
    else go<DK, 128, 2>(a, keyvec, bf16, s);
}

}  // namespace

hipError_t launch_chunk_forward(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64) go_dv<64>(a, dv, keyvec, bf16, s);
    else go_dv<128>(a, dv, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
