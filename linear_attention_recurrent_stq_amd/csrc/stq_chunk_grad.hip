// The gradients of a chunk's inputs (the last part of stq_chunk_backward): one workgroup
// per (chunk, head), all chunks at once.
//
// From the chunk's first state S, the gradient dS behind it, its delta errors w (u = beta w)
// and y (beta y: the gradient of v), per token i, with G_i the gates up to i, E_i those after it:
//   dq_i = G_i S dO_i                       + sum_{j<=i} dP_ij  k_j prod_{j<s<=i} a_s
//   dk_i = -beta_i G_i S y_i  (it reads)    + sum_{j<i}  dA_ij  k_j prod_{j<s<=i} a_s
//          + beta_i E_i dS w_i  (it writes) + sum_{j>i} dA_ji k_j prod + sum_{j>=i} dP_ji q_j prod
//   dbeta_i = y_i . w_i;   dP_ij = beta_j dO_i . w_j;   dA_ij = -beta_i beta_j y_i . w_j.
// Gates: a_t scales whatever passes from before t to t or later.  Per channel, with e_i = q_i dq_i +
// k_i (dk_i's reading parts) - k_i (its writing parts inside the chunk) and f_j = k_j (its
// part beta E dS w):
//   a_t da_t = G_64 sum_v dS S + sum_{i>=t} e_i + sum_{j<t} f_j
// (summed over channels for scalar gates); the quotient by a_t is taken last.
//
// Everything is formed transposed, tokens in the lanes: wave (I, half) takes the 16 tokens
// of block I and half of the channels.  Its own dO, y and w are right operands in its registers
// (eight values of a row a lane); the states and the other tokens' rows are
// left operands in LDS, in the same form.  dP and dA come out as tiles that are right operands of
// the products with K^T and Q^T as they stand, both ways round (j up to I and j from I on), ten
// 16x16 tiles in every wave.
//
// Scalar gates multiply dP and dA.  Key-vector gates stand inside the products: between
// blocks they are split as in the preparation (k suf and (q, k) pre, and whole blocks between
// one step of the sum and the next); inside a block each of the fifteen distances is vector
// code, the other token read across the lanes of a row of 16.
//
// A workgroup holds about 117 KB of LDS and eight waves of 200 to 256 registers, so one a CU: the bound
// is its vector instructions (49 % of the cycles with scalar gates, 57 % with key-vector ones) and
// what they wait for. Measured, bf16, d_k = d_v = 128, 16 heads, MI355X: scalar gates, 16384 tokens 494 us
// (887 MB, S and dS most of it: 1.8 TB/s); key-vector gates, 8192 tokens 359 us.

#include "stq_chunk.h"

namespace stq {
namespace {

template <bool BF16> struct Four;  // four elements as they are in memory
template <> struct Four<true> {
    uint2 w;
    __device__ void get(float (&x)[4]) const {
        x[0] = bf16_lo(w.x);
        x[1] = bf16_hi(w.x);
        x[2] = bf16_lo(w.y);
        x[3] = bf16_hi(w.y);
    }
    __device__ void set(const float (&x)[4]) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        w.x = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[0], (__bf16)x[1]});
        w.y = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[2], (__bf16)x[3]});
    }
};
template <> struct Four<false> {
    float4 w;
    __device__ void get(float (&x)[4]) const {
        x[0] = w.x;
        x[1] = w.y;
        x[2] = w.z;
        x[3] = w.w;
    }
    __device__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
};

__device__ inline int place(int row16, int g, int ks) { return g * 16 + (row16 ^ ((4 * g + ks) & 15)); }

template <int DK, int DV, bool KEYVEC, bool BF16>
struct GradShared {
    static constexpr int DVS = DV / 32, CT = DK / 16, NO = BF16 ? 1 : 2, NK = BF16 ? 1 : 2;
    union {
        struct {
            half8 w[2][4][DVS][64], y[2][4][DVS][64], o[NO][4][DVS][64];  // rows of all tokens
        } t;
        half8 st[2][CT][DVS][64];        // a state
        struct {
            half8 k[NK][CT][2][64], q[NK][CT][2][64];                     // K^T, Q^T
        } c;
        struct {
            half4 y[2][CT][4][64], x[2][CT][4][64], z[2][CT][4][64];      // (K suf)^T, (K pre)^T, (Q pre)^T
        } v;
    };
    alignas(16) float iw[kC], iy[kC], io[kC], ik[kC], iq[kC], be[kC], ga[kC], pre[kC], suf[kC];
    float srow[DK], rho[DK];             // scales of a state's rows; sum over v of dS S
    alignas(16) float B[4][DK];          // key-vector gates: products of the blocks
    float d[2][4][16][17];               // key-vector gates: dP, dA inside the blocks [i][j]
    alignas(16) float te[4][DK], tf[4][DK];  // key-vector gates: sums of e and f of the blocks
    float es[2][kC], fs[2][kC];          // scalar gates: e and f by halves of the channels
};

// The passes leave states, w and y as result tiles, [tile][lane][4]: lane (c, g) has rows 4 g .. + 3
// of column c.  Of a tile, lane (c, g) here gets columns 4 g .. + 3 of row c: quads read one row's
// four groups, and turn them.
__device__ inline int untwist() {
    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
    return 4 * g + (c16 & 3) + 16 * (c16 >> 2);
}
__device__ inline void load_turned(const float *tile, float (&x)[4]) {
    const floatx4 v = four(tile + 4 * untwist());
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = v[r];
    quad_transpose(x);
}

// Left (lh, ll) times right (rh, rl) operand; lo parts as far as they are there.
template <bool LL, bool RL>
__device__ inline floatx4 mul(half8 lh, half8 ll, half8 rh, half8 rl, floatx4 c) {
    c = mfma16(lh, rh, c);
    if constexpr (RL) c = mfma16(lh, rl, c);
    if constexpr (LL) c = mfma16(ll, rh, c);
    return c;
}
__device__ inline floatx4 mul4(half4 lh, half4 ll, half4 rh, half4 rl, floatx4 c) {
    c = __builtin_amdgcn_mfma_f32_16x16x16f16(lh, rh, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x16f16(lh, rl, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x16f16(ll, rh, c, 0, 0, 0);
}
__device__ inline void split4(floatx4 x, float s, half4 &hi, half4 &lo) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        _Float16 a, b;
        split(x[r], s, a, b);
        hi[r] = a;
        lo[r] = b;
    }
}
__device__ inline float tiles_max(const floatx4 (&x)[4], float m = 0.f) {
#pragma unroll
    for (int J = 0; J < 4; ++J)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(x[J][r]));
    return m;
}

// Distances D and up inside a block (key-vector gates): one token's pairs (i, i - D) and
// (i + D, i) for T tiles of channels.
template <int D, int T, class Sh>
__device__ inline void distances(const Sh &sh, int w, int c16, const float (&k)[T][4], const float (&q)[T][4],
                                 const float (&a)[T][4], float (&before)[T][4], float (&after)[T][4],
                                 float (&dq)[T][4], float (&dr)[T][4], float (&dw)[T][4]) {
    const bool lo = c16 >= D, hi = c16 + D < 16;
    const int j = lo ? c16 - D : 0, i = hi ? c16 + D : 15;
    float p0 = sh.d[0][w][c16][j], a0 = sh.d[1][w][c16][j], p1 = sh.d[0][w][i][c16], a1 = sh.d[1][w][i][c16];
    p0 = lo ? p0 : 0.f;
    a0 = lo ? a0 : 0.f;
    p1 = hi ? p1 : 0.f;
    a1 = hi ? a1 : 0.f;
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            // gates of i - D + 1 .. i, and of i + 1 .. i + D
            before[t][r] = D == 1 ? a[t][r] : before[t][r] * dpp0<kShr + (D > 1 ? D - 1 : 1)>(a[t][r]);
            after[t][r] = D == 1 ? dpp0<kShl + 1>(a[t][r]) : after[t][r] * dpp0<kShl + D>(a[t][r]);
            const float x = before[t][r] * dpp0<kShr + D>(k[t][r]);
            dq[t][r] = __builtin_fmaf(p0, x, dq[t][r]);
            dr[t][r] = __builtin_fmaf(a0, x, dr[t][r]);
            const float y = __builtin_fmaf(p1, dpp0<kShl + D>(q[t][r]), a1 * dpp0<kShl + D>(k[t][r]));
            dw[t][r] = __builtin_fmaf(after[t][r], y, dw[t][r]);
            // formed here: moved to where the sums are used, which lanes past the last token skip, they
            // would keep every distance's values of other lanes until then
            asm volatile("" : "+v"(dq[t][r]), "+v"(dr[t][r]), "+v"(dw[t][r]));
        }
    }
    if constexpr (D < 15) distances<D + 1, T>(sh, w, c16, k, q, a, before, after, dq, dr, dw);
}

template <int DK, int DV, bool KEYVEC, bool BF16>
__global__ void __launch_bounds__(512) k_chunk_grad(const ChunkArgs A) {
    typedef GradShared<DK, DV, KEYVEC, BF16> Shared;
    constexpr int DVS = Shared::DVS, CT = Shared::CT, NO = Shared::NO, NK = Shared::NK, T = CT / 2;
    __shared__ Shared sh;
    const SeqArgs &s = A.s;
    uint32_t slot, h;
    xcd_place(blockIdx.x, s.H, slot, h);
    const int tid = threadIdx.x, lane = tid & 63, w = wave_index() & 3, half = wave_index() >> 2, c16 = lane & 15,
              g = lane >> 4;
    int b, first;
    const int n = chunk_of_slot(s, slot, b, first);
    if (n == 0) return;
    const size_t entry = (size_t)slot * s.H + h;
    const ChunkMeta &m = A.prep[entry].m;
    const int own = 16 * w + c16;        // the lane's token
    const bool on = own < n;
    const size_t tok = (size_t)(first + min(own, n - 1)) * s.H + h;

    // the states' tiles on their way before they are wanted: the gradient's while the first one is
    // multiplied
    floatx4 S[DV / 16], dS[DV / 16];
    auto fetch = [&](const float *states, floatx4 (&x)[DV / 16]) {
        const int ct = min(wave_index(), CT - 1);
#pragma unroll
        for (int cb = 0; cb < DV / 16; ++cb) x[cb] = four(states + entry * (DK * DV) + (cb * CT + ct) * 256 + 4 * untwist());
    };
    // ---- own rows of dO, y and w as right operands
    half8 oh[DVS], ol[NO == 2 ? DVS : 1], yh[DVS], yl[DVS], wh[DVS], wl[DVS];
    float own_io, own_iy, own_iw;
    {
        float x[DVS][8], z[DVS][8], mx = 0.f, dot = 0.f, sc;
        const float *yp = A.y + entry * (kC * DV), *wp = A.w + entry * (kC * DV);
#pragma unroll
        for (int cb = 0; cb < DV / 16; ++cb) {
            float a[4], b[4];
            load_turned(yp + (cb * 4 + w) * 256, a);
            load_turned(wp + (cb * 4 + w) * 256, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[cb >> 1][4 * (cb & 1) + e] = a[e];
                z[cb >> 1][4 * (cb & 1) + e] = b[e];
                dot = __builtin_fmaf(a[e], b[e], dot);
                mx = fmaxf(mx, fabsf(a[e]));
            }
        }
        fetch(A.S, S);
        sc = scale_to(max_groups(mx), 13, own_iy);
#pragma unroll
        for (int i = 0; i < DVS; ++i) split8(x[i], sc, yh[i], yl[i]);
        mx = 0.f;
#pragma unroll
        for (int i = 0; i < DVS; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(z[i][e]));
        sc = scale_to(max_groups(mx), 13, own_iw);
#pragma unroll
        for (int i = 0; i < DVS; ++i) split8(z[i], sc, wh[i], wl[i]);
        dot = sum_groups(dot);
        if (half == 0 && g == 0 && on) A.dbeta[tok] = dot;
        mx = 0.f;
#pragma unroll
        for (int cb = 0; cb < DV / 16; ++cb) {
            float a[4];
            static_cast<const Four<BF16> *>(A.dout)[(tok * DV + 16 * cb) / 4 + g].get(a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[cb >> 1][4 * (cb & 1) + e] = on ? a[e] : 0.f;  // past the last token: 0
                mx = fmaxf(mx, fabsf(x[cb >> 1][4 * (cb & 1) + e]));
            }
        }
        sc = scale_to(max_groups(mx), 13, own_io);
#pragma unroll
        for (int i = 0; i < DVS; ++i) {
            half8 lo;
            split8(x[i], sc, oh[i], lo);
            if constexpr (NO == 2) ol[i] = lo;
        }
    }
    const float own_be = m.be[own], sk = m.sk[own], sq = m.sq[own];
    const float own_ik = 1.f / sk, own_iq = 1.f / sq;  // (powers of two)
    if (half == 0 && g == 0) {
        sh.iw[own] = own_iw;
        sh.iy[own] = own_iy;
        sh.io[own] = own_io;
        sh.ik[own] = own_ik;
        sh.iq[own] = own_iq;
        sh.be[own] = own_be;
    }
    // scalar gates: products inside blocks, one token a lane
    float gB[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (!KEYVEC) {
        const float a = lane < n ? s.a[(size_t)(first + lane) * s.H + h] : 1.f;
        float p = a, f = dpp<kShl + 1>(a, 1.f);
        p *= dpp<kShr + 1>(p, 1.f);
        p *= dpp<kShr + 2>(p, 1.f);
        p *= dpp<kShr + 4>(p, 1.f);
        p *= dpp<kShr + 8>(p, 1.f);
        f *= dpp<kShl + 1>(f, 1.f);
        f *= dpp<kShl + 2>(f, 1.f);
        f *= dpp<kShl + 4>(f, 1.f);
        f *= dpp<kShl + 8>(f, 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gB[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), 16 * i + 15));
        if (wave_index() == 0) {
            sh.pre[lane] = p;
            sh.suf[lane] = f;
            sh.ga[lane] = a;
        }
    }

    // ---- the states' parts: S dO, S y, dS w over the wave's half of the channels
    floatx4 vq[T], vk[T], vw[T];
    // a wave turns 16 channels of a state (tile), as they come (raw), into left operands
    const int tile = wave_index();
    auto put = [&](const floatx4 (&raw)[DV / 16], const floatx4 *dot_with) {
        if (tile < CT) {
            float x[DV / 16][4], mx = 0.f, inv;
            floatx4 dot = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int cb = 0; cb < DV / 16; ++cb) {
                if (dot_with) dot += raw[cb] * dot_with[cb];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[cb][r] = raw[cb][r];
                quad_transpose(x[cb]);
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, fabsf(x[cb][r]));
            }
            const float sc = scale_to(max_groups(mx), 10, inv);
#pragma unroll
            for (int cb = 0; cb < DV / 16; ++cb) {
                half4 hi, lo;
                split4(floatx4{x[cb][0], x[cb][1], x[cb][2], x[cb][3]}, sc, hi, lo);
                const int at = place(c16, g, cb >> 1);
                reinterpret_cast<half4 *>(&sh.st[0][tile][cb >> 1][at])[cb & 1] = hi;
                reinterpret_cast<half4 *>(&sh.st[1][tile][cb >> 1][at])[cb & 1] = lo;
            }
            if (g == 0) sh.srow[16 * tile + c16] = inv;
            if (dot_with) {              // before the turn a lane has a column of channels 4 (c16 / 4) ..
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float d = dot[r];
                    d += dpp0<quad(1, 0, 3, 2)>(d);
                    d += dpp0<quad(2, 3, 0, 1)>(d);
                    dot[r] = sum_groups(d);
                }
                if (g == 0 && (c16 & 3) == 0) *reinterpret_cast<floatx4 *>(&sh.rho[16 * tile + c16]) = dot;
            }
        }
        __syncthreads();
    };
    put(S, nullptr);
    fetch(A.dS, dS);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int ct = half * T + t;
        vq[t] = vk[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < DVS; ++i) {
            const int at = place(c16, g, i);
            const half8 lh = sh.st[0][ct][i][at], ll = sh.st[1][ct][i][at];
            vq[t] = mul<true, NO == 2>(lh, ll, oh[i], ol[NO == 2 ? i : 0], vq[t]);
            vk[t] = mul<true, true>(lh, ll, yh[i], yl[i], vk[t]);
        }
        const floatx4 f = four(&sh.srow[16 * ct + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            vq[t][r] = (vq[t][r] * f[r]) * own_io;
            vk[t][r] = -((vk[t][r] * f[r]) * own_iy) * own_be;
        }
    }
    __syncthreads();
    put(dS, S);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int ct = half * T + t;
        vw[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < DVS; ++i) {
            const int at = place(c16, g, i);
            vw[t] = mul<true, true>(sh.st[0][ct][i][at], sh.st[1][ct][i][at], wh[i], wl[i], vw[t]);
        }
        const floatx4 f = four(&sh.srow[16 * ct + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) vw[t][r] = ((vw[t][r] * f[r]) * own_iw) * own_be;
    }
    __syncthreads();


    if (half == 0) {
#pragma unroll
        for (int i = 0; i < DVS; ++i) {
            sh.t.w[0][w][i][lane] = wh[i];
            sh.t.w[1][w][i][lane] = wl[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < DVS; ++i) {
            sh.t.y[0][w][i][lane] = yh[i];
            sh.t.y[1][w][i][lane] = yl[i];
            sh.t.o[0][w][i][lane] = oh[i];
            if constexpr (NO == 2) sh.t.o[NO - 1][w][i][lane] = ol[i];
        }
    }
    __syncthreads();

    // ---- dP and dA: as columns of the own tokens, up to them (PT, AT) and from them on (P, Q)
    floatx4 PT[4], AT[4], PF[4], AF[4];
    {
        float near[2][4] = {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}};  // scalar decays inside the block
        if constexpr (!KEYVEC) {
            floatx4 gate[4];             // (read by all lanes: a choice of loads would be a branch each)
#pragma unroll
            for (int i = 0; i < 4; ++i) gate[i] = four(&sh.ga[16 * w + 4 * i]);
            float run = 1.f;             // rows j before the own token
#pragma unroll
            for (int j = 15; j >= 0; --j) {
                if (j < 15) run *= j < c16 ? gate[(j + 1) >> 2][(j + 1) & 3] : 1.f;
                near[0][j & 3] = j >> 2 == g ? run : near[0][j & 3];
            }
            run = 1.f;                   // rows i behind it
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                run *= i > c16 ? gate[i >> 2][i & 3] : 1.f;
                near[1][i & 3] = i >> 2 == g ? run : near[1][i & 3];
            }
        }
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            PT[J] = AT[J] = PF[J] = AF[J] = floatx4{0.f, 0.f, 0.f, 0.f};
            if (J <= w) {
#pragma unroll
                for (int i = 0; i < DVS; ++i) {
                    const half8 lh = sh.t.w[0][J][i][lane], ll = sh.t.w[1][J][i][lane];
                    PT[J] = mul<true, NO == 2>(lh, ll, oh[i], ol[NO == 2 ? i : 0], PT[J]);
                    AT[J] = mul<true, true>(lh, ll, yh[i], yl[i], AT[J]);
                }
                float d = 1.f;
                if constexpr (!KEYVEC) {
                    d = J < w ? sh.pre[own] : 1.f;
#pragma unroll
                    for (int x = 1; x < 3; ++x) d *= x > J && x < w ? gB[x] : 1.f;
                }
                const floatx4 be = four(&sh.be[16 * J + 4 * g]), iw = four(&sh.iw[16 * J + 4 * g]),
                              suf = KEYVEC ? be : four(&sh.suf[16 * J + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float f = be[r] * d;
                    if constexpr (!KEYVEC) f *= J < w ? suf[r] : near[0][r];
                    const float p = (PT[J][r] * iw[r] * own_io) * f, a = -(AT[J][r] * iw[r] * own_iy) * (f * own_be);
                    PT[J][r] = J < w || 4 * g + r <= c16 ? p : 0.f;
                    AT[J][r] = J < w || 4 * g + r < c16 ? a : 0.f;
                }
            }
            if (J >= w) {
#pragma unroll
                for (int i = 0; i < DVS; ++i) {
                    const half8 lh = sh.t.o[0][J][i][lane], ll = sh.t.o[NO - 1][J][i][lane];
                    PF[J] = mul<NO == 2, true>(lh, ll, wh[i], wl[i], PF[J]);
                    AF[J] = mul<true, true>(sh.t.y[0][J][i][lane], sh.t.y[1][J][i][lane], wh[i], wl[i], AF[J]);
                }
                float d = own_be;
                if constexpr (!KEYVEC) {
                    d *= J > w ? sh.suf[own] : 1.f;
#pragma unroll
                    for (int x = 1; x < 3; ++x) d *= x > w && x < J ? gB[x] : 1.f;
                }
                const floatx4 be = four(&sh.be[16 * J + 4 * g]), io = four(&sh.io[16 * J + 4 * g]),
                              iy = four(&sh.iy[16 * J + 4 * g]), pre = KEYVEC ? be : four(&sh.pre[16 * J + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float f = d;
                    if constexpr (!KEYVEC) f *= J > w ? pre[r] : near[1][r];
                    const float p = (PF[J][r] * io[r] * own_iw) * f, a = -(AF[J][r] * iy[r] * own_iw) * (f * be[r]);
                    PF[J][r] = J > w || 4 * g + r >= c16 ? p : 0.f;
                    AF[J][r] = J > w || 4 * g + r > c16 ? a : 0.f;
                }
            }
        }
    }
    if constexpr (KEYVEC) {
#pragma unroll
        for (int J = 0; J < 4; ++J)
            if (J == w && half == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    sh.d[0][w][c16][4 * g + r] = PT[J][r];
                    sh.d[1][w][c16][4 * g + r] = AT[J][r];
                }
    }

    __syncthreads();

    // ---- own rows of k and q with tokens in the lanes: channels 16 ct + 4 g .. + 3 of tile ct
    float k[T][4], q[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const size_t at = (tok * DK + 16 * (half * T + t)) / 4 + g;
        static_cast<const Four<BF16> *>(s.k)[at].get(k[t]);
        static_cast<const Four<BF16> *>(s.q)[at].get(q[t]);
    }
    // where the quad's turned values go: channel 4 g + c16 % 4, tokens 4 (c16 / 4) .. + 3
    const int turned = 4 * g + (c16 & 3) + 16 * (c16 >> 2);
    float dq[T][4], dr[T][4], dwr[T][4];  // dq; dk's reading parts; its writing parts inside the chunk
    Four<BF16> out;
    auto store = [&](void *to, int t, const float (&x)[4]) {
        out.set(x);
        if (on) static_cast<Four<BF16> *>(to)[(tok * DK + 16 * (half * T + t)) / 4 + g] = out;
    };

    if constexpr (!KEYVEC) {
        auto turn = [&](const float (&x)[4], float sc, half8 (&to)[NK][CT][2][64], int ct) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = x[r] * sc;
            quad_transpose(y);
            half4 hi, lo;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                _Float16 a, b;
                split(y[r], a, b);
                hi[r] = a;
                lo[r] = b;
            }
            reinterpret_cast<half4 *>(&to[0][ct][w >> 1][turned])[w & 1] = hi;
            if constexpr (NK == 2) reinterpret_cast<half4 *>(&to[NK - 1][ct][w >> 1][turned])[w & 1] = lo;
        };
        {
            // (the scales stand on the tokens, which are summed over: right operands take them off, so each
            // token has its own lane's)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                turn(k[t], sk, sh.c.k, half * T + t);
                turn(q[t], sq, sh.c.q, half * T + t);
            }
        }
        floatx4 YK[4], YQ[4];
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            const floatx4 ik = four(&sh.ik[16 * J + 4 * g]), iq = four(&sh.iq[16 * J + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                PT[J][r] *= ik[r];
                AT[J][r] *= ik[r];
                YK[J][r] = AF[J][r] * ik[r];
                YQ[J][r] = PF[J][r] * iq[r];
            }
        }
        float up, ua, uw;
        const float sp = scale_to(max_groups(tiles_max(PT)), 13, up), sa = scale_to(max_groups(tiles_max(AT)), 13, ua),
                    sw = scale_to(max_groups(tiles_max(YK, tiles_max(YQ))), 13, uw);
        half8 ph[2], pl[2], ah[2], al[2], kh[2], kl[2], qh[2], ql[2];
        auto pair = [&](const floatx4 (&X)[4], float sc, half8 (&hi)[2], half8 (&lo)[2]) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                half4 h0, l0, h1, l1;
                split4(X[2 * p], sc, h0, l0);
                split4(X[2 * p + 1], sc, h1, l1);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    hi[p][r] = h0[r];
                    hi[p][4 + r] = h1[r];
                    lo[p][r] = l0[r];
                    lo[p][4 + r] = l1[r];
                }
            }
        };
        pair(PT, sp, ph, pl);
        pair(AT, sa, ah, al);
        pair(YK, sw, kh, kl);
        pair(YQ, sw, qh, ql);
        __syncthreads();
        const float G = (w > 0 ? gB[0] : 1.f) * (w > 1 ? gB[1] : 1.f) * (w > 2 ? gB[2] : 1.f) * sh.pre[own];
        const float E = (w < 1 ? gB[1] : 1.f) * (w < 2 ? gB[2] : 1.f) * (w < 3 ? gB[3] : 1.f) * sh.suf[own];
        float e = 0.f, f = 0.f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int ct = half * T + t;
            floatx4 xp = {0.f, 0.f, 0.f, 0.f}, xa = xp, xw = xp;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const half8 a = sh.c.k[0][ct][p][lane], a2 = sh.c.k[NK - 1][ct][p][lane],
                            c = sh.c.q[0][ct][p][lane], c2 = sh.c.q[NK - 1][ct][p][lane];
                xp = mul<NK == 2, true>(a, a2, ph[p], pl[p], xp);
                xa = mul<NK == 2, true>(a, a2, ah[p], al[p], xa);
                xw = mul<NK == 2, true>(a, a2, kh[p], kl[p], xw);
                xw = mul<NK == 2, true>(c, c2, qh[p], ql[p], xw);
            }
            float all[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[t][r] = __builtin_fmaf(xp[r], up, G * vq[t][r]);
                dr[t][r] = __builtin_fmaf(xa[r], ua, G * vk[t][r]);
                dwr[t][r] = xw[r] * uw;
                const float ws = E * vw[t][r];
                e = __builtin_fmaf(q[t][r], dq[t][r], e);
                e = __builtin_fmaf(k[t][r], dr[t][r] - dwr[t][r], e);
                f = __builtin_fmaf(k[t][r], ws, f);
                all[r] = dr[t][r] + dwr[t][r] + ws;
            }
            store(A.dq, t, dq[t]);
            store(A.dk, t, all);
        }
        e = sum_groups(on ? e : 0.f);
        f = sum_groups(on ? f : 0.f);
        if (g == 0) {
            sh.es[half][own] = e;
            sh.fs[half][own] = f;
        }
        __syncthreads();
        if (wave_index() == 0) {
            float x = sh.es[0][lane] + sh.es[1][lane], y = sh.fs[0][lane] + sh.fs[1][lane], z = 0.f;
            for (int c = lane; c < DK; c += 64) z += sh.rho[c];
#pragma unroll
            for (int i = 1; i < 64; i <<= 1) {
                const float up = __shfl_down(x, i), down = __shfl_up(y, i);
                z += __shfl_xor(z, i);
                x += lane + i < 64 ? up : 0.f;
                y += lane >= i ? down : 0.f;
            }
            y = __shfl_up(y, 1);         // of the tokens before
            y = lane ? y : 0.f;
            const float a = sh.ga[lane], num = gB[0] * gB[1] * gB[2] * gB[3] * z + x + y;
            if (lane < n) A.da[(size_t)(first + lane) * s.H + h] = a > 0.f ? num / a : 0.f;
        }
    } else {
        float a[T][4], up[T][4], past[T][4];  // gates; their products in the block up to the token and past it
        const bool b1 = c16 & 1, b2 = c16 & 2, b4 = c16 & 4, b8 = c16 & 8;
        auto turn = [&](const float (&x)[4], float sc, half4 (&to)[2][CT][4][64], int ct) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = x[r] * sc;
            quad_transpose(y);
            half4 hi, lo;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                _Float16 a, b;
                split(y[r], a, b);
                hi[r] = a;
                lo[r] = b;
            }
            to[0][ct][w][turned] = hi;
            to[1][ct][w][turned] = lo;
        };
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int ct = half * T + t;
            const floatx4 av = four(s.a + tok * DK + 16 * ct + 4 * g);
            float ks[4], kp[4], qp[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x = on ? av[r] : 1.f;
                a[t][r] = x;
                const float p2 = pick(b1, dpp0<quad(0, 0, 2, 2)>(x) * x, x);
                const float p4 = pick(b2, dpp0<quad(1, 1, 1, 1)>(p2) * p2, p2);
                const float t4 = dpp0<quad(3, 3, 3, 3)>(p4);
                const float p8 = pick(b4, dpp0<kShr + 4>(t4) * p4, p4);
                up[t][r] = pick(b8, dpp0<kBcast + 7>(p8) * p8, p8);
                float f = pick(b1, 1.f, dpp0<quad(1, 1, 3, 3)>(x));
                f = pick(b2, f, dpp0<quad(3, 3, 3, 3)>(p2) * f);
                f = pick(b4, f, dpp0<kShl + 4>(t4) * f);
                past[t][r] = pick(b8, f, dpp0<kBcast + 15>(p8) * f);
                ks[r] = k[t][r] * past[t][r];
                kp[r] = k[t][r] * up[t][r];
                qp[r] = q[t][r] * up[t][r];
            }
            if (c16 == 15)
                *reinterpret_cast<floatx4 *>(&sh.B[w][16 * ct + 4 * g]) = floatx4{up[t][0], up[t][1], up[t][2], up[t][3]};
            turn(ks, sk, sh.v.y, ct);
            turn(kp, sk, sh.v.x, ct);
            turn(qp, sq, sh.v.z, ct);
        }
        // right operands: the other blocks' tiles
        floatx4 YK[4], YQ[4];
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            const floatx4 ik = four(&sh.ik[16 * J + 4 * g]), iq = four(&sh.iq[16 * J + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                PT[J][r] = J < w ? PT[J][r] * ik[r] : 0.f;
                AT[J][r] = J < w ? AT[J][r] * ik[r] : 0.f;
                YK[J][r] = J > w ? AF[J][r] * ik[r] : 0.f;
                YQ[J][r] = J > w ? PF[J][r] * iq[r] : 0.f;
            }
        }
        float undo_p, undo_a, undo_w;
        const float sp = scale_to(max_groups(tiles_max(PT)), 13, undo_p),
                    sa = scale_to(max_groups(tiles_max(AT)), 13, undo_a),
                    sw = scale_to(max_groups(tiles_max(YK, tiles_max(YQ))), 13, undo_w);
        __syncthreads();
        floatx4 xp[T], xa[T], xw[T];
#pragma unroll
        for (int t = 0; t < T; ++t) xp[t] = xa[t] = xw[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int J = 0; J < 3; ++J) {
            if (J >= w) continue;
            half4 ph, pl, ah, al;
            split4(PT[J], sp, ph, pl);
            split4(AT[J], sa, ah, al);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int ct = half * T + t;
                if (J > 0) {             // what came from before block J passes through it
                    const floatx4 f = four(&sh.B[J][16 * ct + 4 * g]);
                    xp[t] *= f;
                    xa[t] *= f;
                }
                const half4 lh = sh.v.y[0][ct][J][lane], ll = sh.v.y[1][ct][J][lane];
                xp[t] = mul4(lh, ll, ph, pl, xp[t]);
                xa[t] = mul4(lh, ll, ah, al, xa[t]);
            }
        }
#pragma unroll
        for (int J = 3; J > 0; --J) {
            if (J <= w) continue;
            half4 kh, kl, qh, ql;
            split4(YK[J], sw, kh, kl);
            split4(YQ[J], sw, qh, ql);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int ct = half * T + t;
                if (J < 3) xw[t] *= four(&sh.B[J][16 * ct + 4 * g]);
                xw[t] = mul4(sh.v.x[0][ct][J][lane], sh.v.x[1][ct][J][lane], kh, kl, xw[t]);
                xw[t] = mul4(sh.v.z[0][ct][J][lane], sh.v.z[1][ct][J][lane], qh, ql, xw[t]);
            }
        }
        const float pii = sh.d[0][w][c16][c16];
        float f[T][4];                   // k (beta E dS w)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int ct = half * T + t;
            floatx4 G = {1.f, 1.f, 1.f, 1.f}, E = G;
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                const floatx4 x = four(&sh.B[J][16 * ct + 4 * g]);
                if (J < w) G *= x;
                if (J > w) E *= x;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[t][r] = up[t][r] * __builtin_fmaf(xp[t][r], undo_p, G[r] * vq[t][r]);
                dr[t][r] = up[t][r] * __builtin_fmaf(xa[t][r], undo_a, G[r] * vk[t][r]);
                dwr[t][r] = past[t][r] * (xw[t][r] * undo_w);
                vw[t][r] *= past[t][r] * E[r];
                f[t][r] = k[t][r] * vw[t][r];
                dq[t][r] = __builtin_fmaf(pii, k[t][r], dq[t][r]);
                dwr[t][r] = __builtin_fmaf(pii, q[t][r], dwr[t][r]);
            }
        }
        distances<1, T>(sh, w, c16, k, q, a, up, past, dq, dr, dwr);
        // sums over the tokens behind (e) and before (f), within the block by lanes
        float e[T][4];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int ct = half * T + t;
            float all[4];
            floatx4 se, sf;              // sums over the block
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                all[r] = dr[t][r] + dwr[t][r] + vw[t][r];
                float x = __builtin_fmaf(q[t][r], dq[t][r], k[t][r] * (dr[t][r] - dwr[t][r]));
                x = on ? x : 0.f;
                x += dpp0<kShl + 1>(x);
                x += dpp0<kShl + 2>(x);
                x += dpp0<kShl + 4>(x);
                x += dpp0<kShl + 8>(x);
                e[t][r] = x;
                float y = on ? f[t][r] : 0.f;
                y += dpp0<kShr + 1>(y);
                y += dpp0<kShr + 2>(y);
                y += dpp0<kShr + 4>(y);
                y += dpp0<kShr + 8>(y);
                se[r] = x;
                sf[r] = y;
                f[t][r] = dpp0<kShr + 1>(y);
            }
            if (c16 == 0) *reinterpret_cast<floatx4 *>(&sh.te[w][16 * ct + 4 * g]) = se;
            if (c16 == 15) *reinterpret_cast<floatx4 *>(&sh.tf[w][16 * ct + 4 * g]) = sf;
            store(A.dq, t, dq[t]);
            store(A.dk, t, all);
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int ct = half * T + t;
            floatx4 x = four(&sh.rho[16 * ct + 4 * g]), sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                x *= four(&sh.B[J][16 * ct + 4 * g]);
                if (J > w) sum += four(&sh.te[J][16 * ct + 4 * g]);
                if (J < w) sum += four(&sh.tf[J][16 * ct + 4 * g]);
            }
            floatx4 d;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float num = x[r] + sum[r] + e[t][r] + f[t][r];
                d[r] = a[t][r] > 0.f ? num / a[t][r] : 0.f;
            }
            if (on) *reinterpret_cast<floatx4 *>(A.da + tok * DK + 16 * ct + 4 * g) = d;
        }
    }
}

template <int DK, int DV>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)a.slots * (unsigned)a.s.H);
    if (keyvec && bf16) k_chunk_grad<DK, DV, true, true><<<grid, 512, 0, s>>>(a);
    else if (keyvec) k_chunk_grad<DK, DV, true, false><<<grid, 512, 0, s>>>(a);
    else if (bf16) k_chunk_grad<DK, DV, false, true><<<grid, 512, 0, s>>>(a);
    else k_chunk_grad<DK, DV, false, false><<<grid, 512, 0, s>>>(a);
}

}  // namespace

hipError_t launch_chunk_grad(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && dv == 64) go<64, 64>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, 128>(a, keyvec, bf16, s);
    else if (dv == 64) go<128, 64>(a, keyvec, bf16, s);
    else go<128, 128>(a, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
