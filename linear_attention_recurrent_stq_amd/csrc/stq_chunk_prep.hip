// What the chunks of a batch need before the state passes through them:
// T and P (stq_chunk.h) and the factors of every token.  One workgroup of four
// waves per (chunk, head), all chunks at once; wave w holds rows 16 w .. 16 w + 15 as
// matrix operands, lane (r, g) the row r's channels 32 s + 8 g .. + 7.
//
// A and P are lower triangular, in 16x16 blocks (I, J).  With pre_i the product of
// the gates from its block's start to i, suf_j of those after j in its block, and
// mid the product of the blocks between, a block off the diagonal has the decay
// pre_i mid suf_j: products of gates only, at most 1.
//
// Scalar gates: A and P are K K^T and Q K^T times the decay; bf16 rows multiply
// exactly on bf16 matrix instructions, fp32 rows on fp32 ones.  Inside a diagonal block
// the decay is a running product down each column.
//
// Key-vector gates: the decay sits inside the sum over channels, so the rows are
// multiplied by it first, (q, k) pre (mid) against k suf.  A diagonal block is cut the
// same way, at 8 and at 4 (X of the later half's rows and, in the rows that it
// leaves free, Q's: one product a cut), down to 4x4 blocks, which are vector code:
// the three earlier rows of a quad of lanes are read across lanes.  Products of gates
// within 2, 4, 8 and 16 rows come from one scan across the lanes of a row of 16.  These
// operands are scaled fp16 pairs.
//
// T: the 16x16 diagonal blocks of I + diag(beta) A are inverted by forward
// substitution, a wave each; a wave then builds one block column of the inverse,
// T_IJ = -X_I sum_m M_Im T_mJ, with fp32 matrix instructions.  A result tile is a
// right operand in the registers it is in, so the chain needs no exchange.
//
// The bound is vector instructions (65 to 69 % of the cycles, the rest latency). Measured, bf16, d_k
// 128, 32 heads, MI355X: scalar gates, 24000 tokens 215 us (478 MB: 2.2 TB/s); key-vector gates,
// 16001 tokens 361 to 377 us (589 MB: 1.6 TB/s).
//
// Rows past a chunk's last token repeat it, with beta 0 and gate 1: their rows and
// columns of T are 0, and their outputs are not stored.
#include "stq_chunk.h"

namespace stq {
namespace {

constexpr int LD = kC + 4;  // row stride of M in LDS

template <int DK, bool BF16>
struct Rows {
    Row8<BF16> k[DK / 32], q[DK / 32];
    size_t at;                       // of the lane's first channel
    float sk, ik, sq, iq;            // scales of the row and what undoes them

    __device__ void load(const SeqArgs &s, int h, int first, int n) {
        const int lane = threadIdx.x & 63, row = 16 * wave_index() + (lane & 15);
        at = ((size_t)(first + min(row, n - 1)) * s.H + h) * DK + 8 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            k[i].load(s.k, at + 32 * i);
            q[i].load(s.q, at + 32 * i);
        }
    }
    __device__ void scales() {
        float mk = 0.f, mq = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mk = fmaxf(mk, fabsf(k[i].get(e)));
                mq = fmaxf(mq, fabsf(q[i].get(e)));
            }
        sk = scale_to(max_groups(mk), 10, ik);
        sq = scale_to(max_groups(mq), 10, iq);
    }
};

// A 16x16 result tile times its rows' scales s, as fp16 pairs in fragment order;
// tile (I, J) of a lower triangular matrix.  LO: with the lo part.
template <bool LO>
__device__ inline void store_tile(floatx4 x, floatx4 s, int I, int J, uint16_t (&to)[2][kTri][kFrag]) {
    const int c16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = x[r] * s[r];
    quad_transpose(y);
    half4 hi, lo;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        _Float16 a, b;
        split(y[r], a, b);
        hi[r] = a;
        lo[r] = b;
    }
    const int f = I < 2 ? I : 2 + 2 * (I - 2) + (J >> 1);
    const int at = (4 * g + (c16 & 3) + 16 * (c16 >> 2)) * 8 + (J & 1) * 4;
    *reinterpret_cast<half4 *>(&to[0][f][at]) = hi;
    if constexpr (LO) *reinterpret_cast<half4 *>(&to[1][f][at]) = lo;
}

// The transpose of tile (I, J) times its rows' scale s (columns of the tile): a lane
// holds four of its row's values as they stand in the fragment.
__device__ inline void store_transposed(floatx4 x, float s, int I, int J, uint16_t (&to)[2][kTri][kFrag]) {
    half4 hi, lo;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        _Float16 a, b;
        split(x[r], s, a, b);
        hi[r] = a;
        lo[r] = b;
    }
    const int f = J < 2 ? 2 * J + (I >> 1) : 2 + J, at = (threadIdx.x & 63) * 8 + (I & 1) * 4;
    *reinterpret_cast<half4 *>(&to[0][f][at]) = hi;
    *reinterpret_cast<half4 *>(&to[1][f][at]) = lo;
}

// Row w of the blocks of P, transposed (backward); `tm`: [4][64] in LDS, written here.
__device__ inline void store_pt(const floatx4 (&p)[4], float (*tm)[kC], ChunkMeta &m, ChunkBack &out) {
    const int lane = threadIdx.x & 63, w = wave_index(), c16 = lane & 15;
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        float x = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) x = fmaxf(x, J <= w ? fabsf(p[J][r]) : 0.f);
        x = max_groups(x);
        if (lane < 16) tm[w][16 * J + c16] = x;
    }
    __syncthreads();
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        float x = 0.f, inv;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fmaxf(x, tm[i][16 * J + c16]);
        const float sc = scale_to(x, 10, inv);
        if (J <= (w | 1)) store_transposed(J <= w ? p[J] : floatx4{0.f, 0.f, 0.f, 0.f}, sc, w, J, out.P);
        if (J == w && lane < 16) m.rpt[16 * J + c16] = inv;
    }
    __syncthreads();
}

// Row w of P's blocks.  LO: for fp32 outputs; bf16 ones take the hi part alone.
template <bool LO>
__device__ inline void store_p(const floatx4 (&p)[4], ChunkPrep &out) {
    const int lane = threadIdx.x & 63, w = wave_index(), c16 = lane & 15, g = lane >> 4;
    floatx4 s, inv;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float m = 0.f, x;
#pragma unroll
        for (int J = 0; J < 4; ++J) m = fmaxf(m, J <= w ? fabsf(p[J][r]) : 0.f);
        s[r] = scale_to(max_row(m), 10, x);
        inv[r] = x;
    }
#pragma unroll
    for (int J = 0; J < 4; ++J)
        if (J <= (w | 1)) store_tile<LO>(J <= w ? p[J] : floatx4{0.f, 0.f, 0.f, 0.f}, s, w, J, out.P);
    if (c16 == 0) *reinterpret_cast<floatx4 *>(&out.m.rp[16 * w + 4 * g]) = inv;
}

// Block column `wave` of the inverse of I + M, M strictly lower triangular in LDS (what lies above
// the diagonal is not read).
__device__ inline void invert(const float (*M)[LD], float (*X)[20], floatx4 (&t)[4]) {
    const int lane = threadIdx.x & 63, wave = wave_index(), j = lane & 15, g = lane >> 4;
    // inverse of the diagonal block `wave`, column j
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == j ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < i; m += 4) {
            const floatx4 f = four(&M[16 * wave + i][16 * wave + m]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < i) s = __builtin_fmaf(-f[e], x[m + e], s);
        }
        x[i] = s;
    }
    if (g == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) X[16 * wave + i][j] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int I = 0; I < 4; ++I) {
        if (I < wave) {
            t[I] = floatx4{0.f, 0.f, 0.f, 0.f};
        } else if (I == wave) {
#pragma unroll
            for (int r = 0; r < 4; ++r) t[I][r] = X[16 * I + 4 * g + r][j];
        } else {
            floatx4 y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
            for (int m = 0; m < I; ++m) {
                if (m < wave) continue;
                const floatx4 a = four(&M[16 * I + j][16 * m + 4 * g]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y = mfma_f32(a[e], t[m][e], y);
            }
            const floatx4 a = four(&X[16 * I + j][4 * g]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z = mfma_f32(-a[e], y[e], z);
            t[I] = z;
        }
    }
}

// From M = diag(beta) A in LDS to T; backward: to N^T, and from A diag(beta), written over M, to
// N' = (I + A diag(beta))^-1, which takes R to the delta errors w, in T's place.
template <bool BACK>
__device__ inline void store_t(float (*M)[LD], float (*X)[20], float (*tm)[kC], const float *be, const floatx4 (&A)[4],
                               ChunkPrep &out, ChunkBack *back) {
    const int lane = threadIdx.x & 63, wave = wave_index(), j = lane & 15, g = lane >> 4;
    floatx4 t[4];
    invert(M, X, t);
    const float b = be[16 * wave + j];
    if constexpr (BACK) {
        float m = 0.f, inv;
#pragma unroll
        for (int I = 0; I < 4; ++I)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(t[I][r]));
        const float s = scale_to(max_groups(m), 10, inv);
#pragma unroll
        for (int I = 0; I < 4; ++I)
            if ((I | 1) >= wave) store_transposed(t[I], s, I, wave, back->N);
        if (g == 0) {
            out.m.rn[16 * wave + j] = inv;
            out.m.be[16 * wave + j] = b;
        }
        __syncthreads();
#pragma unroll
        for (int J = 0; J < 4; ++J)
            if (J <= wave)
#pragma unroll
                for (int r = 0; r < 4; ++r) M[16 * wave + 4 * g + r][16 * J + j] = A[J][r] * be[16 * J + j];
        __syncthreads();
        invert(M, X, t);
    }
#pragma unroll
    for (int I = 0; I < 4; ++I) {
        floatx4 m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (!BACK) t[I][r] *= b;
            m[r] = max_row(fabsf(t[I][r]));
        }
        if (j == 0) *reinterpret_cast<floatx4 *>(&tm[wave][16 * I + 4 * g]) = m;
    }
    __syncthreads();
#pragma unroll
    for (int I = 0; I < 4; ++I) {
        if ((I | 1) < wave) continue;
        floatx4 m = four(&tm[0][16 * I + 4 * g]), s, inv;
#pragma unroll
        for (int J = 1; J < 4; ++J)
#pragma unroll
            for (int r = 0; r < 4; ++r) m[r] = fmaxf(m[r], tm[J][16 * I + 4 * g + r]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float x;
            s[r] = scale_to(m[r], 10, x);
            inv[r] = x;
        }
        store_tile<true>(t[I], s, I, wave, out.T);
        if (I == wave && j == 0) *reinterpret_cast<floatx4 *>(&out.m.rt[16 * I + 4 * g]) = inv;
    }
}

// The sequences by length, longest first (one workgroup): the pass of the state takes as
// long as its last sequence to end, and few sequences fill the chip at a time.
__device__ inline void order_sequences(const ChunkArgs &A, int *len) {
    for (int b = threadIdx.x; b < A.s.B; b += 256) {
        int t0, t1;
        seq_range(A.s, b, t0, t1);
        len[b] = t1 - t0;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < A.s.B; b += 256) {
        int at = 0;
        for (int i = 0; i < A.s.B; ++i) at += len[i] > len[b] || (len[i] == len[b] && i < b);
        A.order[at] = b;
    }
}

// BACK: what the backward pass reads (N' in T's place, N^T and P^T).
template <int DK, bool BF16, bool BACK>
__global__ void __launch_bounds__(256) k_prep_scalar(const ChunkArgs A) {
    constexpr int KS = DK / 32;
    __shared__ union {
        float M[kC][LD];
        Row8<BF16> rows[4][KS][64];  // K as operands, until M is written
    } big;
    __shared__ __align__(16) float X[kC][20], tm[4][kC], pre[kC], suf[kC], ga[kC], be[kC];
    const SeqArgs &s = A.s;
    static_assert(sizeof(X) >= kOrdered * sizeof(int), "the lengths fit");
    if (blockIdx.x == (uint32_t)A.slots * (uint32_t)s.H) return order_sequences(A, reinterpret_cast<int *>(&X[0][0]));
    uint32_t slot, h;
    xcd_place(blockIdx.x, s.H, slot, h);
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index(), c16 = lane & 15, g = lane >> 4;
    int b, first;
    const int n = chunk_of_slot(s, slot, b, first);
    if (n == 0) return;
    ChunkPrep &out = A.prep[(size_t)slot * s.H + h];
    Rows<DK, BF16> x;
    x.load(s, h, first, n);
    // gates of all 64 tokens, one a lane
    const size_t tok = (size_t)(first + min(lane, n - 1)) * s.H + h;
    const float a = lane < n ? s.a[tok] : 1.f, beta = lane < n ? s.beta[tok] : 0.f;
    float p = a, f = dpp<kShl + 1>(a, 1.f);
    p *= dpp<kShr + 1>(p, 1.f);
    p *= dpp<kShr + 2>(p, 1.f);
    p *= dpp<kShr + 4>(p, 1.f);
    p *= dpp<kShr + 8>(p, 1.f);
    f *= dpp<kShl + 1>(f, 1.f);
    f *= dpp<kShl + 2>(f, 1.f);
    f *= dpp<kShl + 4>(f, 1.f);
    f *= dpp<kShl + 8>(f, 1.f);
    float B[4];                      // products of the blocks
#pragma unroll
    for (int i = 0; i < 4; ++i)
        B[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), 16 * i + 15));
    if (wave == 0) {
        pre[lane] = p;
        suf[lane] = f;
        ga[lane] = a;
        be[lane] = beta;
    }
    x.scales();
#pragma unroll
    for (int i = 0; i < KS; ++i) big.rows[wave][i][lane] = x.k[i];
    const int row = 16 * wave + c16;
    __syncthreads();
    if (g == 0) {
        const float G = (wave > 0 ? B[0] : 1.f) * (wave > 1 ? B[1] : 1.f) * (wave > 2 ? B[2] : 1.f) * pre[row];
        const float E = (wave < 1 ? B[1] : 1.f) * (wave < 2 ? B[2] : 1.f) * (wave < 3 ? B[3] : 1.f) * suf[row];
        out.m.sk[row] = x.sk;
        out.m.sq[row] = x.sq;
        out.m.rk[row] = x.ik * G;
        out.m.rq[row] = x.iq * G;
        out.m.rw[row] = x.ik * E;
    }
    if (tid < 128) out.m.dec[tid] = B[0] * B[1] * B[2] * B[3];

    floatx4 aa[4], pp[4];
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        aa[J] = pp[J] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (J > wave) continue;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const Row8<BF16> y = big.rows[J][i][lane];
            if constexpr (BF16) {
                const bf16x8 kr = __builtin_bit_cast(bf16x8, x.k[i].w), qr = __builtin_bit_cast(bf16x8, x.q[i].w);
                const bf16x8 kc = __builtin_bit_cast(bf16x8, y.w);
                aa[J] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kr, kc, aa[J], 0, 0, 0);
                pp[J] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qr, kc, pp[J], 0, 0, 0);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    aa[J] = mfma_f32(x.k[i].get(e), y.get(e), aa[J]);
                    pp[J] = mfma_f32(x.q[i].get(e), y.get(e), pp[J]);
                }
            }
        }
    }
    const floatx4 pi = four(&pre[16 * wave + 4 * g]), bi = four(&be[16 * wave + 4 * g]);
    floatx4 dd;                      // decay inside the diagonal block
    {
        float run = 1.f;
        floatx4 gate[4];             // (read by all lanes: a choice of loads would be a branch each)
#pragma unroll
        for (int i = 0; i < 4; ++i) gate[i] = four(&ga[16 * wave + 4 * i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            run *= i > c16 ? gate[i >> 2][i & 3] : 1.f;
            dd[i & 3] = i >> 2 == g ? run : i < 4 ? 1.f : dd[i & 3];
        }
    }
    __syncthreads();
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        if (J > wave) continue;
        float sj = suf[16 * J + c16];
#pragma unroll
        for (int m = 1; m < 3; ++m) sj *= m > J && m < wave ? B[m] : 1.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * g + r;
            const float d = J < wave ? pi[r] * sj : i >= c16 ? dd[r] : 0.f;
            aa[J][r] = J < wave || i > c16 ? aa[J][r] * d : 0.f;
            big.M[16 * wave + i][16 * J + c16] = bi[r] * aa[J][r];
            pp[J][r] = J < wave || i >= c16 ? pp[J][r] * d : 0.f;
        }
    }
    ChunkBack *back = nullptr;
    if constexpr (BACK) {
        back = A.back + (size_t)slot * s.H + h;
        store_pt(pp, tm, out.m, *back);
    } else {
        store_p<!BF16>(pp, out);
    }
    __syncthreads();
    store_t<BACK>(big.M, X, tm, be, aa, out, back);
}

template <int DK, bool BF16, bool BACK>
__global__ void __launch_bounds__(256, 2) k_prep_keyvec(const ChunkArgs A) {
    constexpr int KS = DK / 32;
    __shared__ union {
        float M[kC][LD];
        float g[2][kC / 4][DK];      // products up to and after each four rows of a block, until M is written
    } big;
    __shared__ __align__(16) union {
        half8 Y[3][KS][2][64];       // k suf of waves 0 to 2
        struct {
            float X[kC][20], dp[4][16][20], da[4][16][20];  // once Y is done with
        } f;
    } two;
    auto &Y = two.Y;
    auto &X = two.f.X;
    auto &dp = two.f.dp;
    auto &da_ = two.f.da;
    __shared__ __align__(16) float tm[4][kC], ik[kC], iq[kC], be[kC];
    const SeqArgs &s = A.s;
    static_assert(sizeof(X) >= kOrdered * sizeof(int), "the lengths fit");
    if (blockIdx.x == (uint32_t)A.slots * (uint32_t)s.H) return order_sequences(A, reinterpret_cast<int *>(&X[0][0]));
    uint32_t slot, h;
    xcd_place(blockIdx.x, s.H, slot, h);
    const int tid = threadIdx.x, lane = tid & 63, w = wave_index(), c16 = lane & 15, g = lane >> 4;
    int b, first;
    const int n = chunk_of_slot(s, slot, b, first);
    if (n == 0) return;
    ChunkPrep &out = A.prep[(size_t)slot * s.H + h];
    Rows<DK, BF16> x;
    x.load(s, h, first, n);
    x.scales();
    const int row = 16 * w + c16;
    if (g == 0) {
        ik[row] = x.ik;
        iq[row] = x.iq;
        be[row] = row < n ? s.beta[(size_t)(first + row) * s.H + h] : 0.f;
        out.m.sk[row] = x.sk;
        out.m.sq[row] = x.sq;
        out.m.rk[row] = out.m.rw[row] = x.ik;
        out.m.rq[row] = x.iq;
    }
    const bool b1 = c16 & 1, b2 = c16 & 2, b4 = c16 & 4, b8 = c16 & 8, on = row < n;
    float kp[KS][8], qp[KS][8];      // k pre, q pre, scaled
    floatx4 cut4 = {0.f, 0.f, 0.f, 0.f}, cut8 = cut4;
    float da[3] = {}, dq[4] = {};    // 4x4 blocks: rows d earlier, A for d = 1, 2, 3 and P for d = 0 .. 3
    floatx4 n0 = four(s.a + x.at), n1 = four(s.a + x.at + 4);  // the next channels' gates
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const floatx4 a0 = n0, a1 = n1;
        if (i + 1 < KS) {
            n0 = four(s.a + x.at + 32 * i + 32);
            n1 = four(s.a + x.at + 32 * i + 36);
        }
        __builtin_amdgcn_sched_barrier(0);
        float z4[8], z8[8], y4[8], y8[8], y16[8];
        floatx4 pe[2], fe[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = on ? e < 4 ? a0[e & 3] : a1[e & 3] : 1.f, k = x.k[i].get(e), q = x.q[i].get(e);
            // 4x4 blocks
            dq[0] = __builtin_fmaf(q, k, dq[0]);
            float v = dpp0<kShr + 1>(k) * a;
            da[0] = __builtin_fmaf(k, v, da[0]);
            dq[1] = __builtin_fmaf(q, v, dq[1]);
            float d = a * dpp0<kShr + 1>(a);
            v = dpp0<kShr + 2>(k) * d;
            da[1] = __builtin_fmaf(k, v, da[1]);
            dq[2] = __builtin_fmaf(q, v, dq[2]);
            d *= dpp0<kShr + 2>(a);
            v = dpp0<kShr + 3>(k) * d;
            da[2] = __builtin_fmaf(k, v, da[2]);
            dq[3] = __builtin_fmaf(q, v, dq[3]);
            // products within 2, 4, 8 and 16 rows: up to the row (p), after it (f)
            // (the value across lanes is multiplied first and chosen then: it folds into the product)
            const float p2 = pick(b1, dpp0<quad(0, 0, 2, 2)>(a) * a, a);
            const float p4 = pick(b2, dpp0<quad(1, 1, 1, 1)>(p2) * p2, p2);
            const float t4 = dpp0<quad(3, 3, 3, 3)>(p4);
            const float p8 = pick(b4, dpp0<kShr + 4>(t4) * p4, p4);
            const float p16 = pick(b8, dpp0<kBcast + 7>(p8) * p8, p8);
            const float ks = k * x.sk, qs = q * x.sq;  // (powers of two)
            float f = pick(b1, 1.f, dpp0<quad(1, 1, 3, 3)>(a));
            f = pick(b2, f, dpp0<quad(3, 3, 3, 3)>(p2) * f);
            y4[e] = ks * f;
            f = pick(b4, f, dpp0<kShl + 4>(t4) * f);
            y8[e] = ks * f;
            f = pick(b8, f, dpp0<kBcast + 15>(p8) * f);
            y16[e] = ks * f;
            // the later half's rows of K, and of Q in the rows that the earlier half leaves free
            z4[e] = pick(b4, ks * p4, dpp0<kShl + 4>(qs * p4));
            z8[e] = pick(b8, ks * p8, dpp0<kShl + 8>(qs * p8));
            kp[i][e] = ks * p16;
            qp[i][e] = qs * p16;
            asm volatile("" : "+v"(kp[i][e]), "+v"(qp[i][e]));  // (formed here, not where a wave uses them)
            pe[e >> 2][e & 3] = p16;
            fe[e >> 2][e & 3] = f;
        }
        // (sums formed here: moved to where they are used they would keep every term)
        asm volatile("" : "+v"(da[0]), "+v"(da[1]), "+v"(da[2]), "+v"(dq[0]), "+v"(dq[1]), "+v"(dq[2]), "+v"(dq[3]));
        if ((c16 & 3) == 3) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                *reinterpret_cast<floatx4 *>(&big.g[0][row >> 2][32 * i + 8 * g + 4 * e]) = pe[e];
                *reinterpret_cast<floatx4 *>(&big.g[1][row >> 2][32 * i + 8 * g + 4 * e]) = fe[e];
            }
        }
        half8 zh, zl, yh, yl;
        split8(z4, zh, zl);
        split8(y4, yh, yl);
        cut4 = mfma_pairs(zh, zl, yh, yl, cut4);
        split8(z8, zh, zl);
        split8(y8, yh, yl);
        cut8 = mfma_pairs(zh, zl, yh, yl, cut8);
        if (w < 3) {
            split8(y16, yh, yl);
            Y[w][i][0][lane] = yh;
            Y[w][i][1][lane] = yl;
        }
    }
    __syncthreads();
    // gate products of the whole chunk before and after each four tokens
    {
        ChunkGates &o = A.gates[(size_t)slot * s.H + h];
        const int c = tid % DK;
        float B[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) B[i] = big.g[0][4 * i + 3][c];
#pragma unroll
        for (int i = 0; i < 16 * DK / 256; ++i) {
            const int q4 = tid / DK + 256 / DK * i, blk = q4 >> 2;
            float u = big.g[0][q4 ? q4 - 1 : 0][c], v = big.g[1][q4][c];
            u = q4 & 3 ? u : 1.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                u *= m < blk ? B[m] : 1.f;
                v *= m > blk ? B[m] : 1.f;
            }
            o.pre[q4][c] = u;
            o.suf[q4][c] = v;
        }
        if (tid < DK) out.m.dec[c] = B[0] * B[1] * B[2] * B[3];
    }
    floatx4 aa[4], pp[4];
#pragma unroll
    for (int J = 2; J >= 0; --J) {
        aa[J] = pp[J] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (J >= w) continue;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (J < w - 1) {         // the block between, J + 1, comes in
                const float *m = &big.g[0][4 * J + 7][32 * i + 8 * g];
                const floatx4 m0 = four(m), m1 = four(m + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    kp[i][e] *= e < 4 ? m0[e & 3] : m1[e & 3];
                    qp[i][e] *= e < 4 ? m0[e & 3] : m1[e & 3];
                }
            }
            const half8 yh = Y[J][i][0][lane], yl = Y[J][i][1][lane];
            half8 zh, zl;
            split8(kp[i], zh, zl);
            aa[J] = mfma_pairs(zh, zl, yh, yl, aa[J]);
            split8(qp[i], zh, zl);
            pp[J] = mfma_pairs(zh, zl, yh, yl, pp[J]);
        }
    }
    __syncthreads();
    const floatx4 bi = four(&be[16 * w + 4 * g]), iki = four(&ik[16 * w + 4 * g]), iqi = four(&iq[16 * w + 4 * g]);
#pragma unroll
    for (int J = 0; J < 3; ++J) {
        if (J >= w) continue;
        const float ikj = ik[16 * J + c16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            aa[J][r] = aa[J][r] * iki[r] * ikj;
            big.M[16 * w + 4 * g + r][16 * J + c16] = bi[r] * aa[J][r];
            pp[J][r] = pp[J][r] * iqi[r] * ikj;
        }
    }
    // the diagonal block, from its cuts
    const bool both = g & 1;         // cut 4: groups 1 and 3 hold A of rows 4 g .., 0 and 2 P of rows 4 g + 4 ..
    if (g < 2 ? c16 < 4 : c16 >= 8 && c16 < 12) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * (g | 1) + r;
            if (both) da_[w][i][c16] = cut4[r] * ik[16 * w + i] * x.ik;
            else dp[w][i][c16] = cut4[r] * iq[16 * w + i] * x.ik;
        }
    }
    if (c16 < 8) {                   // cut 8: groups 2 and 3 A of rows 4 g .., 0 and 1 P of rows 4 g + 8 ..
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * (g | 2) + r;
            if (g & 2) da_[w][i][c16] = cut8[r] * ik[16 * w + i] * x.ik;
            else dp[w][i][c16] = cut8[r] * iq[16 * w + i] * x.ik;
        }
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float p = sum_groups(dq[d]), m = sum_groups(d ? da[d - 1] : 0.f);
        if (g == 0 && (c16 & 3) >= d) {
            dp[w][c16][c16 - d] = p;
            da_[w][c16][c16 - d] = m;
        }
    }
    __syncthreads();
#pragma unroll
    for (int J = 0; J < 4; ++J)
        if (J == w)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * g + r;
                const float p = dp[w][i][c16], m = da_[w][i][c16];
                pp[J][r] = i >= c16 ? p : 0.f;
                aa[J][r] = i > c16 ? m : 0.f;
                big.M[16 * w + i][16 * w + c16] = bi[r] * aa[J][r];
            }
    ChunkBack *back = nullptr;
    if constexpr (BACK) {
        back = A.back + (size_t)slot * s.H + h;
        store_pt(pp, tm, out.m, *back);
    } else {
        store_p<!BF16>(pp, out);
    }
    __syncthreads();
    store_t<BACK>(big.M, X, tm, be, aa, out, back);
}

template <int DK, bool BACK>
void go(const ChunkArgs &a, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)a.slots * (unsigned)a.s.H + (a.order ? 1u : 0u));
    if (keyvec && bf16) k_prep_keyvec<DK, true, BACK><<<grid, 256, 0, s>>>(a);
    else if (keyvec) k_prep_keyvec<DK, false, BACK><<<grid, 256, 0, s>>>(a);
    else if (bf16) k_prep_scalar<DK, true, BACK><<<grid, 256, 0, s>>>(a);
    else k_prep_scalar<DK, false, BACK><<<grid, 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_chunk_prep(const ChunkArgs &a, int dk, bool keyvec, bool bf16, hipStream_t s) {
    if (dk == 64 && a.back) go<64, true>(a, keyvec, bf16, s);
    else if (dk == 64) go<64, false>(a, keyvec, bf16, s);
    else if (a.back) go<128, true>(a, keyvec, bf16, s);
    else go<128, false>(a, keyvec, bf16, s);
    return hipGetLastError();
}

}  // namespace stq
