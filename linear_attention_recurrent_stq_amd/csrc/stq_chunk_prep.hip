// What the chunks of a batch need before the state passes through them:
// T and P (stq_chunk.h) and the factors of every token.  One workgroup of four
// waves per (chunk, head); all chunks at once.
//
// Scalar gates: A and P are K K^T and Q K^T times D_ij = prod_{j<s<=i} a_s.  The
// products of bf16 rows run on bf16 matrix instructions (exact products, fp32
// sums), fp32 rows on fp32 ones.  D is formed by running products down its
// columns, 16 rows at a time by 256 threads.
//
// Key-vector gates: the decay sits inside the sum over channels.  It is split at
// a token between i and j: at 32 for the lower left quarter, at 16 and 48 for
// the blocks next to the diagonal ones, so that both factors, prod from the
// split to i and prod from j to the split, are products of gates (at most 1)
// and the block is one matrix product (fp32 matrix instructions).  The four
// 16x16 blocks on the diagonal have no such split: a lane holds k_j for 32
// channels, multiplies a_i in for each next i and forms the dot products with k_i
// and q_i; they are vector code.
//
// T: the 16x16 diagonal blocks of I + diag(beta) A are inverted by forward
// substitution, a wave each; a wave then builds one block column of the inverse,
// T_IJ = -X_I sum_m M_Im T_mJ, with fp32 matrix instructions.  A result tile is a
// right operand in the registers it is in, so the chain needs no exchange.
#include "stq_chunk.h"

namespace stq {
namespace {

constexpr int LD = kC + 4;  // row stride of 64x64 matrices in LDS

struct PrepShared {
    float be[kC], ik[kC], iq[kC];    // beta; inverse scales of K and Q rows
};

// Row scales of K and Q: thread (row, quarter) looks at a quarter of the row.
// Rows past the last token take its scales: the pass of the state reads its row there.
template <int DK, bool BF16>
__device__ inline void row_scales(const SeqArgs &s, int h, int first, int n, ChunkMeta &m, PrepShared &sh) {
    constexpr int W = DK / 4;
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
    float mk = 0.f, mq = 0.f, x[W], y[W];
    const size_t at = ((size_t)(first + min(row, n - 1)) * s.H + h) * DK + part * W;
    load_row<BF16>(s.k, at, x);
    load_row<BF16>(s.q, at, y);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        mk = fmaxf(mk, fabsf(x[i]));
        mq = fmaxf(mq, fabsf(y[i]));
    }
    mk = fmaxf(mk, __shfl_xor(mk, 1));
    mk = fmaxf(mk, __shfl_xor(mk, 2));
    mq = fmaxf(mq, __shfl_xor(mq, 1));
    mq = fmaxf(mq, __shfl_xor(mq, 2));
    if (part == 0) {
        float ik, iq;
        m.sk[row] = scale_to(mk, 10, ik);
        m.sq[row] = scale_to(mq, 10, iq);
        sh.ik[row] = ik;
        sh.iq[row] = iq;
        sh.be[row] = row < n ? s.beta[(size_t)(first + row) * s.H + h] : 0.f;
    }
}

// A row of a 64x64 LDS matrix, thread (row, 16 columns), as scaled fp16 pairs
// in fragment order.
__device__ inline void store_tri(const float (*X)[LD], uint16_t (&to)[2][kTri][kFrag], float *undo) {
    const int i = threadIdx.x >> 2, qq = threadIdx.x & 3, rt = i >> 4;
    const int ks = qq >> 1;
    const bool kept = ks <= rt / 2;  // what lies further right is 0 and has no fragment
    float x[16], m = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        x[c] = kept ? X[i][16 * qq + c] : 0.f;
        m = fmaxf(m, fabsf(x[c]));
    }
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    float inv;
    const float s = scale_to(m, 10, inv);
    if (qq == 0) undo[i] = inv;
    if (!kept) return;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        half4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            _Float16 a, b;
            split(x[4 * g + e], s, a, b);
            hi[e] = a;
            lo[e] = b;
        }
        const int at = ((i & 15) + 16 * g) * 8 + (qq & 1) * 4;
        *reinterpret_cast<half4 *>(&to[0][tri(rt, ks)][at]) = hi;
        *reinterpret_cast<half4 *>(&to[1][tri(rt, ks)][at]) = lo;
    }
}

// From M = diag(beta) A (strictly lower; what lies above the diagonal is not
// read) and P in LDS to what the entry holds.  T is written over `Tx`.
__device__ inline void finish(const float (*M)[LD], const float (*Px)[LD], float (*Tx)[LD], float (*X)[20],
                              const float *be, ChunkPrep &out) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
    // inverse of the diagonal block `wave`, column j
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == j ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < i; ++m) s = __builtin_fmaf(-M[16 * wave + i][16 * wave + m], x[m], s);
        x[i] = s;
    }
    if (g == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) X[16 * wave + i][j] = x[i];
    }
    __syncthreads();
    floatx4 t[4];  // blocks of column `wave`
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
                const float4 a = *reinterpret_cast<const float4 *>(&M[16 * I + j][16 * m + 4 * g]);
                y = mfma_f32(a.x, t[m][0], y);
                y = mfma_f32(a.y, t[m][1], y);
                y = mfma_f32(a.z, t[m][2], y);
                y = mfma_f32(a.w, t[m][3], y);
            }
            const float4 a = *reinterpret_cast<const float4 *>(&X[16 * I + j][4 * g]);
            z = mfma_f32(-a.x, y[0], z);
            z = mfma_f32(-a.y, y[1], z);
            z = mfma_f32(-a.z, y[2], z);
            z = mfma_f32(-a.w, y[3], z);
            t[I] = z;
        }
    }
    const float b = be[16 * wave + j];
#pragma unroll
    for (int I = 0; I < 4; ++I)
#pragma unroll
        for (int r = 0; r < 4; ++r) Tx[16 * I + 4 * g + r][16 * wave + j] = t[I][r] * b;
    __syncthreads();
    store_tri(Tx, out.T, out.m.rt);
    store_tri(Px, out.P, out.m.rp);
}

// Eight channels of row `row` for a matrix instruction; 0 past the last token.
template <int DK>
__device__ inline bf16x8 frag_bf16(const void *p, const SeqArgs &s, int h, int first, int n, int row, int c) {
    union { uint4 w; bf16x8 v; } x;
    x.w = make_uint4(0, 0, 0, 0);
    if (row < n)
        x.w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) +
                                               ((size_t)(first + row) * s.H + h) * DK + c);
    return x.v;
}
template <int DK>
__device__ inline float4 frag_f32(const void *p, const SeqArgs &s, int h, int first, int n, int row, int c) {
    if (row >= n) return make_float4(0.f, 0.f, 0.f, 0.f);
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) +
                                             ((size_t)(first + row) * s.H + h) * DK + c);
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(256) k_prep_scalar(const ChunkArgs A) {
    __shared__ float M[kC][LD], Px[kC][LD], D[kC][LD], X[kC][20], F[4][kC], ga[kC];
    __shared__ PrepShared sh;
    const SeqArgs &s = A.s;
    const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int b, first;
    const int n = chunk_of_slot(s, blockIdx.x, b, first);
    if (n == 0) return;
    ChunkPrep &out = A.prep[(size_t)blockIdx.x * s.H + h];
    row_scales<DK, BF16>(s, h, first, n, out.m, sh);
    if (tid < kC) ga[tid] = tid < n ? s.a[(size_t)(first + tid) * s.H + h] : 1.f;
    __syncthreads();
    {  // D inside 16-row blocks; F: the factor from j's block to block I
        const int j = lane, I = wave;
        if (I >= j >> 4) {
            float run = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (16 * I + i > j) run *= ga[16 * I + i];
                D[16 * I + i][j] = run;
            }
        }
        __syncthreads();
        float f = 1.f;
        for (int m = j >> 4; m < I; ++m) f *= D[16 * m + 15][j];
        F[I][j] = f;
    }
    __syncthreads();
    if (tid < kC) {
        const float G = ga[0] * D[tid][0] * F[tid >> 4][0];
        out.m.rk[tid] = sh.ik[tid] * G;
        out.m.rq[tid] = sh.iq[tid] * G;
        out.m.rw[tid] = sh.ik[tid] * D[kC - 1][tid] * F[3][tid];
    }
    if (tid < 128) out.m.dec[tid] = ga[0] * D[kC - 1][0] * F[3][0];

    const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        if (ct > (wave | 1)) continue;
        floatx4 aa = {0.f, 0.f, 0.f, 0.f}, pp = aa;
        if (ct <= wave) {
            if constexpr (BF16) {
#pragma unroll
                for (int c = 0; c < DK; c += 32) {
                    const bf16x8 kr = frag_bf16<DK>(s.k, s, h, first, n, 16 * wave + r16, c + 8 * g);
                    const bf16x8 qr = frag_bf16<DK>(s.q, s, h, first, n, 16 * wave + r16, c + 8 * g);
                    const bf16x8 kc = frag_bf16<DK>(s.k, s, h, first, n, 16 * ct + r16, c + 8 * g);
                    aa = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kr, kc, aa, 0, 0, 0);
                    pp = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qr, kc, pp, 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int c = 0; c < DK; c += 16) {
                    const float4 kr = frag_f32<DK>(s.k, s, h, first, n, 16 * wave + r16, c + 4 * g);
                    const float4 qr = frag_f32<DK>(s.q, s, h, first, n, 16 * wave + r16, c + 4 * g);
                    const float4 kc = frag_f32<DK>(s.k, s, h, first, n, 16 * ct + r16, c + 4 * g);
                    aa = mfma_f32(kr.x, kc.x, aa);
                    aa = mfma_f32(kr.y, kc.y, aa);
                    aa = mfma_f32(kr.z, kc.z, aa);
                    aa = mfma_f32(kr.w, kc.w, aa);
                    pp = mfma_f32(qr.x, kc.x, pp);
                    pp = mfma_f32(qr.y, kc.y, pp);
                    pp = mfma_f32(qr.z, kc.z, pp);
                    pp = mfma_f32(qr.w, kc.w, pp);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * wave + 4 * g + r, j = 16 * ct + r16;
            const float d = i >= j ? D[i][j] * F[wave][j] : 0.f;
            M[i][j] = i > j ? sh.be[i] * (aa[r] * d) : 0.f;
            Px[i][j] = i >= j ? pp[r] * d : 0.f;
        }
    }
    __syncthreads();
    finish(M, Px, D, X, sh.be, out);
}

// Rows of an operand times the factors of a level, from LDS.
template <int L>
__device__ inline float4 row_times(const float (*x)[L], const float (*f)[L], int row, int c) {
    const float4 a = *reinterpret_cast<const float4 *>(&x[row][c]);
    const float4 b = *reinterpret_cast<const float4 *>(&f[row][c]);
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

template <int DK, int L>
__device__ inline floatx4 block_product(const float (*x)[L], const float (*k)[L], const float (*f)[L], int I, int J) {
    const int r16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < DK; c += 16) {
        const float4 a = row_times<L>(x, f, 16 * I + r16, c + 4 * g);
        const float4 b = row_times<L>(k, f, 16 * J + r16, c + 4 * g);
        acc = mfma_f32(a.x, b.x, acc);
        acc = mfma_f32(a.y, b.y, acc);
        acc = mfma_f32(a.z, b.z, acc);
        acc = mfma_f32(a.w, b.w, acc);
    }
    return acc;
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(256) k_prep_keyvec(const ChunkArgs A) {
    constexpr int L = DK + 4, G4 = 256 / DK;  // G4 groups of DK threads
    __shared__ float K[kC][L], Q[kC][L], Ga[kC][L], F[kC][L], dg[2][4][16][17];
    __shared__ PrepShared sh;
    const SeqArgs &s = A.s;
    const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int b, first;
    const int n = chunk_of_slot(s, blockIdx.x, b, first);
    if (n == 0) return;
    ChunkPrep &out = A.prep[(size_t)blockIdx.x * s.H + h];
    row_scales<DK, BF16>(s, h, first, n, out.m, sh);
    for (int i = tid; i < kC * (DK / 4); i += 256) {
        const int row = i / (DK / 4), c = i % (DK / 4) * 4;
        float k[4] = {}, q[4] = {}, a[4] = {1.f, 1.f, 1.f, 1.f};
        if (row < n) {
            const size_t at = ((size_t)(first + row) * s.H + h) * DK + c;
            load_row<BF16>(s.k, at, k);
            load_row<BF16>(s.q, at, q);
            load_f32(s.a + at, a);
        }
        *reinterpret_cast<float4 *>(&K[row][c]) = make_float4(k[0], k[1], k[2], k[3]);
        *reinterpret_cast<float4 *>(&Q[row][c]) = make_float4(q[0], q[1], q[2], q[3]);
        *reinterpret_cast<float4 *>(&Ga[row][c]) = make_float4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    if (tid < kC) {
        out.m.rk[tid] = sh.ik[tid];
        out.m.rq[tid] = sh.iq[tid];
        out.m.rw[tid] = sh.ik[tid];
    }
    {  // gate products before and after each four tokens
        ChunkGates &o = A.gates[(size_t)blockIdx.x * s.H + h];
        const int c = tid % DK;
        float run = 1.f;
        if (tid < DK) {
#pragma unroll 16
            for (int i = 0; i < kC; ++i) {
                if (i % 4 == 0) o.pre[i / 4][c] = run;
                run *= Ga[i][c];
            }
        } else if (tid < 2 * DK) {
#pragma unroll 16
            for (int i = kC - 1; i >= 0; --i) {
                if (i % 4 == 3) o.suf[i / 4][c] = run;
                run *= Ga[i][c];
            }
        }
    }
    // splits at 16 and 48: rows of blocks 0 and 2 carry the product up to the
    // block's end, rows of blocks 1 and 3 the product from the block's start
    const int c = tid % DK, grp = tid / DK;
    for (int blk = grp; blk < 4; blk += G4) {
        float run = 1.f;
        if (blk & 1) {
            for (int i = 16 * blk; i < 16 * blk + 16; ++i) {
                run *= Ga[i][c];
                F[i][c] = run;
            }
        } else {
            for (int i = 16 * blk + 15; i >= 16 * blk; --i) {
                F[i][c] = run;
                run *= Ga[i][c];
            }
        }
    }
    __syncthreads();
    const int pair = wave & 1;  // blocks (1, 0) and (3, 2); A by waves 0 and 1, P by 2 and 3
    const floatx4 near = block_product<DK, L>(wave < 2 ? K : Q, K, F, 2 * pair + 1, 2 * pair);
    __syncthreads();
    // split at 32
    if (grp == 0) {
        float run = 1.f;
        for (int i = 31; i >= 0; --i) {
            F[i][c] = run;
            run *= Ga[i][c];
        }
    } else if (grp == 1) {
        float run = 1.f;
        for (int i = 32; i < kC; ++i) {
            run *= Ga[i][c];
            F[i][c] = run;
        }
    }
    __syncthreads();
    const int fi = 2 + (wave & 1), fj = wave >> 1;
    const floatx4 farA = block_product<DK, L>(K, K, F, fi, fj);
    const floatx4 farP = block_product<DK, L>(Q, K, F, fi, fj);
    if (tid < DK) out.m.dec[tid] = F[0][tid] * Ga[0][tid] * F[kC - 1][tid];
    // diagonal block `wave`: lane (j, g) follows k_j over the channels of group g
    const int j = lane & 15, g = lane >> 4;
    {
        constexpr int W = DK / 4;
        float w[W];
        const int row0 = 16 * wave;
#pragma unroll
        for (int x = 0; x < W; x += 4) {
            const float4 k = *reinterpret_cast<const float4 *>(&K[row0 + j][W * g + x]);
            w[x] = k.x;
            w[x + 1] = k.y;
            w[x + 2] = k.z;
            w[x + 3] = k.w;
        }
        for (int i = 0; i < 16; ++i) {
            float da = 0.f, dp = 0.f;
            const bool on = i > j;
#pragma unroll
            for (int x = 0; x < W; x += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&Ga[row0 + i][W * g + x]);
                const float4 k = *reinterpret_cast<const float4 *>(&K[row0 + i][W * g + x]);
                const float4 q = *reinterpret_cast<const float4 *>(&Q[row0 + i][W * g + x]);
                w[x] *= on ? a.x : 1.f;
                w[x + 1] *= on ? a.y : 1.f;
                w[x + 2] *= on ? a.z : 1.f;
                w[x + 3] *= on ? a.w : 1.f;
                da = __builtin_fmaf(k.x, w[x], da);
                da = __builtin_fmaf(k.y, w[x + 1], da);
                da = __builtin_fmaf(k.z, w[x + 2], da);
                da = __builtin_fmaf(k.w, w[x + 3], da);
                dp = __builtin_fmaf(q.x, w[x], dp);
                dp = __builtin_fmaf(q.y, w[x + 1], dp);
                dp = __builtin_fmaf(q.z, w[x + 2], dp);
                dp = __builtin_fmaf(q.w, w[x + 3], dp);
            }
            da += __shfl_xor(da, 16);
            da += __shfl_xor(da, 32);
            dp += __shfl_xor(dp, 16);
            dp += __shfl_xor(dp, 32);
            if (g == 0) {
                dg[0][wave][i][j] = on ? da : 0.f;
                dg[1][wave][i][j] = i >= j ? dp : 0.f;
            }
        }
    }
    __syncthreads();
    // K, Q, Ga and F are done with: M, P, T and X take their places
    static_assert(sizeof(K) >= sizeof(float) * kC * LD, "a 64x64 matrix fits");
    float(*M)[LD] = reinterpret_cast<float(*)[LD]>(&K[0][0]);
    float(*Px)[LD] = reinterpret_cast<float(*)[LD]>(&Q[0][0]);
    float(*Tx)[LD] = reinterpret_cast<float(*)[LD]>(&Ga[0][0]);
    float(*X)[20] = reinterpret_cast<float(*)[20]>(&F[0][0]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i1 = 16 * (2 * pair + 1) + 4 * g + r, j1 = 16 * (2 * pair) + j;
        if (wave < 2) M[i1][j1] = sh.be[i1] * near[r];
        else Px[i1][j1] = near[r];
        const int i2 = 16 * fi + 4 * g + r, j2 = 16 * fj + j;
        M[i2][j2] = sh.be[i2] * farA[r];
        Px[i2][j2] = farP[r];
        const int i3 = 16 * wave + 4 * g + r;
        M[i3][16 * wave + j] = sh.be[i3] * dg[0][wave][4 * g + r][j];
        Px[i3][16 * wave + j] = dg[1][wave][4 * g + r][j];
        if (!(wave & 1)) {  // the block right of an even diagonal block
            M[i3][16 * wave + 16 + j] = 0.f;
            Px[i3][16 * wave + 16 + j] = 0.f;
        }
    }
    __syncthreads();
    finish(M, Px, Tx, X, sh.be, out);
}

}  // namespace

hipError_t launch_chunk_prep(const ChunkArgs &a, int dk, bool keyvec, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)a.slots, (unsigned)a.s.H);
    if (keyvec) {
        if (dk == 64 && bf16) k_prep_keyvec<64, true><<<grid, 256, 0, s>>>(a);
        else if (dk == 64) k_prep_keyvec<64, false><<<grid, 256, 0, s>>>(a);
        else if (bf16) k_prep_keyvec<128, true><<<grid, 256, 0, s>>>(a);
        else k_prep_keyvec<128, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (dk == 64 && bf16) k_prep_scalar<64, true><<<grid, 256, 0, s>>>(a);
        else if (dk == 64) k_prep_scalar<64, false><<<grid, 256, 0, s>>>(a);
        else if (bf16) k_prep_scalar<128, true><<<grid, 256, 0, s>>>(a);
        else k_prep_scalar<128, false><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace stq
