// Shared pieces of the chunked gated delta rule (forward and backward): the
// chunk table, the scaled fp16 pairs that carry fp32 values through the matrix
// instructions, and fragment layouts.  Not part of the ABI.
//
// A sequence is cut into chunks of 64 tokens.  With G_i the product of the
// gates of a chunk's tokens up to i (per key channel; one value per token for
// scalar gates), S0 the state at its start, row-major d_k x d_v:
//   A_ij = sum_c k_ic k_jc prod_{j<s<=i} a_sc  (i > j)
//   P_ij = sum_c q_ic k_jc prod_{j<s<=i} a_sc  (i >= j)
//   T = (I + diag(beta) A)^-1 diag(beta)
//   u = T (V - (K G) S0);   O = (Q G) S0 + P u;   S1 = diag(G_64) S0 + (K G_64/G)^T u
// Every gate product, G_64/G_i among them, is formed by multiplying gates, never by a
// quotient, so gates that underflow, or are 0, are right.
//
// Numbers.  States, sums and u are fp32.  A matrix instruction takes an fp32
// operand x as two fp16 values, x 2^e = hi + lo (22 bits and more), with e
// chosen per row of a left or per column of a right operand so that its
// largest value is near 2^10 (left) or 2^14 (right); the product hi hi + hi lo + lo hi
// leaves out lo lo, at most 2^-22 of the operands' largest values, so results
// keep fp32's accuracy relative to a row's and column's norm.  bf16 inputs are
// exact in the hi part alone (a value under 2^-24 of its row's largest loses bits).
#pragma once

#include "stq_seq.h"

namespace stq {

constexpr int kC = 64;               // tokens of a chunk
constexpr int kFrag = 512;           // halves of one 16x32 fragment (64 lanes x 8)
constexpr int kTri = 6;              // 16x32 fragments of a lower triangular 64x64 matrix

// What k_chunk_prep leaves for one (chunk, head): T and P as fragments (hi,
// then lo), and per-token factors.
struct ChunkMeta {
    float sk[kC], sq[kC];            // 2^e of the rows of K and Q
    float rk[kC], rq[kC];            // factors that undo it (and G_i for scalar gates)
    float rt[kC], rp[kC];            // factors that undo the row scales of T and P
    float rw[kC];                    // factor of u_i in the state's update: 2^-e (and G_64/G_i)
    float dec[128];                  // G_64 per key channel
    float rn[kC], rpt[kC];           // backward: factors that undo the row scales of N^T and P^T
    float be[kC];                    // backward: beta, 0 past the last token
};
struct ChunkPrep {
    uint16_t T[2][kTri][kFrag];      // backward: N' = (I + A diag(beta))^-1
    uint16_t P[2][kTri][kFrag];
    ChunkMeta m;
};
// The backward pass's other matrices: N^T, N = (I + diag(beta) A)^-1, and P^T, upper
// triangular, fragments in the order rows 0 (k steps 0, 1), 1 (0, 1), 2 (1), 3 (1).
struct ChunkBack {
    uint16_t N[2][kTri][kFrag];
    uint16_t P[2][kTri][kFrag];
};
static_assert(sizeof(ChunkPrep) % 256 == 0, "entries of the workspace stay aligned");

// Key-vector gates: per channel, the products of the gates before and after each
// four tokens of a chunk.
struct ChunkGates {
    float pre[kC / 4][128], suf[kC / 4][128];
};

struct ChunkArgs {
    SeqArgs s;
    const float *initial;            // [B,H,d_k,d_v] or nullptr
    float *last;                     // [B,H,d_k,d_v] or nullptr
    void *o;                         // [N,H,d_v] io dtype
    ChunkPrep *prep;                 // [chunk slots][H]
    ChunkGates *gates;               // the same, key-vector gates only
    int32_t slots;                   // chunk slots: N / 64 + B
    int32_t *order;                  // [B] sequences, longest first, or nullptr: as they come
    // Sequences cut into `segs` segments (chunk_segments; 1: they are not), per (sequence, head)
    int32_t segs;
    float *steps;                    // [segs - 1][d_k][d_v + d_k]: a segment's end from no state | its matrix
    float *starts;                   // [segs][d_k][d_v]: the state before each segment
    // The backward pass (back not nullptr): per (chunk, head)
    ChunkBack *back;
    float *S, *dS;                   // first state; gradient of the last one [d_k,d_v]
    float *w, *y;                    // delta errors (u = beta w); gradients of u through N^T [64,d_v]
                                     // (these four as result tiles: [column / 16][row / 16][lane][4])
    const void *dout;                // [N,H,d_v] io dtype
    const float *dlast;              // [B,H,d_k,d_v] or nullptr
    void *dq, *dk, *dv;              // io dtype
    float *da, *dbeta, *dinitial;    // (dinitial may be nullptr)
};

constexpr int kOrdered = 1024;       // sequences that are put in order of length

// Chunk c of sequence b (first token t0) has slot t0 / 64 + b + c: slots of
// different chunks differ, and none reaches N / 64 + B.
inline int chunk_slots(int N, int B) { return N / kC + B; }

// Few long sequences leave most of the 256 CUs without work, for a pass goes through a
// sequence's chunks in turn.  Then each is cut into segments, and the state passes through
// all of them at once, from no state, and so do the unit vectors of the state's rows, which
// gives the segment's matrix (columns never meet, so those are d_k columns more); the states
// before the segments follow, one small product each, and then the outputs of all segments at once.
// That is twice the work and d_k columns more, so it is done where all of it runs side by
// side, one workgroup a CU, in segments of at least kSegment chunks: from 3 segments on
// (2 of them take as long as none: each half twice).
constexpr int kSegment = 16;
inline int chunk_segments(int H, int dk, int dv, int B, int N) {
    const int64_t heads = (int64_t)B * H;
    for (int s = B > 0 ? (N / kC / B / kSegment < 16 ? N / kC / B / kSegment : 16) : 1; s > 2; --s)
        if (heads * ((s - 1) * (dv / 64) + (s - 2) * (dk / 64)) <= 256) return s;
    return 1;
}
// No call with at most N tokens has more (sequence, head, segment) triples that are not a
// sequence's last: heads * (s - 1) stays under both.
inline int64_t chunk_steps(int H, int dv, int N) {
    const int64_t a = 256 / (dv / 64), b = (int64_t)H * (N / kC / kSegment);
    return a < b ? a : b;
}

hipError_t launch_chunk_prep(const ChunkArgs &a, int dk, bool keyvec, bool bf16, hipStream_t s);
// (through segments where a.segs > 1)
hipError_t launch_chunk_forward(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s);

hipError_t launch_chunk_reverse(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s);
hipError_t launch_chunk_grad(const ChunkArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s);

#if defined(__HIPCC__)

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// A wave's number in its workgroup, in a scalar register: branches on it are the whole
// wave's (matrix instructions write their results whatever lanes are on).
__device__ inline int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Workgroup `id` of a line of groups of `m` (the heads of a sequence or chunk):
// its group and its place in it.  Workgroups go to the eight XCDs in turn.  A head's rows
// lie H d elements apart, often a multiple of the L2's channel interleave, so a head stays in
// one or two channels: with heads dealt out in turn an XCD would only see heads, and
// channels, a multiple of 8 apart.  Here it takes m / 8 neighbouring heads of every
// group, other ones in the next group.  (Chunk preparation: 240 -> 234 us with scalar, 825 -> 788 us
// with key-vector gates when it came; the passes neither gain nor lose.)
__device__ inline void xcd_place(uint32_t id, uint32_t m, uint32_t &group, uint32_t &at) {
    if (m & 7) {
        group = id / m;
        at = id % m;
        return;
    }
    const uint32_t each = m >> 3, xcd = id & 7, i = id >> 3;
    group = i / each;
    at = ((xcd + group) & 7) * each + i % each;
}

// The chunk of slot x: its sequence, first token and number of tokens; 0 tokens
// where the slot holds none.  Called by whole waves: the sequence is searched for 64
// candidates at a time.
__device__ inline int chunk_of_slot(const SeqArgs &s, int x, int &b, int &first) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = s.B;
    while (n > 1) {
        const int step = (n + 63) >> 6, at = lane * step;
        bool ok = false;
        if (at < n) ok = min(max(s.cu[lo + at], 0), s.N) / kC + lo + at <= x;
        const int i = max(__popcll(__ballot(ok)), 1) - 1;  // the last candidate at or before x
        lo += i * step;
        n = min(step, n - i * step);
    }
    b = __builtin_amdgcn_readfirstlane(lo);
    int t0, t1;
    seq_range(s, b, t0, t1);
    const int c = x - (t0 / kC + b);
    first = t0 + c * kC;
    return c < 0 ? 0 : min(max(t1 - first, 0), kC);
}

// 2^(top - floor(log2 m)) and its inverse, for m >= 0 (tiny m: as for 2^(top - 112)).
__device__ inline float scale_to(float m, int top, float &inv) {
    const int e = max((int)(__float_as_uint(m) >> 23) & 255, top + 1);
    inv = __uint_as_float((uint32_t)(e - top) << 23);
    return __uint_as_float((uint32_t)(254 + top - e) << 23);
}

__device__ inline floatx4 mfma16(half8 a, half8 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ inline floatx4 mfma_f32(float a, float b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// x s as hi + lo
__device__ inline void split(float x, float s, _Float16 &hi, _Float16 &lo) {
    hi = (_Float16)(x * s);
    lo = (_Float16)__builtin_fmaf(x, s, -(float)hi);
}
// x, scaled already, as hi + lo.  (The 1 is hidden from the compiler: x - hi would be three
// instructions, the mixed product and sum with its rounding is one.  So is where x comes from: a product
// is else rounded to hi at once in one place, and by way of fp32 in the other, and the two differ now and
// then by a step of fp16.)
__device__ inline void split(float x, _Float16 &hi, _Float16 &lo) {
    float one = 1.f;
    asm("" : "+s"(one));
    asm("" : "+v"(x));
    hi = (_Float16)x;
    lo = (_Float16)__builtin_fmaf(x, one, -(float)hi);
}

// Lanes l and l ^ 16, or l ^ 32, exchanged by one vector instruction: both of a pair get
// both values.  (Values of at least 0 are in the order of their bits; as numbers they would be
// quieted first, an instruction each, and not fold a value across lanes in.)
__device__ inline float max_groups(float x) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    const uint32_t m = max((uint32_t)r[0], (uint32_t)r[1]);
    r = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return __uint_as_float(max((uint32_t)r[0], (uint32_t)r[1]));
}

// The value of another lane of the row of 16 (`old` where there is none).
template <int ctrl>
__device__ inline float dpp(float x, float old = 0.f) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), ctrl, 0xf, 0xf, false));
}
// The same, 0 where there is none: it folds into the instruction that takes it.
template <int ctrl>
__device__ inline float dpp0(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), ctrl, 0xf, 0xf, true));
}
constexpr int kShl = 0x100, kShr = 0x110, kRor = 0x120, kBcast = 0x150;  // lane i + n, i - n, i - n mod 16, n
constexpr int quad(int a, int b, int c, int d) { return a | b << 2 | c << 4 | d << 6; }

// A choice whose both values are formed by every lane: a value read across lanes
// inside a branch would find the other lanes switched off.
__device__ inline float pick(bool c, float x, float y) { return c ? x : y; }

// max over the lanes of a row of 16, of values of at least 0
template <int ctrl>
__device__ inline uint32_t max_dpp(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, ctrl, 0xf, 0xf, true));
}
__device__ inline float max_row(float x) {
    return __uint_as_float(max_dpp<kRor + 1>(max_dpp<kRor + 2>(max_dpp<kRor + 4>(max_dpp<kRor + 8>(__float_as_uint(x))))));
}
// sum over the lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ inline float sum_groups(float x) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline floatx4 four(const float *p) { return *reinterpret_cast<const floatx4 *>(p); }

// Eight consecutive channels as they are in memory.
template <bool BF16> struct Row8;
template <> struct Row8<true> {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 w;
    __device__ void load(const void *p, size_t at) {
        w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
    }
    __device__ float get(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};
template <> struct Row8<false> {
    floatx4 x, y;
    __device__ void load(const void *p, size_t at) {
        x = four(static_cast<const float *>(p) + at);
        y = four(static_cast<const float *>(p) + at + 4);
    }
    __device__ float get(int i) const { return i < 4 ? x[i] : y[i - 4]; }
};

// Eight of them (hi parts are rounded two at a time).
__device__ inline void split8(const float (&x)[8], half8 &hi, half8 &lo) {
    typedef _Float16 half2 __attribute__((ext_vector_type(2)));
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    float one = 1.f;
    asm("" : "+s"(one));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float a = x[e], b = x[e + 1];
        asm("" : "+v"(a), "+v"(b));
        const half2 h = __builtin_convertvector((floatx2{a, b}), half2);
        hi[e] = h[0];
        hi[e + 1] = h[1];
        lo[e] = (_Float16)__builtin_fmaf(a, one, -(float)h[0]);
        lo[e + 1] = (_Float16)__builtin_fmaf(b, one, -(float)h[1]);
    }
}
// x s of eight channels as fp16 pairs
__device__ inline void split8(const float (&x)[8], float s, half8 &hi, half8 &lo) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        _Float16 a, b;
        split(x[e], s, a, b);
        hi[e] = a;
        lo[e] = b;
    }
}
__device__ inline floatx4 mfma_pairs(half8 ah, half8 al, half8 bh, half8 bl, floatx4 c) {
    c = mfma16(ah, bh, c);
    c = mfma16(ah, bl, c);
    return mfma16(al, bh, c);
}

// x[j] of lane i of a quad becomes x[i] of lane j.
template <int ctrl>
__device__ inline float quad_swap(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, 0xf, 0xf, true));
}
__device__ inline void quad_transpose(float (&x)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
    for (int p = 0; p < 4; p += 2) {
        const float r = quad_swap<0xB1>(odd ? x[p] : x[p + 1]);
        x[p] = odd ? r : x[p];
        x[p + 1] = odd ? x[p + 1] : r;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const float r = quad_swap<0x4E>(high ? x[p] : x[p + 2]);
        x[p] = high ? r : x[p];
        x[p + 2] = high ? x[p + 2] : r;
    }
}

// A workgroup barrier for values in LDS: it waits for this wave's LDS accesses, not for
// its loads from memory, which stay in flight.
__device__ inline void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Index of fragment (row tile, k step) of a lower triangular matrix.
__device__ constexpr int tri(int rt, int ks) { return rt < 2 ? rt : 2 + 2 * (rt - 2) + ks; }

#endif  // __HIPCC__

}  // namespace stq
