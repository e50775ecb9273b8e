// Acceptance of drafted tokens and the choice of the next one (stq_verify_draft).
//
// Token t stands while r_t q_t(x_t) < p_t(x_t): the product of two fp32 values
// is exact in 64 bits, so the comparison is exact.  The next token is the
// smallest index whose running weight passes r_T times the whole weight, over
// w = max(p - q, 0) of the first token that does not stand (p alone where all
// stand).  The weights of one row per request are what has to be read: 2 V
// values; the bound is their bytes, or for few requests the latency of two
// launches.
//
// k_verify_sum: a workgroup per (segment of the vocabulary, request) finds the
// accepted count itself (a handful of gathers; cheaper than a launch of its
// own) and sums its segment's w and p in 64 bits.  k_verify_pick: a workgroup
// per request adds up the segment sums, finds the segment that the draw falls
// into, and scans that segment alone, which is still in the cache.  Measured, MI355X: 96 requests over
// 129281 fp32 probabilities 13.3 and 7.0 us (99 MB), one over 32000 3.6 and 4.8 us.
#include "stq_seq.h"

namespace stq {
namespace {

constexpr int kT = 256;  // threads of both kernels

template <bool BF16>
__device__ inline float prob(const void *p, size_t at) {
    if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at] << 16);
    else return static_cast<const float *>(p)[at];
}

// A weight: what is not a positive number (NaN among it) counts as 0.
__device__ inline double weight(float p) { return p > 0.f ? (double)p : 0.0; }
__device__ inline double residual(float p, float q) { return p > q ? (double)p - (double)q : 0.0; }

__device__ inline double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// Drafted tokens of request b.
__device__ inline int draft_len(const VerifyArgs &A, int b) {
    return A.len ? min(max(A.len[b], 0), A.T) : A.T;
}

// Leading drafted tokens of request b that stand (called by whole waves).
template <bool BF16>
__device__ int accepted(const VerifyArgs &A, int b, int n) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < n; base += 64) {
        const int t = base + lane;
        bool stands = false;
        if (t < n) {
            const int x = A.tokens[(size_t)b * A.T + t];
            if (x >= 0 && x < A.V) {
                const double p = prob<BF16>(A.p, ((size_t)b * (A.T + 1) + t) * A.V + x);
                const double q = prob<BF16>(A.q, ((size_t)b * A.T + t) * A.V + x);
                stands = (double)A.uniform[(size_t)b * (A.T + 1) + t] * q < p;
            }
        }
        const uint64_t m = __ballot(t < n && !stands);
        if (m) return base + __builtin_ctzll(m);
    }
    return n;
}

template <bool BF16>
__global__ void __launch_bounds__(kT) k_verify_sum(const VerifyArgs A) {
    const int b = blockIdx.y, seg = blockIdx.x, tid = threadIdx.x;
    const int n = draft_len(A, b), acc = accepted<BF16>(A, b, n);
    const int lo = seg * A.seg, hi = min(lo + A.seg, A.V);
    const size_t pr = ((size_t)b * (A.T + 1) + acc) * A.V, qr = ((size_t)b * A.T + acc) * A.V;
    double w = 0.0, f = 0.0;
    if (acc < n) {
#pragma unroll 8
        for (int i = lo + tid; i < hi; i += kT) {
            const float p = prob<BF16>(A.p, pr + i), q = prob<BF16>(A.q, qr + i);
            f += weight(p);
            w += residual(p, q);
        }
    } else {
#pragma unroll 8
        for (int i = lo + tid; i < hi; i += kT) f += weight(prob<BF16>(A.p, pr + i));
    }
    __shared__ double part[2][kT / 64];
    w = wave_sum(w);
    f = wave_sum(f);
    if ((tid & 63) == 0) {
        part[0][tid >> 6] = w;
        part[1][tid >> 6] = f;
    }
    __syncthreads();
    if (tid < 2)
        A.part[((size_t)b * A.nseg + seg) * 2 + tid] = (part[tid][0] + part[tid][1]) + (part[tid][2] + part[tid][3]);
    if (seg == 0 && tid == 0) A.accepted[b] = acc;
}

template <bool BF16>
__global__ void __launch_bounds__(kT) k_verify_pick(const VerifyArgs A) {
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = draft_len(A, b), acc = A.accepted[b];
    __shared__ double scan[kT / 64];
    __shared__ int found[kT / 64], last[kT / 64];
    // segment sums, one a lane (at most 64), the same in every wave
    double w = 0.0, f = 0.0;
    if (lane < A.nseg) {
        w = A.part[((size_t)b * A.nseg + lane) * 2];
        f = A.part[((size_t)b * A.nseg + lane) * 2 + 1];
    }
    const bool rest = acc < n && __ballot(w > 0.0) != 0;
    const double s = rest ? w : f;
    double c = s;  // inclusive running sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double x = __shfl_up(c, d);
        if (lane >= d) c += x;
    }
    const uint64_t some = __ballot(s > 0.0);
    if (!some) {
        if (tid == 0) A.next[b] = -1;
        return;
    }
    const double draw = fmin(fmax((double)A.uniform[(size_t)b * (A.T + 1) + A.T], 0.0), 1.0);
    const double aim = draw * __shfl(c, A.nseg - 1);
    const uint64_t past = __ballot(lane < A.nseg && c > aim);
    // (a draw of 1, or one that is no number: the last segment with weight)
    const int seg = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
    const double before = seg ? __shfl(c, seg - 1) : 0.0;

    const int lo = seg * A.seg, hi = min(lo + A.seg, A.V);
    const int each = (hi - lo + kT - 1) / kT, i0 = min(lo + tid * each, hi), i1 = min(i0 + each, hi);
    const size_t pr = ((size_t)b * (A.T + 1) + acc) * A.V, qr = ((size_t)b * A.T + acc) * A.V;
    auto at = [&](int i) {
        const float p = prob<BF16>(A.p, pr + i);
        return rest ? residual(p, prob<BF16>(A.q, qr + i)) : weight(p);
    };
    double mine = 0.0;
    for (int i = i0; i < i1; ++i) mine += at(i);
    double run = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double x = __shfl_up(run, d);
        if (lane >= d) run += x;
    }
    if (lane == 63) scan[wave] = run;
    __syncthreads();
    double base = before;
    for (int i = 0; i < wave; ++i) base += scan[i];
    double cum = base + (run - mine);
    int hit = INT32_MAX, end = -1;
    for (int i = i0; i < i1; ++i) {
        const double x = at(i);
        cum += x;
        if (x > 0.0) {
            end = i;
            if (cum > aim && hit == INT32_MAX) hit = i;
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        hit = min(hit, __shfl_xor(hit, d));
        end = max(end, __shfl_xor(end, d));
    }
    if (lane == 0) {
        found[wave] = hit;
        last[wave] = end;
    }
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kT / 64; ++i) {
            hit = min(hit, found[i]);
            end = max(end, last[i]);
        }
        // the segment's own sum may fall short of the first kernel's by a rounding
        A.next[b] = hit != INT32_MAX ? hit : end;
    }
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)a.nseg, (unsigned)a.B);
    if (bf16) {
        k_verify_sum<true><<<grid, kT, 0, s>>>(a);
        k_verify_pick<true><<<(unsigned)a.B, kT, 0, s>>>(a);
    } else {
        k_verify_sum<false><<<grid, kT, 0, s>>>(a);
        k_verify_pick<false><<<(unsigned)a.B, kT, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace stq
