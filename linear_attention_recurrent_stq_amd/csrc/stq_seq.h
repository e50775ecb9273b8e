// Shared definitions of the sequence operators (recurrent step, chunked
// forward and backward, draft verification): kernel arguments, launchers, and
// the device helpers they have in common.  Not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

namespace stq {

// A packed batch of sequences and the rule's inputs.
struct SeqArgs {
    const int32_t *cu;           // [B+1]
    const void *q, *k, *v;       // [N,H,d] io dtype
    const float *a;              // [N,H] or [N,H,d_k]
    const float *beta;           // [N,H]
    int32_t B, N, H;
};

struct RecurrentArgs {
    SeqArgs s;
    float *state;                // [slots,H,d_k,d_v]
    const int32_t *slot_ids;     // [B] or nullptr
    const int32_t *commit;       // [B] or nullptr
    float *o;                    // [N,H,d_v] fp32
    int32_t slots;
};

struct VerifyArgs {
    const int32_t *tokens, *len; // [B,T], [B] or nullptr
    const void *p, *q;           // [B,T+1,V], [B,T,V]
    const float *uniform;        // [B,T+1]
    int32_t *accepted, *next;    // [B]
    double *part;                // [B][nseg][2]
    int32_t B, T, V, seg, nseg;
};

// Segments of a vocabulary of V tokens: at most kVerifySegs, of a length that
// depends on V alone.
constexpr int kVerifySegs = 64;
inline int verify_seg(int V) {
    const int s = (V + kVerifySegs - 1) / kVerifySegs;
    return s < 2048 ? 2048 : (s + 255) / 256 * 256;
}
inline int verify_nseg(int V) { return (V + verify_seg(V) - 1) / verify_seg(V); }

hipError_t launch_recurrent(const RecurrentArgs &a, int dk, int dv, bool keyvec, bool bf16, hipStream_t s);
hipError_t launch_verify(const VerifyArgs &a, bool bf16, hipStream_t s);

#if defined(__HIPCC__)

// Tokens of sequence b, clamped so that every access stays in the N tokens.
__device__ inline void seq_range(const SeqArgs &s, int b, int &t0, int &t1) {
    t0 = min(max(s.cu[b], 0), s.N);
    t1 = min(max(s.cu[b + 1], t0), s.N);
}

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// n (a multiple of 4) consecutive elements from p, which is 8-byte aligned for
// bf16 and 16-byte aligned for fp32.
template <bool BF16, int n>
__device__ inline void load_row(const void *p, size_t at, float (&x)[n]) {
    if constexpr (BF16) {
        const uint2 *s = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < n / 4; ++i) {
            const uint2 w = s[i];
            x[4 * i] = bf16_lo(w.x);
            x[4 * i + 1] = bf16_hi(w.x);
            x[4 * i + 2] = bf16_lo(w.y);
            x[4 * i + 3] = bf16_hi(w.y);
        }
    } else {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int i = 0; i < n / 4; ++i) {
            const float4 w = s[i];
            x[4 * i] = w.x;
            x[4 * i + 1] = w.y;
            x[4 * i + 2] = w.z;
            x[4 * i + 3] = w.w;
        }
    }
}

template <int n>
__device__ inline void load_f32(const float *p, float (&x)[n]) {
    load_row<false, n>(p, 0, x);
}

#endif  // __HIPCC__

}  // namespace stq
