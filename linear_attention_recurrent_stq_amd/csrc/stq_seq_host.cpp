// Host side of the sequence operators (include/stq.h, second part): argument
// checks, workspace carving and launches.  Nothing here synchronizes the device.
#include <cstdio>
#include <string>
#include <vector>

#include "stq.h"

#include "stq_chunk.h"

namespace stq {
void set_error(const std::string &msg);  // stq_host.cpp
}

namespace {

stq_status fail(stq_status s, const std::string &msg) {
    stq::set_error(msg);
    return s;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

stq_status launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(STQ_ERR_DEVICE, std::string(what) + ": " + hipGetErrorString(e));
    return STQ_OK;
}

stq_status check_rule(const stq_rule *r) {
    if (!r) return fail(STQ_ERR_INVALID, "rule is NULL");
    if (r->H < 1 || r->H > 4096) return fail(STQ_ERR_INVALID, "H must be in [1, 4096]");
    if ((r->d_k != 64 && r->d_k != 128) || (r->d_v != 64 && r->d_v != 128))
        return fail(STQ_ERR_UNSUPPORTED, "d_k and d_v must each be 64 or 128");
    if (r->gate != STQ_GATE_SCALAR && r->gate != STQ_GATE_KEYVEC) return fail(STQ_ERR_INVALID, "bad gate");
    if (r->io_dtype != STQ_BF16 && r->io_dtype != STQ_F32)
        return fail(STQ_ERR_INVALID, "io_dtype must be STQ_BF16 or STQ_F32");
    return STQ_OK;
}

// A launch's threads must stay under 2^32: a sequence and head take up to four workgroups of 768 threads,
// a chunk and head up to 512 (in stq_chunk_workspace).
stq_status check_sizes(const stq_rule *r, int32_t B, int32_t N) {
    if (B < 0 || N < 0) return fail(STQ_ERR_INVALID, "B and N must be >= 0");
    if ((int64_t)B * r->H > 1 << 20) return fail(STQ_ERR_UNSUPPORTED, "B * H exceeds 2^20");
    return STQ_OK;
}

// Every pointer given and 16-byte aligned.
stq_status check_ptrs(std::initializer_list<const void *> ps) {
    for (const void *p : ps) {
        if (!p) return fail(STQ_ERR_INVALID, "an input or output pointer is NULL");
        if (!aligned(p, 16)) return fail(STQ_ERR_ALIGN, "device pointers must be 16-byte aligned");
    }
    return STQ_OK;
}

// Small int32 tables: 4-byte aligned; `need`: not NULL.
stq_status check_ints(const void *p, bool need, const char *what) {
    if (!p) return need ? fail(STQ_ERR_INVALID, std::string(what) + " is NULL") : STQ_OK;
    if (!aligned(p, 4)) return fail(STQ_ERR_ALIGN, std::string(what) + " must be 4-byte aligned");
    return STQ_OK;
}

stq::SeqArgs seq_args(const stq_rule *r, int32_t B, int32_t N, const int32_t *cu, const void *q,
                      const void *k, const void *v, const float *a, const float *beta) {
    stq::SeqArgs s{};
    s.cu = cu;
    s.q = q;
    s.k = k;
    s.v = v;
    s.a = a;
    s.beta = beta;
    s.B = B;
    s.N = N;
    s.H = r->H;
    return s;
}

// The parts of a chunk workspace at `base`, into *a (both may be NULL); its size.
size_t carve(const stq_rule *r, int32_t B, int32_t N, bool backward, void *base, stq::ChunkArgs *a) {
    const size_t entries = (size_t)stq::chunk_slots(N, B) * r->H;
    size_t at = sizeof(int32_t) * stq::kOrdered;
    auto take = [&](size_t bytes) -> void * {
        void *p = base ? static_cast<char *>(base) + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    stq::ChunkArgs none{};
    if (!a) a = &none;
    a->slots = stq::chunk_slots(N, B);
    a->order = B > 1 && B <= stq::kOrdered ? static_cast<int32_t *>(base) : nullptr;
    a->prep = static_cast<stq::ChunkPrep *>(take(sizeof(stq::ChunkPrep) * entries));
    if (r->gate == STQ_GATE_KEYVEC) a->gates = static_cast<stq::ChunkGates *>(take(sizeof(stq::ChunkGates) * entries));
    const int64_t steps = stq::chunk_steps(r->H, r->d_v, N);
    if (!backward && steps > 0) {
        a->steps = static_cast<float *>(take(sizeof(float) * (size_t)steps * r->d_k * (r->d_v + r->d_k)));
        a->starts = static_cast<float *>(take(sizeof(float) * (size_t)steps * 2 * r->d_k * r->d_v));
    }
    a->segs = backward ? 1 : stq::chunk_segments(r->H, r->d_k, r->d_v, B, N);
    if (backward) {
        const size_t state = sizeof(float) * r->d_k * r->d_v * entries, rows = sizeof(float) * stq::kC * r->d_v * entries;
        a->back = static_cast<stq::ChunkBack *>(take(sizeof(stq::ChunkBack) * entries));
        a->S = static_cast<float *>(take(state));
        a->dS = static_cast<float *>(take(state));
        a->w = static_cast<float *>(take(rows));
        a->y = static_cast<float *>(take(rows));
    }
    return at;
}

}  // namespace

extern "C" {

stq_status stq_recurrent_step(const stq_rule *rule, int32_t B, int32_t N, const int32_t *d_cu_seqlens,
                              const void *d_q, const void *d_k, const void *d_v, const float *d_a,
                              const float *d_beta, float *d_state, int32_t slots,
                              const int32_t *d_slot_ids, const int32_t *d_commit, float *d_o,
                              void *stream) {
    stq::set_error("");
    if (stq_status s = check_rule(rule)) return s;
    if (stq_status s = check_sizes(rule, B, N)) return s;
    if (slots < 0 || B > slots) return fail(STQ_ERR_INVALID, "B exceeds the number of slots");
    if (B == 0 || N == 0) return STQ_OK;
    if (stq_status s = check_ints(d_cu_seqlens, true, "cu_seqlens")) return s;
    if (stq_status s = check_ints(d_slot_ids, false, "slot ids")) return s;
    if (stq_status s = check_ints(d_commit, false, "commit")) return s;
    if (stq_status s = check_ptrs({d_q, d_k, d_v, d_a, d_beta, d_state, d_o})) return s;
#if STQ_DEBUG_VALIDATE
    // debug builds: copy the ids back (a synchronizing copy) and check them
    if (d_slot_ids) {
        std::vector<int32_t> ids((size_t)B);
        std::vector<uint8_t> seen((size_t)slots, 0);
        const hipError_t e = hipMemcpy(ids.data(), d_slot_ids, sizeof(int32_t) * (size_t)B, hipMemcpyDeviceToHost);
        if (stq_status s = launched(e, "slot id copy")) return s;
        for (int32_t id : ids) {
            if (id < 0 || id >= slots) return fail(STQ_ERR_INVALID, "a slot id is outside [0, slots)");
            if (seen[(size_t)id]++) return fail(STQ_ERR_INVALID, "a slot id appears twice in the batch");
        }
    }
#endif
    stq::RecurrentArgs a{};
    a.s = seq_args(rule, B, N, d_cu_seqlens, d_q, d_k, d_v, d_a, d_beta);
    a.state = d_state;
    a.slot_ids = d_slot_ids;
    a.commit = d_commit;
    a.o = d_o;
    a.slots = slots;
    return launched(stq::launch_recurrent(a, rule->d_k, rule->d_v, rule->gate == STQ_GATE_KEYVEC,
                                          rule->io_dtype == STQ_BF16, static_cast<hipStream_t>(stream)),
                    "recurrent step");
}

stq_status stq_chunk_workspace(const stq_rule *rule, int32_t B, int32_t N, int32_t backward,
                               size_t *bytes) {
    stq::set_error("");
    if (stq_status s = check_rule(rule)) return s;
    if (stq_status s = check_sizes(rule, B, N)) return s;
    if (!bytes) return fail(STQ_ERR_INVALID, "bytes is NULL");
    if (((int64_t)N / stq::kC + B) * rule->H >= 1 << 23)
        return fail(STQ_ERR_UNSUPPORTED, "(N / 64 + B) * H exceeds 2^23");
    *bytes = carve(rule, B, N, backward != 0, nullptr, nullptr);
    return STQ_OK;
}

stq_status stq_chunk_forward(const stq_rule *rule, int32_t B, int32_t N, const int32_t *d_cu_seqlens,
                             const void *d_q, const void *d_k, const void *d_v, const float *d_a,
                             const float *d_beta, const float *d_initial, void *d_o, float *d_final,
                             void *d_workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (stq_status s = stq_chunk_workspace(rule, B, N, 0, &need)) return s;
    if (B == 0) return STQ_OK;
    if (stq_status s = check_ints(d_cu_seqlens, true, "cu_seqlens")) return s;
    if (N > 0)  // without tokens the states are passed on and nothing else is touched
        if (stq_status s = check_ptrs({d_q, d_k, d_v, d_a, d_beta, d_o})) return s;
    if (stq_status s = check_ptrs({d_workspace})) return s;
    if (!aligned(d_initial, 16) || !aligned(d_final, 16))
        return fail(STQ_ERR_ALIGN, "states must be 16-byte aligned");
    if (workspace_bytes < need) return fail(STQ_ERR_TOO_SMALL, "workspace smaller than stq_chunk_workspace");
    stq::ChunkArgs a{};
    a.s = seq_args(rule, B, N, d_cu_seqlens, d_q, d_k, d_v, d_a, d_beta);
    a.initial = d_initial;
    a.last = d_final;
    a.o = d_o;
    carve(rule, B, N, false, d_workspace, &a);
    const bool keyvec = rule->gate == STQ_GATE_KEYVEC, bf16 = rule->io_dtype == STQ_BF16;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (stq_status s = launched(stq::launch_chunk_prep(a, rule->d_k, keyvec, bf16, st), "chunk preparation"))
        return s;
    return launched(stq::launch_chunk_forward(a, rule->d_k, rule->d_v, keyvec, bf16, st), "chunk forward");
}

stq_status stq_chunk_backward(const stq_rule *rule, int32_t B, int32_t N, const int32_t *d_cu_seqlens,
                              const void *d_q, const void *d_k, const void *d_v, const float *d_a,
                              const float *d_beta, const float *d_initial, const void *d_do,
                              const float *d_dfinal, void *d_dq, void *d_dk, void *d_dv, float *d_da,
                              float *d_dbeta, float *d_dinitial, void *d_workspace,
                              size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (stq_status s = stq_chunk_workspace(rule, B, N, 1, &need)) return s;
    if (B == 0) return STQ_OK;
    if (stq_status s = check_ints(d_cu_seqlens, true, "cu_seqlens")) return s;
    if (N > 0)  // without tokens the states' gradients are passed on and nothing else is touched
        if (stq_status s = check_ptrs({d_q, d_k, d_v, d_a, d_beta, d_do, d_dq, d_dk, d_dv, d_da, d_dbeta})) return s;
    if (stq_status s = check_ptrs({d_workspace})) return s;
    if (!aligned(d_initial, 16) || !aligned(d_dfinal, 16) || !aligned(d_dinitial, 16))
        return fail(STQ_ERR_ALIGN, "states must be 16-byte aligned");
    if (workspace_bytes < need) return fail(STQ_ERR_TOO_SMALL, "workspace smaller than stq_chunk_workspace");
    stq::ChunkArgs a{};
    a.s = seq_args(rule, B, N, d_cu_seqlens, d_q, d_k, d_v, d_a, d_beta);
    a.initial = d_initial;
    a.dout = d_do;
    a.dlast = d_dfinal;
    a.dq = d_dq;
    a.dk = d_dk;
    a.dv = d_dv;
    a.da = d_da;
    a.dbeta = d_dbeta;
    a.dinitial = d_dinitial;
    carve(rule, B, N, true, d_workspace, &a);
    const bool keyvec = rule->gate == STQ_GATE_KEYVEC, bf16 = rule->io_dtype == STQ_BF16;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int dk = rule->d_k, dv = rule->d_v;
    if (stq_status s = launched(stq::launch_chunk_prep(a, dk, keyvec, bf16, st), "chunk preparation")) return s;
    if (stq_status s = launched(stq::launch_chunk_forward(a, dk, dv, keyvec, bf16, st), "chunk states")) return s;
    if (stq_status s = launched(stq::launch_chunk_reverse(a, dk, dv, keyvec, bf16, st), "chunk reverse")) return s;
    return launched(stq::launch_chunk_grad(a, dk, dv, keyvec, bf16, st), "chunk gradients");
}

stq_status stq_verify_workspace(int32_t B, int32_t V, size_t *bytes) {
    stq::set_error("");
    if (!bytes) return fail(STQ_ERR_INVALID, "bytes is NULL");
    if (B < 0 || V < 1) return fail(STQ_ERR_INVALID, "B must be >= 0 and V >= 1");
    *bytes = (size_t)B * stq::verify_nseg(V) * 2 * sizeof(double);
    return STQ_OK;
}

stq_status stq_verify_draft(int32_t B, int32_t T, int32_t V, int32_t dtype,
                            const int32_t *d_draft_tokens, const int32_t *d_draft_len,
                            const void *d_target, const void *d_draft, const float *d_uniform,
                            int32_t *d_n_accepted, int32_t *d_next_token, void *d_workspace,
                            size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (stq_status s = stq_verify_workspace(B, V, &need)) return s;
    if (T < 0) return fail(STQ_ERR_INVALID, "T must be >= 0");
    if (B > 65535) return fail(STQ_ERR_UNSUPPORTED, "B exceeds 65535");
    if (V > (1 << 30)) return fail(STQ_ERR_UNSUPPORTED, "V exceeds 2^30");
    if (dtype != STQ_BF16 && dtype != STQ_F32)
        return fail(STQ_ERR_INVALID, "dtype must be STQ_BF16 or STQ_F32");
    if (B == 0) return STQ_OK;
    if (stq_status s = check_ints(d_draft_tokens, T > 0, "draft tokens")) return s;
    if (stq_status s = check_ints(d_draft_len, false, "draft lengths")) return s;
    if (stq_status s = check_ints(d_uniform, true, "uniform")) return s;
    if (stq_status s = check_ints(d_n_accepted, true, "n_accepted")) return s;
    if (stq_status s = check_ints(d_next_token, true, "next_token")) return s;
    if (stq_status s = check_ptrs({d_target, d_workspace})) return s;
    if (T > 0)
        if (stq_status s = check_ptrs({d_draft})) return s;
    if (workspace_bytes < need) return fail(STQ_ERR_TOO_SMALL, "workspace smaller than stq_verify_workspace");
    stq::VerifyArgs a{};
    a.tokens = d_draft_tokens;
    a.len = d_draft_len;
    a.p = d_target;
    a.q = d_draft;
    a.uniform = d_uniform;
    a.accepted = d_n_accepted;
    a.next = d_next_token;
    a.part = static_cast<double *>(d_workspace);
    a.B = B;
    a.T = T;
    a.V = V;
    a.seg = stq::verify_seg(V);
    a.nseg = stq::verify_nseg(V);
    return launched(stq::launch_verify(a, dtype == STQ_BF16, static_cast<hipStream_t>(stream)), "verify draft");
}

}  // extern "C"
