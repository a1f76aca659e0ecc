// C ABI of libgdr: argument validation, kernel selection and launch on the
// caller's stream.  Declarations and the contract are in include/gdr.h.
#include <hip/hip_runtime.h>

#include <mutex>
#include <string.h>

#include "gdr_launch.h"
#include "gdr_attn.h"
#include "gdr_generation.h"

namespace {

constexpr uint32_t kKnownFlags = GDR_ACT_F32 | GDR_OUT_BF16 | GDR_ALPHA_SCALAR | GDR_B_SCALAR |
                                 GDR_W_SCALAR | GDR_FWD_GENERIC | GDR_GATE_LOGITS | GDR_FWD_SPLIT;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool head_size_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Sequences are counted in 32-bit integers inside the kernels and token
// offsets in 64-bit ones: B*H must stay below 2^28 and B*H*T below 2^40, so
// that no product the kernels form can overflow.
bool sizes_ok(int B, int H, int T) {
    return (long long)B * H <= (1LL << 28) && (long long)B * H * (long long)T <= (1LL << 40);
}

// Lazily checks, per device, that the current device is a gfx950.
gdr_status check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GDR_ERR_DEVICE;
    static std::mutex mu;
    static int known[64];  // 0 unknown, 1 ok, 2 bad
    if (dev >= 64) return GDR_ERR_DEVICE;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GDR_ERR_DEVICE;
        known[dev] = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    }
    return known[dev] == 1 ? GDR_OK : GDR_ERR_DEVICE;
}

// A backward workspace also holds, after the chunk kernels are done with it,
// one slot of the token-by-token recompute (checkpoints every 64 tokens and one
// segment's states), for the heads whose decay left the chunk kernels' range.
size_t bwd_need(size_t fast, int T, int d_k, int d_v) {
    if (fast == 0 || T <= 0) return fast;
    const size_t slot = gdr::exact_bwd_slot_bytes(T, d_k, d_v);
    return fast > slot ? fast : slot;
}

gdr_status from_hip(hipError_t e) {
    if (e == hipSuccess) return GDR_OK;
    if (e == hipErrorInvalidValue) return GDR_ERR_UNSUPPORTED;
    return GDR_ERR_LAUNCH;
}

// The attention layer's sizes: (batch, head) units and 16-row tiles are numbered
// in 32 bits, element offsets in 64.
bool attn_sizes_ok(int B, long long H, int T) {
    return H <= (1LL << 28) && (long long)B * H <= (1LL << 28) && (long long)B * H * (((long long)T + 15) / 16) <= (1LL << 31) - 1;
}

// A launch takes 2^32 - 1 threads along its first axis: so many workgroups of 256.
constexpr long long kMostWorkgroups = (1LL << 24) - 1;
bool grid_ok(long long workgroups) { return workgroups <= kMostWorkgroups; }

constexpr int kMostSequences = 1 << 30;               // attention: the kernels number them in 32 bits

gdr_status attn_args(int B, int Hq, int Hkv, int Tq, int Tk, int d, int window, float scale, uint32_t flags) {
    if (flags & ~(GDR_ACT_F32 | GDR_TOKEN_MAJOR)) return GDR_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hkv < 1 || Tq < 0 || Tk < 0 || window < 0) return GDR_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale >= 1e-30f) || !(scale - scale == 0.f)) return GDR_ERR_INVALID_ARG;
    // byte offsets inside a tile of 64 rows are signed 32-bit
    if (Hq > (1 << 16)) return GDR_ERR_INVALID_ARG;
    // places of queries and keys are signed 32-bit, with room for a tile behind the last
    if (Tq > (1 << 30) || Tk > (1 << 30)) return GDR_ERR_INVALID_ARG;
    if (!attn_sizes_ok(B, Hq, Tq) || !attn_sizes_ok(B, Hq, Tk)) return GDR_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || (flags & GDR_ACT_F32)) return GDR_ERR_UNSUPPORTED;
    if (!grid_ok(gdr::attn_fwd_workgroups(B, Hq, Tq))) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

// of the backward as well
gdr_status attn_bwd_args(int B, int Hq, int Hkv, int Tq, int Tk, int d, int window, float scale, uint32_t flags) {
    const gdr_status st = attn_args(B, Hq, Hkv, Tq, Tk, d, window, scale, flags);
    if (st == GDR_OK && !grid_ok(gdr::attn_bwd_workgroups(B, Hq, Hkv, Tq, Tk, d))) return GDR_ERR_INVALID_ARG;
    return st;
}

gdr::AttnStrides attn_strides(int H, int T, int d, bool token_major) {
    if (token_major) return {(long long)T * H * d, d, (long long)H * d};
    return {(long long)H * T * d, (long long)T * d, d};
}

gdr::AttnParams attn_params(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Tq, int Tk,
                            int d, int window, float scale, uint32_t flags) {
    gdr::AttnParams p = {};
    p.q = q; p.k = k; p.v = v;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Tq = Tq; p.Tk = Tk; p.d = d;
    // a window that reaches behind the first key is none
    p.window = window < Tk ? window : 0;
    p.scale = scale; p.splits = 1; p.few = false; p.split_steps = 0;
    p.sq = attn_strides(Hq, Tq, d, (flags & GDR_TOKEN_MAJOR) != 0);
    p.sk = attn_strides(Hkv, Tk, d, (flags & GDR_TOKEN_MAJOR) != 0);
    return p;
}

size_t attn_delta_bytes(int B, int Hq, int Tq) {
    return (2 * (size_t)B * Hq * Tq * sizeof(float) + 255) / 256 * 256;   // D, then the log-sum-exps
}

gdr_status attn_bwd_run(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                        void* dq, void* dk, void* dv, const int* cu_seqlens, int nseq, int B, int Hq, int Hkv, int Tq,
                        int Tk, int d, int window, float scale, uint32_t flags, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv, workspace};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    const size_t need = gdr_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::AttnParams p = attn_params(q, k, v, B, Hq, Hkv, Tq, Tk, d, window, scale, flags);
    p.o = const_cast<void*>(o); p.lse = const_cast<float*>(lse);
    p.dO = dO; p.dq = dq; p.dk = dk; p.dv = dv;
    p.cu_seqlens = cu_seqlens; p.nseq = nseq;
    p.delta = static_cast<float*>(workspace);
    p.splits = gdr::attn_bwd_splits(B, Hq, Hkv, Tq, Tk);
    if (p.splits > 1)
        p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + attn_delta_bytes(B, Hq, Tq));
    return from_hip(gdr::launch_attn_bwd(p, (hipStream_t)stream));
}

gdr_status decode_args(int N, int Hq, int Hkv, int d, int n_pages, int max_pages, int window, float scale,
                       uint32_t flags) {
    if (flags & ~GDR_OUT_BF16) return GDR_ERR_INVALID_ARG;
    if (N < 1 || Hq < 1 || Hkv < 1 || n_pages < 1 || max_pages < 1 || window < 0) return GDR_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale >= 1e-30f) || !(scale - scale == 0.f)) return GDR_ERR_INVALID_ARG;
    // (sequence, head) pairs and a sequence's tokens are numbered in 32 bits
    if ((long long)N * Hq > (1LL << 28) || max_pages > (1 << 24)) return GDR_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    if (!grid_ok(gdr::attn_decode_workgroups(N, Hq, Hkv))) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

// Rows of a block table, and pages, are numbered in 32 bits, as are all rows' pages together.
gdr_status pages_args(int N, int Hkv, int d, int n_pages, int max_pages, uint32_t flags) {
    if (flags != 0) return GDR_ERR_INVALID_ARG;
    if (N < 1 || Hkv < 1 || n_pages < 1 || max_pages < 1) return GDR_ERR_INVALID_ARG;
    if (N > (1 << 20) || Hkv > 65535 || n_pages > (1 << 30) || max_pages > (1 << 24)) return GDR_ERR_INVALID_ARG;
    if ((long long)N * max_pages > (1LL << 31) - 1) return GDR_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

gdr_status beam_args(int G, int K, int M, int V, long long stride, int end_token, uint32_t flags) {
    if (flags & ~(GDR_ACT_F32 | GDR_KEEP_SLOTS)) return GDR_ERR_INVALID_ARG;
    if (G < 1 || K < 1 || M < 1 || V < 1 || stride < V || end_token < -1 || end_token >= V)
        return GDR_ERR_INVALID_ARG;
    if ((long long)K * V < M || ((flags & GDR_KEEP_SLOTS) && M != K)) return GDR_ERR_INVALID_ARG;
    if (K > gdr::kMostBeams || M > gdr::kMostSelected || V > gdr::kMostTokens) return GDR_ERR_UNSUPPORTED;
    // rows are on the grid's second axis; element offsets in 64 bits
    if ((long long)G * K > 65535 || stride > (1LL << 40)) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_abi_version(void) { return GDR_ABI_VERSION; }

const char* gdr_status_string(gdr_status s) {
    switch (s) {
        case GDR_OK: return "ok";
        case GDR_ERR_INVALID_ARG: return "invalid argument";
        case GDR_ERR_UNSUPPORTED: return "unsupported shape, chunk or dtype";
        case GDR_ERR_WORKSPACE: return "workspace missing or too small";
        case GDR_ERR_LAUNCH: return "kernel launch failed";
        case GDR_ERR_DEVICE: return "no usable gfx950 device";
    }
    return "unknown status";
}

size_t gdr_chunk_fwd_workspace_bytes(int B, int H, int T, int d_k, int d_v, int chunk,
                                     uint32_t flags) {
    if (B < 1 || H < 1 || T < 1 || !(chunk == 16 || chunk == 32 || chunk == 64)) return 0;
    if (T % chunk != 0 || !sizes_ok(B, H, T)) return 0;
    if (!gdr::fwd_wy_supported(d_k, d_v, chunk, flags)) return 0;
    return gdr::fwd_fz_workspace_bytes(B * H, T, d_k, d_v);
}

gdr_status gdr_chunk_fwd(const void* q, const void* k, const void* v, const float* log_alpha,
                         const void* b, const void* w, const float* S0, void* o, float* S_final,
                         int B, int H, int T, int d_k, int d_v, int chunk, uint32_t flags,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (flags & ~kKnownFlags) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0) return GDR_ERR_INVALID_ARG;
    if (!(chunk == 16 || chunk == 32 || chunk == 64)) return GDR_ERR_INVALID_ARG;
    if (T % chunk != 0) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d_k) || !head_size_ok(d_v)) return GDR_ERR_UNSUPPORTED;
    if (T > 0 && (!q || !k || !v || !log_alpha || !b || !w || !o)) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, b, w, S0, o, S_final, workspace};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (!sizes_ok(B, H, T)) return GDR_ERR_INVALID_ARG;
    if (!gdr::fwd_supported(d_k, d_v, chunk, flags)) return GDR_ERR_UNSUPPORTED;
    const size_t need = gdr_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk, flags);
    const bool two_pass = workspace != nullptr && need > 0;
    if (two_pass && workspace_bytes < need) return GDR_ERR_WORKSPACE;
    if ((flags & GDR_GATE_LOGITS) && T > 0 && !two_pass) return GDR_ERR_UNSUPPORTED;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;

    gdr::FwdParams p;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w;
    p.S0 = S0; p.o = o; p.Sf = S_final; p.states = nullptr; p.state_frags = nullptr;
    p.cu_seqlens = nullptr; p.chunk_off = nullptr; p.chunk_tab = nullptr; p.seq_order = nullptr; p.nseq = 0;
    p.BH = B * H; p.T = T; p.flags = flags;
    if (two_pass) return from_hip(gdr::launch_fwd_fz(p, d_k, d_v, workspace, (hipStream_t)stream));
    int used = 0;
    const hipError_t e = gdr::launch_fwd(p, d_k, d_v, chunk, (hipStream_t)stream, &used);
    if (e != hipSuccess) return from_hip(e);
    // heads whose decay left the chunk kernel's operand range: token by token
    return from_hip(gdr::launch_exact_fwd(p, d_k, d_v, (hipStream_t)stream));
}

size_t gdr_chunk_fwd_varlen_workspace_bytes(int nseq, int H, int T, int d_k, int d_v,
                                            uint32_t flags) {
    if (nseq < 1 || H < 1 || T < 0 || (long long)nseq * H > (1LL << 28)) return 0;
    if ((flags & ~kKnownFlags) || !gdr::fwd_wy_supported(d_k, d_v, 64, flags)) return 0;
    return gdr::fwd_fz_varlen_workspace_bytes(H, T, nseq, d_k, d_v);
}

gdr_status gdr_chunk_fwd_varlen(const void* q, const void* k, const void* v,
                                const float* log_alpha, const void* b, const void* w,
                                const float* S0, void* o, float* S_final,
                                const int* cu_seqlens, int nseq, int H, int T,
                                int d_k, int d_v, uint32_t flags, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (flags & ~kKnownFlags) return GDR_ERR_INVALID_ARG;
    if (nseq < 1 || H < 1 || T < 0 || !cu_seqlens) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d_k) || !head_size_ok(d_v)) return GDR_ERR_UNSUPPORTED;
    if (T > 0 && (!q || !k || !v || !log_alpha || !b || !w || !o)) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, b, w, S0, o, S_final, workspace};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    // work items (head, chunk) are numbered in 32-bit integers
    if ((long long)nseq * H > (1LL << 28) || (long long)H * (T / 64 + nseq) > (1LL << 30))
        return GDR_ERR_INVALID_ARG;
    if (!gdr::fwd_wy_supported(d_k, d_v, 64, flags)) return GDR_ERR_UNSUPPORTED;
    const size_t need = gdr::fwd_fz_varlen_workspace_bytes(H, T, nseq, d_k, d_v);
    if (!workspace || workspace_bytes < need) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;

    gdr::FwdParams p;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w;
    p.S0 = S0; p.o = o; p.Sf = S_final; p.states = nullptr; p.state_frags = nullptr;
    p.cu_seqlens = cu_seqlens; p.chunk_off = nullptr; p.chunk_tab = nullptr; p.seq_order = nullptr; p.nseq = nseq;
    p.BH = H; p.T = T; p.flags = flags;
    // the producer over every packed chunk, then one chain per (sequence, head);
    // their operands reference each block's own decay, so any decay gives values
    return from_hip(gdr::launch_fwd_fz_varlen(p, d_k, d_v, workspace, workspace_bytes, (hipStream_t)stream));
}

gdr_status gdr_decode_step(const void* q, const void* k, const void* v, const float* log_alpha,
                           const void* b, const void* w, float* S, void* o, int N, int H,
                           int d_k, int d_v, uint32_t flags, void* stream) {
    if (flags & ~(kKnownFlags & ~GDR_FWD_SPLIT)) return GDR_ERR_INVALID_ARG;
    if (N < 1 || H < 1) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d_k) || !head_size_ok(d_v)) return GDR_ERR_UNSUPPORTED;
    if (!q || !k || !v || !log_alpha || !b || !w || !S || !o) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, b, w, S, o};
    for (const void* ptr : ptrs)
        if (!aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if ((long long)N * H > (1LL << 31) - 1) return GDR_ERR_INVALID_ARG;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;

    gdr::DecodeParams p;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w; p.S = S; p.o = o;
    p.NH = (long long)N * H; p.flags = flags;
    return from_hip(gdr::launch_decode(p, d_k, d_v, (hipStream_t)stream));
}

size_t gdr_chunk_bwd_workspace_bytes(int B, int H, int T, int d_k, int d_v, int chunk,
                                     uint32_t flags) {
    if (B < 1 || H < 1 || T < 0 || !(chunk == 16 || chunk == 32 || chunk == 64)) return 0;
    if (T % chunk != 0 || !sizes_ok(B, H, T)) return 0;
    if (!gdr::bwd_supported(d_k, d_v, chunk, flags)) return 0;
    return bwd_need(gdr::bwd_workspace_bytes(B * H, T, d_k, d_v, chunk, flags), T, d_k, d_v);
}

gdr_status gdr_chunk_bwd(const void* q, const void* k, const void* v, const float* log_alpha,
                         const void* b, const void* w, const float* S0, const void* dO,
                         const float* dS_final, float* dq, float* dk, float* dv,
                         float* dlog_alpha, float* db, float* dw, float* dS0, int B, int H,
                         int T, int d_k, int d_v, int chunk, uint32_t flags, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (flags & ~(kKnownFlags & ~GDR_OUT_BF16)) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0) return GDR_ERR_INVALID_ARG;
    if (!(chunk == 16 || chunk == 32 || chunk == 64)) return GDR_ERR_INVALID_ARG;
    if (T % chunk != 0) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d_k) || !head_size_ok(d_v)) return GDR_ERR_UNSUPPORTED;
    if (T > 0 && (!q || !k || !v || !log_alpha || !b || !w || !dO || !dq || !dk || !dv ||
                  !dlog_alpha || !db || !dw))
        return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, b, w, S0, dO, dS_final, dq, dk, dv,
                          dlog_alpha, db, dw, dS0, workspace};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (!sizes_ok(B, H, T)) return GDR_ERR_INVALID_ARG;
    if (!gdr::bwd_supported(d_k, d_v, chunk, flags)) return GDR_ERR_UNSUPPORTED;
    if ((flags & GDR_GATE_LOGITS) && T > 0 && !gdr::bwd_two_pass_supported(d_k, d_v, chunk, flags))
        return GDR_ERR_UNSUPPORTED;
    const size_t need = gdr::bwd_workspace_bytes(B * H, T, d_k, d_v, chunk, flags);
    if (need > 0 && (!workspace || workspace_bytes < bwd_need(need, T, d_k, d_v))) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;

    gdr::BwdParams p;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w; p.S0 = S0;
    p.dO = dO; p.dSf = dS_final;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dla = dlog_alpha; p.db = db; p.dw = dw; p.dS0 = dS0;
    p.states = nullptr; p.dstates = nullptr; p.records = nullptr;
    p.state_frags = nullptr; p.dstate_frags = nullptr;
    p.cu_seqlens = nullptr; p.chunk_off = nullptr; p.chunk_tab = nullptr; p.seq_order = nullptr; p.nseq = 0;
    p.BH = B * H; p.T = T; p.flags = flags;
    if (need > 0) {
        const size_t sb = gdr::bwd_states_bytes(B * H, T, d_k, d_v, chunk, flags);
        char* base = reinterpret_cast<char*>(workspace);
        // states, then state gradients (fp32 rows for the generic path, f16
        // fragments for the two-pass path), then the two-pass forward's records
        p.states = reinterpret_cast<float*>(base);
        p.dstates = reinterpret_cast<float*>(base + sb);
        p.state_frags = base;
        p.dstate_frags = base + sb;
        if (need > 2 * sb) p.records = base + 2 * sb;
    }
    const hipError_t e = gdr::launch_bwd(p, d_k, d_v, chunk, (hipStream_t)stream);
    if (e != hipSuccess) return from_hip(e);
    // heads whose decay left the chunk kernels' operand range: token by token,
    // in the workspace the chunk kernels are done with
    return from_hip(gdr::launch_exact_bwd(p, d_k, d_v, workspace, workspace_bytes, (hipStream_t)stream));
}

size_t gdr_chunk_bwd_varlen_workspace_bytes(int nseq, int H, int T, int d_k, int d_v, uint32_t flags) {
    if (nseq < 1 || H < 1 || T < 0 || (long long)nseq * H > (1LL << 28)) return 0;
    if ((flags & ~(kKnownFlags & ~GDR_OUT_BF16)) || !gdr::fwd_wy_supported(d_k, d_v, 64, flags)) return 0;
    return bwd_need(gdr::bwd_varlen_workspace_bytes(H, T, nseq, d_k, d_v), T, d_k, d_v);
}

gdr_status gdr_chunk_bwd_varlen(const void* q, const void* k, const void* v, const float* log_alpha,
                                const void* b, const void* w, const float* S0, const void* dO,
                                const float* dS_final, float* dq, float* dk, float* dv,
                                float* dlog_alpha, float* db, float* dw, float* dS0,
                                const int* cu_seqlens, int nseq, int H, int T, int d_k, int d_v,
                                uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    if (flags & ~(kKnownFlags & ~GDR_OUT_BF16)) return GDR_ERR_INVALID_ARG;
    if (nseq < 1 || H < 1 || T < 0 || !cu_seqlens) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d_k) || !head_size_ok(d_v)) return GDR_ERR_UNSUPPORTED;
    if (T > 0 && (!q || !k || !v || !log_alpha || !b || !w || !dO || !dq || !dk || !dv ||
                  !dlog_alpha || !db || !dw))
        return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, b, w, S0, dO, dS_final, dq, dk, dv,
                          dlog_alpha, db, dw, dS0, workspace};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    // work items (head, chunk) are numbered in 32-bit integers
    if ((long long)nseq * H > (1LL << 28) || (long long)H * (T / 64 + nseq) > (1LL << 30))
        return GDR_ERR_INVALID_ARG;
    if (d_k != d_v || !gdr::fwd_wy_supported(d_k, d_v, 64, flags)) return GDR_ERR_UNSUPPORTED;
    const size_t need = bwd_need(gdr::bwd_varlen_workspace_bytes(H, T, nseq, d_k, d_v), T, d_k, d_v);
    if (!workspace || workspace_bytes < need) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;

    gdr::BwdParams p;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w; p.S0 = S0;
    p.dO = dO; p.dSf = dS_final;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dla = dlog_alpha; p.db = db; p.dw = dw; p.dS0 = dS0;
    p.states = nullptr; p.dstates = nullptr; p.records = nullptr;
    p.state_frags = nullptr; p.dstate_frags = nullptr;
    p.cu_seqlens = cu_seqlens; p.chunk_off = nullptr; p.chunk_tab = nullptr; p.seq_order = nullptr;
    p.nseq = nseq;
    p.BH = H; p.T = T; p.flags = flags;
    const hipError_t e = gdr::launch_bwd_varlen(p, d_k, d_v, workspace, workspace_bytes, (hipStream_t)stream);
    if (e != hipSuccess) return from_hip(e);
    // sequences whose decay left the chunk kernels' operand range: token by token
    return from_hip(gdr::launch_exact_bwd(p, d_k, d_v, workspace, workspace_bytes, (hipStream_t)stream));
}

gdr_status gdr_mixer_prologue(const void* q_pre, const void* k_pre, const void* v_pre,
                              const float* conv_q, const float* conv_k, const float* conv_v,
                              const float* a_pre, const void* b_pre, const void* w_pre, void* q,
                              void* k, void* v, float* log_alpha, void* b, void* w, int B, int H,
                              int T, int d_k, int d_v, uint32_t flags, void* stream) {
    const uint32_t gate_modes = GDR_ALPHA_SCALAR | GDR_B_SCALAR | GDR_W_SCALAR | GDR_GATE_LOGITS;
    if (flags & ~(kKnownFlags & ~GDR_OUT_BF16 & ~GDR_FWD_GENERIC)) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0) return GDR_ERR_INVALID_ARG;
    if ((long long)B * H > (1LL << 28) || (long long)B * H * (((long long)T + 63) / 64) > (1LL << 31) - 1)
        return GDR_ERR_INVALID_ARG;
    if (!gdr::mixer_supported(d_k) || !gdr::mixer_supported(d_v) || (flags & ~gate_modes))
        return GDR_ERR_UNSUPPORTED;
    // with GDR_GATE_LOGITS the gates stay logits for the recurrence to take:
    // only q, k and v are produced and the gate pointers are not used
    const bool gates = !(flags & GDR_GATE_LOGITS);
    const void* ptrs[] = {q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, q, k, v,
                          a_pre, b_pre, w_pre, log_alpha, b, w};
    for (int i = 0; i < 15; ++i) {
        const void* ptr = ptrs[i];
        if (T > 0 && !ptr && (i < 9 || gates)) return GDR_ERR_INVALID_ARG;
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    }
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::MixerParams p;
    p.q_pre = q_pre; p.k_pre = k_pre; p.v_pre = v_pre;
    p.conv_q = conv_q; p.conv_k = conv_k; p.conv_v = conv_v;
    p.a_pre = a_pre; p.b_pre = b_pre; p.w_pre = w_pre;
    p.q = q; p.k = k; p.v = v; p.la = log_alpha; p.b = b; p.w = w;
    p.BH = B * H; p.H = H; p.T = T; p.flags = flags;
    return from_hip(gdr::launch_mixer_prologue(p, d_k, d_v, (hipStream_t)stream));
}

gdr_status gdr_mixer_epilogue(const float* o, const void* g, const float* norm_weight, void* y,
                              int B, int H, int T, int d_v, uint32_t flags, void* stream) {
    if (flags != 0) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0) return GDR_ERR_INVALID_ARG;
    if ((long long)B * H > (1LL << 28) || (long long)B * H * T > (1LL << 40)) return GDR_ERR_INVALID_ARG;
    if (!gdr::mixer_supported(d_v)) return GDR_ERR_UNSUPPORTED;
    const void* ptrs[] = {o, g, norm_weight, y};
    for (const void* ptr : ptrs) {
        if (T > 0 && !ptr) return GDR_ERR_INVALID_ARG;
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    }
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::EpilogueParams p;
    p.o = o; p.g = g; p.norm_weight = norm_weight; p.y = y;
    p.rows = (long long)B * H * T;
    return from_hip(gdr::launch_mixer_epilogue(p, d_v, (hipStream_t)stream));
}

size_t gdr_mixer_bwd_workspace_bytes(int B, int H, int T, int d_k, int d_v) {
    if (B < 1 || H < 1 || T < 1 || d_k != d_v || !gdr::mixer_supported(d_k)) return 0;
    if ((long long)B * H > (1LL << 28) || (long long)B * H * (((long long)T + 63) / 64) > (1LL << 31) - 1) return 0;
    const size_t pro = gdr::mixer_prologue_bwd_workspace_bytes(B * H, T, d_k, d_v);
    const size_t epi = gdr::mixer_epilogue_bwd_workspace_bytes(d_v);
    return pro > epi ? pro : epi;
}

gdr_status gdr_mixer_prologue_bwd(const void* q_pre, const void* k_pre, const void* v_pre,
                                  const float* conv_q, const float* conv_k, const float* conv_v,
                                  const float* dq, const float* dk, const float* dv, float* dq_pre,
                                  float* dk_pre, float* dv_pre, float* dconv_q, float* dconv_k,
                                  float* dconv_v, int B, int H, int T, int d_k, int d_v,
                                  uint32_t flags, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    if (flags != 0) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 1) return GDR_ERR_INVALID_ARG;
    if (d_k != d_v || !gdr::mixer_supported(d_k)) return GDR_ERR_UNSUPPORTED;
    const void* ptrs[] = {q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, dq, dk, dv, dq_pre, dk_pre,
                          dv_pre, dconv_q, dconv_k, dconv_v, workspace};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    const size_t need = gdr_mixer_bwd_workspace_bytes(B, H, T, d_k, d_v);
    if (need == 0) return GDR_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::MixerBwdParams p;
    p.q_pre = q_pre; p.k_pre = k_pre; p.v_pre = v_pre;
    p.conv_q = conv_q; p.conv_k = conv_k; p.conv_v = conv_v;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dq_pre = dq_pre; p.dk_pre = dk_pre; p.dv_pre = dv_pre;
    p.dconv_q = dconv_q; p.dconv_k = dconv_k; p.dconv_v = dconv_v;
    p.part = reinterpret_cast<float*>(workspace);
    p.BH = B * H; p.H = H; p.T = T;
    return from_hip(gdr::launch_mixer_prologue_bwd(p, d_k, d_v, (hipStream_t)stream));
}

gdr_status gdr_mixer_epilogue_bwd(const float* o, const void* g, const float* norm_weight,
                                  const float* dy, float* d_o, float* dg, float* dnorm_weight,
                                  int B, int H, int T, int d_v, uint32_t flags, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (flags != 0) return GDR_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 1) return GDR_ERR_INVALID_ARG;
    if ((long long)B * H > (1LL << 28) || (long long)B * H * T > (1LL << 40)) return GDR_ERR_INVALID_ARG;
    if (!gdr::mixer_supported(d_v)) return GDR_ERR_UNSUPPORTED;
    const void* ptrs[] = {o, g, norm_weight, dy, d_o, dg, dnorm_weight, workspace};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (workspace_bytes < gdr::mixer_epilogue_bwd_workspace_bytes(d_v)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::EpilogueBwdParams p;
    p.o = o; p.g = g; p.norm_weight = norm_weight; p.dy = dy;
    p.d_o = d_o; p.dg = dg; p.dnorm_weight = dnorm_weight;
    p.part = reinterpret_cast<float*>(workspace);
    p.rows = (long long)B * H * T;
    return from_hip(gdr::launch_mixer_epilogue_bwd(p, d_v, (hipStream_t)stream));
}

gdr_status gdr_rope(const void* q, const void* k, void* q_out, void* k_out, const float* inv_freq,
                    const int* positions, int position0, int B, int Hq, int Hk, int T, int d, int rot_dim,
                    float scale, uint32_t flags, void* stream) {
    if (flags & ~(GDR_ACT_F32 | GDR_TOKEN_MAJOR | GDR_ROPE_INTERLEAVED | GDR_ROPE_INVERSE)) return GDR_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || Hq < 0 || Hk < 0 || (long long)Hq + Hk < 1) return GDR_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return GDR_ERR_UNSUPPORTED;
    if (rot_dim < 1 || rot_dim > d) return GDR_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0) return GDR_ERR_UNSUPPORTED;
    if (!(scale - scale == 0.f)) return GDR_ERR_INVALID_ARG;   // infinite or NaN
    if (!attn_sizes_ok(B, (long long)Hq + Hk, T) || (long long)B * T > (1LL << 31) - 1) return GDR_ERR_INVALID_ARG;
    if (!grid_ok(gdr::rope_workgroups((long long)B * T, d, flags))) return GDR_ERR_INVALID_ARG;
    if (T > 0 && (!inv_freq || (Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)))) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, q_out, k_out, inv_freq, positions};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::RopeParams p;
    p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
    p.inv_freq = inv_freq; p.positions = positions; p.position0 = position0;
    p.rows = (long long)B * T; p.T = T; p.Hq = Hq; p.Hk = Hk; p.d = d; p.rot = rot_dim;
    p.heads = 0; p.scale = scale; p.flags = flags;
    return from_hip(gdr::launch_rope(p, (hipStream_t)stream));
}

gdr_status gdr_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                        int Tq, int Tk, int d, int window, float scale, uint32_t flags, void* stream) {
    const gdr_status st = attn_args(B, Hq, Hkv, Tq, Tk, d, window, scale, flags);
    if (st != GDR_OK) return st;
    if (Tq > 0 && (!q || !o || (Tk > 0 && (!k || !v)))) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, o, lse};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::AttnParams p = attn_params(q, k, v, B, Hq, Hkv, Tq, Tk, d, window, scale, flags);
    p.o = o; p.lse = lse;
    return from_hip(gdr::launch_attn_fwd(p, (hipStream_t)stream));
}

gdr_status gdr_attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int* cu_seqlens, int nseq, int Hq, int Hkv, int T, int d, int window,
                               float scale, uint32_t flags, void* stream) {
    const gdr_status st = attn_args(1, Hq, Hkv, T, T, d, window, scale, flags);
    if (st != GDR_OK) return st;
    if (nseq < 1 || nseq > kMostSequences || !cu_seqlens) return GDR_ERR_INVALID_ARG;
    if (T > 0 && (!q || !o || !k || !v)) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, o, lse, cu_seqlens};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::AttnParams p = attn_params(q, k, v, 1, Hq, Hkv, T, T, d, window, scale, flags);
    p.o = o; p.lse = lse; p.cu_seqlens = cu_seqlens; p.nseq = nseq;
    return from_hip(gdr::launch_attn_fwd(p, (hipStream_t)stream));
}

size_t gdr_attn_bwd_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int d) {
    if (attn_bwd_args(B, Hq, Hkv, Tq, Tk, d, 0, 1.f, 0) != GDR_OK) return 0;
    const int splits = gdr::attn_bwd_splits(B, Hq, Hkv, Tq, Tk);
    const size_t part = splits > 1 ? 2 * (size_t)gdr::attn_bwd_splits_most(splits, Tk) * B * Hkv * Tk * d * sizeof(float) : 0;
    return attn_delta_bytes(B, Hq, Tq) + part;
}

gdr_status gdr_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                        void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Tq, int Tk, int d, int window,
                        float scale, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    const gdr_status st = attn_bwd_args(B, Hq, Hkv, Tq, Tk, d, window, scale, flags);
    if (st != GDR_OK) return st;
    if (Tq > 0 && (!q || !o || !lse || !dO || !dq)) return GDR_ERR_INVALID_ARG;
    if (Tk > 0 && (!k || !v || !dk || !dv)) return GDR_ERR_INVALID_ARG;
    return attn_bwd_run(q, k, v, o, lse, dO, dq, dk, dv, nullptr, 0, B, Hq, Hkv, Tq, Tk, d, window, scale, flags,
                        workspace, workspace_bytes, stream);
}

gdr_status gdr_attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse,
                               const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens, int nseq, int Hq,
                               int Hkv, int T, int d, int window, float scale, uint32_t flags, void* workspace,
                               size_t workspace_bytes, void* stream) {
    const gdr_status st = attn_bwd_args(1, Hq, Hkv, T, T, d, window, scale, flags);
    if (st != GDR_OK) return st;
    if (nseq < 1 || nseq > kMostSequences || !cu_seqlens || !aligned16(cu_seqlens)) return GDR_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv)) return GDR_ERR_INVALID_ARG;
    return attn_bwd_run(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, nseq, 1, Hq, Hkv, T, T, d, window, scale, flags,
                        workspace, workspace_bytes, stream);
}

gdr_status gdr_kv_append(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         const int* block_table, const int* cache_len, const int* cu_seqlens, int nseq, int Hkv,
                         int T, int d, int n_pages, int max_pages, uint32_t flags, void* stream) {
    if (flags & ~GDR_TOKEN_MAJOR) return GDR_ERR_INVALID_ARG;
    if (nseq < 1 || Hkv < 1 || T < 0 || n_pages < 1 || max_pages < 1) return GDR_ERR_INVALID_ARG;
    if (!cu_seqlens && T != nseq) return GDR_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    // (sequence, head) pairs of one call are numbered in 32 bits, heads on the grid's second axis
    if (Hkv > 65535 || T > (1 << 30) || (long long)nseq * Hkv > (1LL << 31) - 1) return GDR_ERR_INVALID_ARG;
    if (!grid_ok(gdr::kv_append_workgroups(nseq, Hkv, T, d, cu_seqlens != nullptr))) return GDR_ERR_INVALID_ARG;
    if ((long long)nseq * max_pages > (1LL << 40)) return GDR_ERR_INVALID_ARG;
    if (T > 0 && (!k || !v)) return GDR_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !cache_len) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, cu_seqlens};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (T == 0) return GDR_OK;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::KvAppendParams p;
    p.k = k; p.v = v;
    p.k_cache = static_cast<uint8_t*>(k_cache); p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.block_table = block_table; p.cache_len = cache_len; p.cu_seqlens = cu_seqlens;
    p.nseq = nseq; p.Hkv = Hkv; p.T = T; p.d = d; p.n_pages = n_pages; p.max_pages = max_pages;
    const bool token_major = !cu_seqlens || (flags & GDR_TOKEN_MAJOR);
    p.st = token_major ? (long long)Hkv * d : d;
    p.sh = token_major ? d : (long long)T * d;
    return from_hip(gdr::launch_kv_append(p, (hipStream_t)stream));
}

size_t gdr_attn_decode_workspace_bytes(int N, int Hq, int Hkv, int d, int max_pages, int window) {
    if (decode_args(N, Hq, Hkv, d, 1, max_pages, window, 1.f, 0) != GDR_OK) return 0;
    int per = 0;
    const int splits = gdr::attn_decode_splits(N, Hq, Hkv, max_pages, window, &per);
    return splits > 1 ? (size_t)splits * N * Hq * (d + 2) * sizeof(float) : 0;
}

gdr_status gdr_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* block_table, const int* cache_len, void* o, int N,
                           int Hq, int Hkv, int d, int n_pages, int max_pages, int window, float scale,
                           uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    const gdr_status st = decode_args(N, Hq, Hkv, d, n_pages, max_pages, window, scale, flags);
    if (st != GDR_OK) return st;
    const void* ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, o};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (workspace && !aligned16(workspace)) return GDR_ERR_INVALID_ARG;
    const size_t need = gdr_attn_decode_workspace_bytes(N, Hq, Hkv, d, max_pages, window);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::AttnDecodeParams p;
    p.q = q;
    p.k_cache = static_cast<const uint8_t*>(k_cache); p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale; p.block_table = block_table; p.cache_len = cache_len; p.o = o;
    p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.n_pages = n_pages; p.max_pages = max_pages; p.window = window;
    p.splits = gdr::attn_decode_splits(N, Hq, Hkv, max_pages, window, &p.split_pages);
    p.part_o = need > 0 ? static_cast<float*>(workspace) : nullptr;
    p.part_ml = need > 0 ? p.part_o + (size_t)p.splits * N * Hq * d : nullptr;
    p.scale = scale; p.flags = flags;
    return from_hip(gdr::launch_attn_decode(p, (hipStream_t)stream));
}

size_t gdr_attn_decode_shared_workspace_bytes(int N, int groups, int Hq, int Hkv, int d, int max_pages, int window) {
    if (decode_args(N, Hq, Hkv, d, 1, max_pages, window, 1.f, 0) != GDR_OK || groups < 1 || groups > gdr::kMostGroups) return 0;
    return gdr::attn_shared_plan(N, groups, Hq, Hkv, d, max_pages, window).bytes;
}

gdr_status gdr_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                  const float* v_scale, const int* block_table, const int* cache_len,
                                  const int* group_start, const int* shared_pages, void* o, int N, int groups, int Hq,
                                  int Hkv, int d, int n_pages, int max_pages, int window, float scale, uint32_t flags,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const gdr_status st = decode_args(N, Hq, Hkv, d, n_pages, max_pages, window, scale, flags);
    if (st != GDR_OK) return st;
    if (groups < 1) return GDR_ERR_INVALID_ARG;
    if (groups > gdr::kMostGroups) return GDR_ERR_UNSUPPORTED;
    const gdr::SharedPlan x = gdr::attn_shared_plan(N, groups, Hq, Hkv, d, max_pages, window);
    if (!grid_ok(gdr::attn_shared_workgroups(x, (long long)N * Hq))) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, group_start, shared_pages, o};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if (workspace && !aligned16(workspace)) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < x.bytes) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::SharedParams p;
    p.q = q;
    p.k_cache = static_cast<const uint8_t*>(k_cache); p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale; p.block_table = block_table; p.cache_len = cache_len;
    p.group_start = group_start; p.shared_pages = shared_pages; p.o = o;
    p.N = N; p.groups = groups; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.n_pages = n_pages; p.max_pages = max_pages;
    p.window = window; p.width = x.width; p.units = (int)x.units; p.workgroups = x.workgroups; p.own_splits = x.own_splits; p.few = x.few;
    p.own_runs = x.own_items * x.own_splits;
    char* ws = static_cast<char*>(workspace);
    p.plan_head = ws + x.at_head;
    p.plan_groups = ws + x.at_groups;
    p.plan_sequences = ws + x.at_sequences;
    p.plan_items = reinterpret_cast<int*>(ws + x.at_items);
    p.part_o = reinterpret_cast<float*>(ws + x.at_part_o);
    p.part_ml = reinterpret_cast<float*>(ws + x.at_part_ml);
    p.own_o = reinterpret_cast<float*>(ws + x.at_own_o);
    p.own_ml = reinterpret_cast<float*>(ws + x.at_own_ml);
    p.scale = scale; p.flags = flags;
    return from_hip(gdr::launch_attn_shared(p, (hipStream_t)stream));
}

size_t gdr_kv_fork_workspace_bytes(int N, int n_pages) {
    if (pages_args(N, 1, 64, n_pages, 1, 0) != GDR_OK) return 0;
    return gdr::kv_fork_workspace(N, n_pages);
}

gdr_status gdr_kv_fork(void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int* block_table,
                       const int* cache_len, const int* parent, const int* room, const uint8_t* held, int* table_out,
                       int* len_out, int* missing, int N_in, int N, int room_all, int Hkv, int d, int n_pages,
                       int max_pages, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    gdr_status st = pages_args(N, Hkv, d, n_pages, max_pages, flags);
    if (st == GDR_OK) st = pages_args(N_in, Hkv, d, n_pages, max_pages, flags);
    if (st != GDR_OK) return st;
    if (room_all < 0 || (!parent && N_in != N)) return GDR_ERR_INVALID_ARG;
    if (!grid_ok(gdr::kv_fork_workgroups(N, Hkv, d, n_pages, max_pages))) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {k_cache, v_cache, k_scale, v_scale, block_table, cache_len, table_out, len_out, missing};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    const void* maybe[] = {parent, room, held, workspace};
    for (const void* ptr : maybe)
        if (ptr && !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    // rows are read by others' workgroups while they are written
    if (parent && (table_out == block_table || len_out == cache_len)) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdr_kv_fork_workspace_bytes(N, n_pages)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::PagesParams p = {};
    p.k_cache = static_cast<uint8_t*>(k_cache); p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.block_table = block_table; p.cache_len = cache_len; p.parent = parent; p.room = room; p.held = held;
    p.table_out = table_out; p.len_out = len_out; p.missing = missing;
    p.N_in = N_in; p.N = N; p.room_all = room_all; p.Hkv = Hkv; p.d = d; p.n_pages = n_pages; p.max_pages = max_pages;
    p.workspace = workspace;
    return from_hip(gdr::launch_kv_fork(p, (hipStream_t)stream));
}

size_t gdr_kv_compact_workspace_bytes(int n_pages) {
    if (pages_args(1, 1, 64, n_pages, 1, 0) != GDR_OK) return 0;
    return gdr::kv_compact_workspace(n_pages);
}

gdr_status gdr_kv_compact(void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int* block_table,
                          const int* cache_len, const uint8_t* held, int* table_out, int* used, int N, int Hkv, int d,
                          int n_pages, int max_pages, uint32_t flags, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const gdr_status st = pages_args(N, Hkv, d, n_pages, max_pages, flags);
    if (st != GDR_OK) return st;
    if (!grid_ok(gdr::kv_compact_workgroups(N, n_pages, max_pages))) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {k_cache, v_cache, k_scale, v_scale, block_table, cache_len, table_out, used};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if ((held && !aligned16(held)) || (workspace && !aligned16(workspace))) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdr_kv_compact_workspace_bytes(n_pages)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::PagesParams p = {};
    p.k_cache = static_cast<uint8_t*>(k_cache); p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.block_table = block_table; p.cache_len = cache_len; p.held = held; p.table_out = table_out; p.used = used;
    p.N_in = N; p.N = N; p.Hkv = Hkv; p.d = d; p.n_pages = n_pages; p.max_pages = max_pages;
    p.workspace = workspace;
    return from_hip(gdr::launch_kv_compact(p, (hipStream_t)stream));
}

size_t gdr_beam_select_workspace_bytes(int G, int K, int M, int V) {
    if (beam_args(G, K, M, V, V, -1, 0) != GDR_OK) return 0;
    return (size_t)G * K * gdr::beam_segments(G, K, V) * (8 * (size_t)M + 8);
}

gdr_status gdr_beam_select(const void* logits, const float* scores, const uint8_t* ended, int* tokens, int* rows,
                           float* scores_out, uint8_t* ended_out, int G, int K, int M, int V, long long stride,
                           int end_token, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    const gdr_status st = beam_args(G, K, M, V, stride, end_token, flags);
    if (st != GDR_OK) return st;
    if (ended && end_token < 0) return GDR_ERR_INVALID_ARG;
    const void* ptrs[] = {logits, scores, tokens, rows, scores_out, ended_out};
    for (const void* ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return GDR_ERR_INVALID_ARG;
    if ((ended && !aligned16(ended)) || (workspace && !aligned16(workspace))) return GDR_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdr_beam_select_workspace_bytes(G, K, M, V)) return GDR_ERR_WORKSPACE;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::BeamParams p;
    p.logits = logits; p.scores = scores; p.ended = ended;
    p.tokens = tokens; p.rows = rows; p.scores_out = scores_out; p.ended_out = ended_out;
    p.G = G; p.K = K; p.M = M; p.V = V; p.end_token = end_token; p.stride = stride; p.flags = flags;
    p.segs = gdr::beam_segments(G, K, V);
    p.best = static_cast<uint64_t*>(workspace);
    p.part = reinterpret_cast<float*>(p.best + (size_t)G * K * p.segs * M);
    return from_hip(gdr::launch_beam_select(p, (hipStream_t)stream));
}

gdr_status gdr_state_reorder(void* state, const int* parent, int layers, int N, int K, size_t row_bytes,
                             uint32_t flags, void* stream) {
    if (flags != 0 || layers < 1 || N < 1 || K < 1 || N % K != 0) return GDR_ERR_INVALID_ARG;
    if (row_bytes < 1 || row_bytes % 16 != 0 || row_bytes > ((size_t)1 << 40)) return GDR_ERR_INVALID_ARG;
    if ((long long)layers * N > (1LL << 28)) return GDR_ERR_INVALID_ARG;
    if (K > gdr::kMostBeams) return GDR_ERR_UNSUPPORTED;
    if (!grid_ok(gdr::state_reorder_workgroups(layers, N, K, (long long)row_bytes))) return GDR_ERR_INVALID_ARG;
    if (!state || !parent || !aligned16(state) || !aligned16(parent)) return GDR_ERR_INVALID_ARG;
    gdr_status ds = check_device();
    if (ds != GDR_OK) return ds;
    gdr::ReorderParams p;
    p.state = static_cast<uint8_t*>(state); p.parent = parent;
    p.layers = layers; p.N = N; p.K = K; p.row_bytes = (long long)row_bytes;
    return from_hip(gdr::launch_state_reorder(p, (hipStream_t)stream));
}

}  // extern "C"
