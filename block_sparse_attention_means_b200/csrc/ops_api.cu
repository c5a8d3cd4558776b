// C ABI of the operators before and beside the layer (rotary positions, the norm of
// queries and keys with the rotation, dense attention): argument checks and launches.
#include <cmath>

#include "dense.cuh"
#include "kernels.h"

namespace park {
namespace {

constexpr long long kMaxRows = 1ll << 31;  // tokens or rows of one call (int32 indices inside the kernels)

int check_head_dim(int D, int dtype) {
    if (dtype != PARK_BF16 && dtype != PARK_F32) return PARK_ERR_INVALID_ARG;
    if (D < 1) return PARK_ERR_INVALID_ARG;
    return D % 32 != 0 || D > 128 ? PARK_ERR_UNSUPPORTED : PARK_OK;
}

// Pointer alignment and strides of [B, H, N, D]; the elements of an output are distinct.
int check_operand(const park_operand* op, int B, long long N, int D, int elt, bool output) {
    if (!op || op->H < 1) return PARK_ERR_INVALID_ARG;
    if (op->H > 65535) return PARK_ERR_UNSUPPORTED;
    if (N == 0) return PARK_OK;
    if (!op->ptr || reinterpret_cast<uintptr_t>(op->ptr) % 16 != 0) return PARK_ERR_INVALID_ARG;
    long long ext[3] = {N, op->H, B}, str[3] = {op->sn, op->sh, op->sb};
    for (int i = 0; i < 3; ++i) {
        if (ext[i] == 1) continue;
        if (str[i] <= 0 || str[i] >= (1ll << 38) || str[i] * elt % 16 != 0) return PARK_ERR_INVALID_ARG;
    }
    if (!output) return PARK_OK;
    for (int i = 0; i < 3; ++i)  // by rising stride
        for (int j = i + 1; j < 3; ++j)
            if (str[j] < str[i]) {
                const long long s = str[i], e = ext[i];
                str[i] = str[j];
                ext[i] = ext[j];
                str[j] = s;
                ext[j] = e;
            }
    long long reach = D - 1;  // largest offset of the axes so far
    for (int i = 0; i < 3; ++i) {
        if (ext[i] == 1) continue;
        if (str[i] <= reach) return PARK_ERR_INVALID_ARG;
        reach += str[i] * (ext[i] - 1);
    }
    return PARK_OK;
}

int check_rope(const park_rope_axes* r, int D) {
    if (!r) return PARK_ERR_INVALID_ARG;
    long long pairs = 0;
    for (int a = 0; a < 3; ++a) {
        if (r->extent[a] < 1 || r->pairs[a] < 0) return PARK_ERR_INVALID_ARG;
        if (r->pairs[a] > 64 || r->extent[a] > (1 << 24)) return PARK_ERR_UNSUPPORTED;
        pairs += r->pairs[a];
    }
    if (D > 0 && pairs > D / 2) return PARK_ERR_INVALID_ARG;
    return PARK_OK;
}

int check_tokens(int B, long long N, const park_rope_axes* rope, const int32_t* pos, int64_t pos_sb, int D,
                 int32_t* status) {
    if (B < 1 || N < 0 || !status) return PARK_ERR_INVALID_ARG;
    if (N >= kMaxRows || B * N >= kMaxRows) return PARK_ERR_UNSUPPORTED;
    if (rope) {
        PARK_CHECK(check_rope(rope, D));
        if (!rope->table || reinterpret_cast<uintptr_t>(rope->table) % 8 != 0) return PARK_ERR_INVALID_ARG;
    }
    if (pos && (!rope || pos_sb < 0 || reinterpret_cast<uintptr_t>(pos) % 4 != 0)) return PARK_ERR_INVALID_ARG;
    return PARK_OK;
}

bool weights_ok(const void* w, int wdtype) {
    return (wdtype == PARK_BF16 || wdtype == PARK_F32) &&
           reinterpret_cast<uintptr_t>(w) % (wdtype == PARK_BF16 ? 2 : 4) == 0;
}

bool eps_ok(float eps) { return eps >= 0x1p-80f && std::isfinite(eps); }  // (the gradient forms 1 / eps)

int sm_count() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        n = 148;
    cudaGetLastError();
    return n > 0 ? n : 148;
}

// ------------------------------------------------------------------ dense attention
int check_attn(const park_attn_shape* s, int Hq, int Hk) {
    if (!s || s->B < 1 || s->Nq < 0 || s->Nk < 0 || s->n_seq < 0 || Hq < 1 || Hk < 1) return PARK_ERR_INVALID_ARG;
    PARK_CHECK(check_head_dim(s->D, s->dtype));
    if (Hq % Hk != 0 || !std::isfinite(s->scale) || !(s->scale > 0.f)) return PARK_ERR_INVALID_ARG;
    if (s->n_seq > 0 && (s->B != 1 || !s->cu_q || !s->cu_k)) return PARK_ERR_INVALID_ARG;
    if (Hq > 65535 || s->B > 65535 || s->n_seq > (1 << 24)) return PARK_ERR_UNSUPPORTED;
    // rows of a key head's group, tiles and coordinates are int32
    if (s->Nq >= kMaxRows || s->Nk >= kMaxRows) return PARK_ERR_UNSUPPORTED;  // (the products below stay in 64 bits)
    if (s->Nq * (Hq / Hk) >= kMaxRows - (1ll << 25) || s->Nk >= kMaxRows - (1ll << 25) ||
        (long long)s->B * Hq * (s->Nq / 8 + 1) >= kMaxRows || (long long)s->B * Hk * (s->Nk / 8 + 1) >= kMaxRows ||
        (long long)s->n_seq * Hq >= kMaxRows / 4)
        return PARK_ERR_UNSUPPORTED;
    return PARK_OK;
}

Op4 op4(const park_operand* o) {
    Op4 r{};
    if (o) r = Op4{static_cast<uint8_t*>(o->ptr), o->sb, o->sh, o->sn};
    return r;
}

DenseArgs dense_args(const park_attn_shape* s, const park_operand* q, const park_operand* k, const park_operand* v,
                     const park_operand* o, float* lse, int32_t* status) {
    DenseArgs a{};
    a.B = s->B;
    a.Hq = q->H;
    a.Hk = k->H;
    a.D = s->D;
    a.n_seq = s->n_seq;
    a.causal = s->causal != 0;
    a.Nq = s->Nq;
    a.Nk = s->Nk;
    a.cu_q = s->cu_q;
    a.cu_k = s->cu_k;
    a.scale = s->scale;
    a.q = op4(q);
    a.k = op4(k);
    a.v = op4(v);
    a.o = op4(o);
    a.lse = lse;
    a.status = status;
    return a;
}

size_t delta_bytes(const park_attn_shape* s, int Hq) { return align_up((size_t)s->B * Hq * (size_t)s->Nq * 4, 256); }

int attn_workspace(const park_attn_shape* s, int Hq, int Hk, int backward, size_t* bytes) {
    if (backward)
        *bytes = delta_bytes(s, Hq) +
                 dense_split_dkv(s->B, Hq, Hk, s->Nq, s->Nk, s->n_seq, s->D, s->dtype == PARK_BF16 ? 128 : 64).bytes;
    else
        *bytes = (s->dtype == PARK_BF16 ? dense_split_tc : dense_split_simt)(s->B, Hq, Hk, s->Nq, s->Nk, s->n_seq, s->D).bytes;
    return PARK_OK;
}

}  // namespace
}  // namespace park

using namespace park;

extern "C" {

size_t park_rope_table_floats(const park_rope_axes* rope) {
    if (check_rope(rope, 0) != PARK_OK) return 0;
    size_t n = 0;
    for (int a = 0; a < 3; ++a) n += (size_t)rope->extent[a] * rope->pairs[a];
    return 2 * n;
}

int park_rope_table(const park_rope_axes* rope, double theta, const double scale[3], void* stream) {
    PARK_CHECK(check_rope(rope, 0));
    if (!rope->table || reinterpret_cast<uintptr_t>(rope->table) % 8 != 0 || !scale) return PARK_ERR_INVALID_ARG;
    if (!(theta > 0.0) || !std::isfinite(theta)) return PARK_ERR_INVALID_ARG;
    for (int a = 0; a < 3; ++a)
        if (!std::isfinite(scale[a])) return PARK_ERR_INVALID_ARG;
    return launch_rope_table(rope, theta, scale, static_cast<cudaStream_t>(stream));
}

int park_rope(const park_operand* x, const park_operand* y, int B, int64_t N, int D, int dtype,
              const park_rope_axes* rope, const int32_t* positions, int64_t pos_sb, int inverse, int32_t* status,
              void* stream) {
    PARK_CHECK(check_head_dim(D, dtype));
    if (!rope) return PARK_ERR_INVALID_ARG;
    PARK_CHECK(check_tokens(B, N, rope, positions, pos_sb, D, status));
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    PARK_CHECK(check_operand(x, B, N, D, elt, false));
    PARK_CHECK(check_operand(y, B, N, D, elt, true));
    if (x->H != y->H) return PARK_ERR_INVALID_ARG;
    if (N == 0) return PARK_OK;
    return launch_rope(x, nullptr, y, nullptr, nullptr, nullptr, PARK_F32, 0.f, false, rope, positions, pos_sb,
                       inverse != 0, B, N, D, dtype, status, sm_count(), static_cast<cudaStream_t>(stream));
}

int park_qk_norm_rope(const park_operand* q, const park_operand* k, const void* wq, const void* wk, int wdtype,
                      float eps, const park_rope_axes* rope, const int32_t* positions, int64_t pos_sb,
                      const park_operand* q_out, const park_operand* k_out, int B, int64_t N, int D, int dtype,
                      int32_t* status, void* stream) {
    PARK_CHECK(check_head_dim(D, dtype));
    PARK_CHECK(check_tokens(B, N, rope, positions, pos_sb, D, status));
    if (!eps_ok(eps) || !weights_ok(wq, wdtype) || !weights_ok(wk, wdtype))
        return PARK_ERR_INVALID_ARG;
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    for (const park_operand* op : {q, k}) PARK_CHECK(check_operand(op, B, N, D, elt, false));
    for (const park_operand* op : {q_out, k_out}) PARK_CHECK(check_operand(op, B, N, D, elt, true));
    if (q->H != q_out->H || k->H != k_out->H) return PARK_ERR_INVALID_ARG;
    if (N == 0) return PARK_OK;
    return launch_rope(q, k, q_out, k_out, wq, wk, wdtype, eps, true, rope, positions, pos_sb, false, B, N, D, dtype,
                       status, sm_count(), static_cast<cudaStream_t>(stream));
}

int park_qk_norm_rope_bwd_workspace(int B, int64_t N, int D, size_t* bytes) {
    if (!bytes || B < 1 || N < 0) return PARK_ERR_INVALID_ARG;
    if (D < 1 || D % 32 != 0 || D > 128 || N >= kMaxRows || B * N >= kMaxRows) return PARK_ERR_UNSUPPORTED;
    *bytes = (size_t)norm_rope_bwd_blocks(B * N) * D * 4;
    return PARK_OK;
}

int park_qk_norm_rope_bwd(const park_operand* dq_out, const park_operand* dk_out, const park_operand* q,
                          const park_operand* k, const void* wq, const void* wk, int wdtype, float eps,
                          const park_rope_axes* rope, const int32_t* positions, int64_t pos_sb,
                          const park_operand* dq, const park_operand* dk, float* dwq, float* dwk, int B, int64_t N,
                          int D, int dtype, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
    PARK_CHECK(check_head_dim(D, dtype));
    PARK_CHECK(check_tokens(B, N, rope, positions, pos_sb, D, status));
    if (!eps_ok(eps) || !weights_ok(wq, wdtype) || !weights_ok(wk, wdtype))
        return PARK_ERR_INVALID_ARG;
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    for (const park_operand* op : {dq_out, dk_out, q, k}) PARK_CHECK(check_operand(op, B, N, D, elt, false));
    for (const park_operand* op : {dq, dk}) PARK_CHECK(check_operand(op, B, N, D, elt, true));
    if (q->H != dq->H || k->H != dk->H || q->H != dq_out->H || k->H != dk_out->H) return PARK_ERR_INVALID_ARG;
    size_t need = 0;
    PARK_CHECK(park_qk_norm_rope_bwd_workspace(B, N, D, &need));
    if (need > 0 && (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0)) return PARK_ERR_INVALID_ARG;
    if (ws_bytes < need) return PARK_ERR_WORKSPACE;
    return launch_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, wq, wk, wdtype, eps, rope, positions, pos_sb, dwq, dwk, B,
                                N, D, dtype, static_cast<float*>(ws), status, sm_count(),
                                static_cast<cudaStream_t>(stream));
}

int park_attention_workspace(const park_attn_shape* shape, int Hq, int Hk, int backward, size_t* bytes) {
    if (!bytes) return PARK_ERR_INVALID_ARG;
    PARK_CHECK(check_attn(shape, Hq, Hk));
    return attn_workspace(shape, Hq, Hk, backward, bytes);
}

int park_attention(const park_attn_shape* shape, const park_operand* q, const park_operand* k, const park_operand* v,
                   const park_operand* o, float* lse, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
    if (!q || !k || !v || !o || !status) return PARK_ERR_INVALID_ARG;
    PARK_CHECK(check_attn(shape, q->H, k->H));
    const park_attn_shape* s = shape;
    const int elt = s->dtype == PARK_BF16 ? 2 : 4;
    PARK_CHECK(check_operand(q, s->B, s->Nq, s->D, elt, false));
    PARK_CHECK(check_operand(k, s->B, s->Nk, s->D, elt, false));
    PARK_CHECK(check_operand(v, s->B, s->Nk, s->D, elt, false));
    PARK_CHECK(check_operand(o, s->B, s->Nq, s->D, elt, true));
    if (v->H != k->H || o->H != q->H) return PARK_ERR_INVALID_ARG;
    size_t need = 0;
    PARK_CHECK(attn_workspace(s, q->H, k->H, 0, &need));
    if (need > 0 && (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0)) return PARK_ERR_INVALID_ARG;
    if (ws_bytes < need) return PARK_ERR_WORKSPACE;
    if (s->Nq == 0) return PARK_OK;
    const DenseArgs a = dense_args(s, q, k, v, o, lse, status);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return s->dtype == PARK_BF16 ? launch_dense_fwd_tc(a, ws, st) : launch_dense_fwd_simt(a, ws, st);
}

int park_attention_bwd(const park_attn_shape* shape, const park_operand* d_o, const park_operand* q,
                       const park_operand* k, const park_operand* v, const park_operand* o, const float* lse,
                       const park_operand* dq, const park_operand* dk, const park_operand* dv, void* ws,
                       size_t ws_bytes, int32_t* status, void* stream) {
    if (!d_o || !q || !k || !v || !o || !dq || !dk || !dv || !status) return PARK_ERR_INVALID_ARG;
    PARK_CHECK(check_attn(shape, q->H, k->H));
    const park_attn_shape* s = shape;
    const int elt = s->dtype == PARK_BF16 ? 2 : 4;
    for (const park_operand* op : {d_o, q, o}) PARK_CHECK(check_operand(op, s->B, s->Nq, s->D, elt, false));
    for (const park_operand* op : {k, v}) PARK_CHECK(check_operand(op, s->B, s->Nk, s->D, elt, false));
    PARK_CHECK(check_operand(dq, s->B, s->Nq, s->D, elt, true));
    for (const park_operand* op : {dk, dv}) PARK_CHECK(check_operand(op, s->B, s->Nk, s->D, elt, true));
    if (v->H != k->H || dk->H != k->H || dv->H != k->H || o->H != q->H || d_o->H != q->H || dq->H != q->H ||
        (!lse && s->Nq > 0))
        return PARK_ERR_INVALID_ARG;
    size_t need = 0;
    PARK_CHECK(attn_workspace(s, q->H, k->H, 1, &need));
    if (need > 0 && (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0)) return PARK_ERR_INVALID_ARG;
    if (ws_bytes < need) return PARK_ERR_WORKSPACE;
    DenseArgs a = dense_args(s, q, k, v, o, const_cast<float*>(lse), status);
    a.d_o = op4(d_o);
    a.dq = op4(dq);
    a.dk = op4(dk);
    a.dv = op4(dv);
    float* delta = static_cast<float*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (s->Nq > 0) PARK_CHECK(launch_dense_delta(a, s->dtype, delta, st));
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + delta_bytes(s, q->H));
    return s->dtype == PARK_BF16 ? launch_dense_bwd_tc(a, delta, parts, st) : launch_dense_bwd_simt(a, delta, parts, st);
}

}  // extern "C"
