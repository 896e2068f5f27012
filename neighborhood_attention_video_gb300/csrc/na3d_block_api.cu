// C entry points of the norm and rotation of queries and keys and of the
// attention to states of another length, forward and backward. Argument checks
// and launches; declared in include/na3d.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "na3d.h"
#include "na3d_cross.cuh"
#include "na3d_host.cuh"
#include "na3d_rope.cuh"

namespace {

using na3d::aligned;
using na3d::is_pow2;
using na3d::mul_ok;
using na3d::overlaps;
using na3d::Span;
using na3d::strided_span;

// Tokens of `row` values, `ts` elements apart.
struct Rows {
    const void* ptr;
    int64_t bytes, ts, row;
};

// Do two tensors of as many tokens share an element? Blocks of one fused tensor
// (equal strides, columns of their own) do not.
bool share(const Rows& a, const Rows& b) {
    if (!a.ptr || !b.ptr || !overlaps(a.ptr, a.bytes, b.ptr, b.bytes)) return false;
    if (a.ts != b.ts) return true;
    const intptr_t d = (reinterpret_cast<intptr_t>(b.ptr) - reinterpret_cast<intptr_t>(a.ptr)) / 2;
    const int64_t off = ((d % a.ts) + a.ts) % a.ts;   // column of b's rows in a's
    return off < a.row || off + b.row > a.ts;
}

bool same(const Rows& a, const Rows& b) { return a.ptr == b.ptr && a.ts == b.ts && a.row == b.row; }

bool share(const Rows& a, const Span& b) { return a.ptr && b.ptr && overlaps(a.ptr, a.bytes, b.ptr, b.bytes); }

constexpr int64_t kLimit = int64_t(1) << 31;

// ------------------------------------------------------------------ norm and rotation

struct RopeSizes {
    int64_t B, T, H, W, NH, NKV, HD, RT, RH, RW;
    int64_t tokens, table_bytes;
};

int check_rope(RopeSizes* z, const float* table, int norm, float q_eps, float k_eps, float q_scale, int interleaved,
               const void* q_weight, const void* k_weight) {
    if (z->B < 1 || z->T < 1 || z->H < 1 || z->W < 1 || z->NH < 1 || z->NKV < 0 || z->HD < 1 || z->RT < 0 || z->RH < 0 || z->RW < 0)
        return NA3D_ERR_SHAPE;
    if (!is_pow2(z->HD) || z->HD < 16) return NA3D_ERR_HEAD_DIM;
    const int64_t lim = z->HD;
    if (z->RT > lim || z->RH > lim || z->RW > lim || z->RT + z->RH + z->RW > lim || (z->RT | z->RH | z->RW) & 1)
        return NA3D_ERR_SHAPE;
    if (z->HD > 512 || (!interleaved && (z->RT + z->RH + z->RW) % 16 != 0)) return NA3D_ERR_UNSUPPORTED;
    if (!(std::isfinite(q_scale)) || (norm && !(q_eps > 0.f && std::isfinite(q_eps))) ||
        (norm && z->NKV && !(k_eps > 0.f && std::isfinite(k_eps))) || (!norm && (q_weight || k_weight)))
        return NA3D_ERR_UNSUPPORTED;
    int64_t n;
    if (!mul_ok(z->B, z->T, &n) || !mul_ok(n, z->H, &n) || !mul_ok(n, z->W, &n) || n >= kLimit ||
        z->NH >= kLimit / z->HD || z->NKV >= kLimit / z->HD)
        return NA3D_ERR_OVERFLOW;
    z->tokens = n;
    z->table_bytes = (z->T * z->RT + z->H * z->RH + z->W * z->RW) * 4;
    if (z->table_bytes >= kLimit) return NA3D_ERR_OVERFLOW;
    if (z->table_bytes && !table) return NA3D_ERR_NULL;
    if (!aligned(table, 8) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return NA3D_ERR_ALIGN;
    return NA3D_OK;
}

int rows_of(const RopeSizes& z, const void* ptr, int64_t ts, int64_t heads, Rows* r) {
    *r = {nullptr, 0, 1, 0};
    if (heads == 0) return NA3D_OK;
    if (!ptr) return NA3D_ERR_NULL;
    if (!aligned(ptr, 16)) return NA3D_ERR_ALIGN;
    *r = {ptr, 0, ts, heads * z.HD};
    return strided_span(z.tokens, 1, ts, r->row, &r->bytes);
}

na3d::RopeParams rope_params(const RopeSizes& z, const float* table, int norm, int interleaved) {
    na3d::RopeParams p{};
    p.table = reinterpret_cast<const float2*>(table);
    p.tokens = z.tokens;
    p.T = int32_t(z.T); p.H = int32_t(z.H); p.W = int32_t(z.W);
    p.PT = int32_t(z.RT / 2); p.PH = int32_t(z.RH / 2); p.PW = int32_t(z.RW / 2);
    p.norm = norm != 0;
    p.interleaved = interleaved != 0;
    return p;
}

}  // namespace

extern "C" {

int na3d_rope_table(float* table, int64_t T, int64_t H, int64_t W, int64_t RT, int64_t RH, int64_t RW, double theta,
                    double t_offset, double h_offset, double w_offset, double t_scale, double h_scale, double w_scale,
                    void* stream) {
    const int64_t n[3] = {T, H, W}, r[3] = {RT, RH, RW};
    const double offset[3] = {t_offset, h_offset, w_offset}, scale[3] = {t_scale, h_scale, w_scale};
    int64_t total = 0;
    for (int a = 0; a < 3; ++a) {
        if (n[a] < 1 || r[a] < 0 || r[a] & 1) return NA3D_ERR_SHAPE;
        int64_t m;
        if (n[a] >= kLimit || r[a] >= kLimit || !mul_ok(n[a], r[a], &m)) return NA3D_ERR_OVERFLOW;
        total += m;
        if (!std::isfinite(offset[a]) || !std::isfinite(scale[a])) return NA3D_ERR_UNSUPPORTED;
    }
    if (total == 0) return NA3D_ERR_SHAPE;
    if (total >= kLimit / 4) return NA3D_ERR_OVERFLOW;
    if (!(theta > 0) || !std::isfinite(theta)) return NA3D_ERR_UNSUPPORTED;
    if (!table) return NA3D_ERR_NULL;
    if (!aligned(table, 8)) return NA3D_ERR_ALIGN;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;
    na3d::RopeTable p{};
    p.table = reinterpret_cast<float2*>(table);
    p.theta = theta;
    for (int a = 0; a < 3; ++a) {
        p.n[a] = int32_t(n[a]);
        p.pairs[a] = int32_t(r[a] / 2);
        p.offset[a] = offset[a];
        p.scale[a] = scale[a];
    }
    return na3d::launch_rope_table(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

int na3d_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight, const void* k_weight,
                   const float* table, int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t NKV, int64_t HD,
                   int64_t RT, int64_t RH, int64_t RW, int64_t q_token_stride, int64_t k_token_stride,
                   int64_t q_out_token_stride, int64_t k_out_token_stride, int norm, float q_eps, float k_eps,
                   float q_scale, int interleaved, void* stream) {
    RopeSizes z{B, T, H, W, NH, NKV, HD, RT, RH, RW, 0, 0};
    if (const int rc = check_rope(&z, table, norm, q_eps, k_eps, q_scale, interleaved, q_weight, k_weight)) return rc;
    Rows in[2], out[2];
    int rc;
    if ((rc = rows_of(z, q, q_token_stride, NH, &in[0])) || (rc = rows_of(z, k, k_token_stride, NKV, &in[1])) ||
        (rc = rows_of(z, q_out, q_out_token_stride, NH, &out[0])) || (rc = rows_of(z, k_out, k_out_token_stride, NKV, &out[1])))
        return rc;
    const Span small[3] = {{q_weight, HD * 2}, {k_weight, HD * 2}, {table, z.table_bytes}};
    for (int i = 0; i < 2; ++i) {
        if (share(out[i], in[1 - i]) || (share(out[i], in[i]) && !same(out[i], in[i]))) return NA3D_ERR_ALIAS;
        for (const Span& s : small)
            if (share(out[i], s)) return NA3D_ERR_ALIAS;
    }
    if (share(out[0], out[1])) return NA3D_ERR_ALIAS;
    int sms;
    if ((rc = na3d::current_device(&sms))) return rc;
    na3d::RopeParams p = rope_params(z, table, norm, interleaved);
    p.side[0] = {static_cast<const uint16_t*>(q), nullptr, static_cast<uint16_t*>(q_out), static_cast<const uint16_t*>(q_weight),
                 nullptr, q_token_stride, 0, q_out_token_stride, int32_t(NH), q_eps, q_scale};
    p.side[1] = {static_cast<const uint16_t*>(k), nullptr, static_cast<uint16_t*>(k_out), static_cast<const uint16_t*>(k_weight),
                 nullptr, k_token_stride, 0, k_out_token_stride, int32_t(NKV), k_eps, 1.f};
    return na3d::launch_rope(int(HD), p, false, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

int64_t na3d_norm_rope_workspace(int64_t HD) {
    return is_pow2(HD) && HD >= 16 && HD <= 512 ? na3d::rope_workspace(HD) : -1;
}

int na3d_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                       float* dq_weight, float* dk_weight, const void* q_weight, const void* k_weight,
                       const float* table, void* work, int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH,
                       int64_t NKV, int64_t HD, int64_t RT, int64_t RH, int64_t RW, int64_t q_token_stride,
                       int64_t k_token_stride, int64_t dq_out_token_stride, int64_t dk_out_token_stride,
                       int64_t dq_token_stride, int64_t dk_token_stride, int norm, float q_eps, float k_eps,
                       float q_scale, int interleaved, void* stream) {
    RopeSizes z{B, T, H, W, NH, NKV, HD, RT, RH, RW, 0, 0};
    if (const int rc = check_rope(&z, table, norm, q_eps, k_eps, q_scale, interleaved, q_weight, k_weight)) return rc;
    // gradients of weights: of the norm's, of tensors that are there
    if ((dq_weight || dk_weight) && (!norm || (dk_weight && !NKV))) return NA3D_ERR_UNSUPPORTED;
    Rows x[2], g[2], out[2];
    int rc;
    if ((rc = rows_of(z, q, q_token_stride, NH, &x[0])) || (rc = rows_of(z, k, k_token_stride, NKV, &x[1])) ||
        (rc = rows_of(z, dq_out, dq_out_token_stride, NH, &g[0])) || (rc = rows_of(z, dk_out, dk_out_token_stride, NKV, &g[1])) ||
        (rc = rows_of(z, dq, dq_token_stride, NH, &out[0])) || (rc = rows_of(z, dk, dk_token_stride, NKV, &out[1])))
        return rc;
    const bool weights = dq_weight || dk_weight;
    if (weights && !work) return NA3D_ERR_NULL;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || (weights && !aligned(work, 16))) return NA3D_ERR_ALIGN;
    const Span small[3] = {{q_weight, HD * 2}, {k_weight, HD * 2}, {table, z.table_bytes}};
    const Span sums[3] = {{dq_weight, HD * 4}, {dk_weight, HD * 4}, {weights ? work : nullptr, na3d::rope_workspace(HD)}};
    for (int i = 0; i < 2; ++i) {
        // the gradient may take the place of the one that it is computed from, or of x
        if (share(out[i], x[1 - i]) || share(out[i], g[1 - i]) || (share(out[i], x[i]) && !same(out[i], x[i])) ||
            (share(out[i], g[i]) && !same(out[i], g[i])))
            return NA3D_ERR_ALIAS;
        for (const Span& s : small)
            if (share(out[i], s)) return NA3D_ERR_ALIAS;
        for (const Span& s : sums)
            if (share(out[i], s) || share(x[i], s) || share(g[i], s)) return NA3D_ERR_ALIAS;
    }
    if (share(out[0], out[1])) return NA3D_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j)
            if (sums[i].ptr && ((small[j].ptr && overlaps(sums[i].ptr, sums[i].bytes, small[j].ptr, small[j].bytes)) ||
                                (j < i && sums[j].ptr && overlaps(sums[i].ptr, sums[i].bytes, sums[j].ptr, sums[j].bytes))))
                return NA3D_ERR_ALIAS;
    int sms;
    if ((rc = na3d::current_device(&sms))) return rc;
    na3d::RopeParams p = rope_params(z, table, norm, interleaved);
    p.work = weights ? static_cast<float*>(work) : nullptr;
    p.side[0] = {static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(dq_out), static_cast<uint16_t*>(dq),
                 static_cast<const uint16_t*>(q_weight), dq_weight, q_token_stride, dq_out_token_stride, dq_token_stride,
                 int32_t(NH), q_eps, q_scale};
    p.side[1] = {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(dk_out), static_cast<uint16_t*>(dk),
                 static_cast<const uint16_t*>(k_weight), dk_weight, k_token_stride, dk_out_token_stride, dk_token_stride,
                 int32_t(NKV), k_eps, 1.f};
    return na3d::launch_rope(int(HD), p, true, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ attention to other states

namespace {

int check_cross(int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD) {
    if (B < 1 || L < 1 || S < 1 || NH < 1 || NKV < 1 || HD < 1 || NH % NKV != 0) return NA3D_ERR_SHAPE;
    if (!is_pow2(HD) || HD < 16) return NA3D_ERR_HEAD_DIM;
    if (HD > 128 || NH / NKV > 64) return NA3D_ERR_UNSUPPORTED;
    int64_t n;
    if (B >= kLimit || L >= kLimit - 256 || S >= kLimit - 256 || NH >= kLimit / HD || !mul_ok(B * NH, L, &n) ||
        n >= (int64_t(1) << 37) || !mul_ok(B * NKV, S, &n) || n >= (int64_t(1) << 37))
        return NA3D_ERR_OVERFLOW;
    return NA3D_OK;
}

// Checks that both directions share, for the tensors that both have.
int check_cross_inputs(const Rows* in, const int32_t* doc, const int32_t* kv_doc) {
    for (int i = 0; i < 3; ++i)
        if (!aligned(in[i].ptr, 16)) return NA3D_ERR_ALIGN;
    return aligned(doc, 4) && aligned(kv_doc, 4) ? NA3D_OK : NA3D_ERR_ALIGN;
}

na3d::CrossParams cross_params(const Rows* in, int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV,
                               const int32_t* doc, const int32_t* kv_doc, void* work) {
    na3d::CrossParams p{};
    p.B = int32_t(B); p.L = int32_t(L); p.S = int32_t(S); p.NH = int32_t(NH); p.NKV = int32_t(NKV);
    p.q_ts = in[0].ts; p.k_ts = in[1].ts; p.v_ts = in[2].ts;
    p.q = static_cast<const uint16_t*>(in[0].ptr);
    p.k = static_cast<const uint16_t*>(in[1].ptr);
    p.v = static_cast<const uint16_t*>(in[2].ptr);
    p.doc = doc;
    p.kv_doc = kv_doc;
    p.work = work;
    return p;
}

int cross_fwd(const void* q, const void* k, const void* v, void* out, float* lse, void* work, int64_t B, int64_t L,
              int64_t S, int64_t NH, int64_t NKV, int64_t HD, int64_t q_token_stride, int64_t k_token_stride,
              int64_t v_token_stride, const int32_t* doc, const int32_t* kv_doc, void* stream, bool withhold) {
    if (const int rc = check_cross(B, L, S, NH, NKV, HD)) return rc;
    const int64_t need = na3d::cross_workspace(B, L, S, NH, NKV, HD, false);
    if (!q || !k || !v || !out || (need && !work)) return NA3D_ERR_NULL;
    Rows in[3] = {{q, 0, q_token_stride, NH * HD}, {k, 0, k_token_stride, NKV * HD}, {v, 0, v_token_stride, NKV * HD}};
    for (int i = 0; i < 3; ++i)
        if (const int rc = strided_span(B * (i ? S : L), i ? S : L, in[i].ts, in[i].row, &in[i].bytes)) return rc;
    if (const int rc = check_cross_inputs(in, doc, kv_doc)) return rc;
    if (!aligned(out, 16) || !aligned(lse, 4) || (need && !aligned(work, 16))) return NA3D_ERR_ALIGN;
    const int64_t rows = B * L * NH;
    const Span written[3] = {{out, rows * HD * 2}, {lse, rows * 4}, {need ? work : nullptr, need}};
    const Span masks[2] = {{doc, B * L * 4}, {kv_doc, B * S * 4}};
    for (int i = 0; i < 3; ++i) {
        if (!written[i].ptr) continue;
        for (const Rows& r : in)
            if (share(r, written[i])) return NA3D_ERR_ALIAS;
        for (const Span& m : masks)
            if (m.ptr && overlaps(written[i].ptr, written[i].bytes, m.ptr, m.bytes)) return NA3D_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (written[j].ptr && overlaps(written[i].ptr, written[i].bytes, written[j].ptr, written[j].bytes))
                return NA3D_ERR_ALIAS;
    }
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;
    na3d::CrossParams p = cross_params(in, B, L, S, NH, NKV, doc, kv_doc, work);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.withhold = withhold;
    return na3d::launch_cross_fwd(int(HD), p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

int cross_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout, void* dq,
              void* dk, void* dv, void* work, int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD,
              int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int64_t dq_token_stride,
              int64_t dk_token_stride, int64_t dv_token_stride, const int32_t* doc, const int32_t* kv_doc, void* stream,
              bool withhold) {
    if (const int rc = check_cross(B, L, S, NH, NKV, HD)) return rc;
    const void* const all[10] = {q, k, v, out, lse, dout, dq, dk, dv, work};
    for (const void* p : all)
        if (!p) return NA3D_ERR_NULL;
    const int64_t rows = B * L * NH, need = na3d::cross_workspace(B, L, S, NH, NKV, HD, true);
    Rows in[3] = {{q, 0, q_token_stride, NH * HD}, {k, 0, k_token_stride, NKV * HD}, {v, 0, v_token_stride, NKV * HD}};
    Rows grad[3] = {{dq, 0, dq_token_stride, NH * HD}, {dk, 0, dk_token_stride, NKV * HD}, {dv, 0, dv_token_stride, NKV * HD}};
    for (int i = 0; i < 3; ++i)
        for (Rows* r : {&in[i], &grad[i]})
            if (const int rc = strided_span(B * (i ? S : L), i ? S : L, r->ts, r->row, &r->bytes)) return rc;
    if (const int rc = check_cross_inputs(in, doc, kv_doc)) return rc;
    if (const int rc = check_cross_inputs(grad, nullptr, nullptr)) return rc;
    if (!aligned(out, 16) || !aligned(dout, 16) || !aligned(work, 16) || !aligned(lse, 4)) return NA3D_ERR_ALIGN;
    const Span read[5] = {{out, rows * HD * 2}, {dout, rows * HD * 2}, {lse, rows * 4}, {doc, B * L * 4}, {kv_doc, B * S * 4}};
    const Span kept{work, need};
    for (int i = 0; i < 3; ++i) {
        if (share(grad[i], kept) || share(in[i], kept)) return NA3D_ERR_ALIAS;
        // only dk and dv are of as many tokens, and may be blocks of one tensor
        for (int j = 0; j < 3; ++j)
            if (overlaps(grad[i].ptr, grad[i].bytes, in[j].ptr, in[j].bytes)) return NA3D_ERR_ALIAS;
        for (const Span& s : read)
            if (share(grad[i], s)) return NA3D_ERR_ALIAS;
    }
    for (const Span& s : read)
        if (s.ptr && overlaps(s.ptr, s.bytes, work, need)) return NA3D_ERR_ALIAS;
    if (overlaps(dq, grad[0].bytes, dk, grad[1].bytes) || overlaps(dq, grad[0].bytes, dv, grad[2].bytes) || share(grad[1], grad[2]))
        return NA3D_ERR_ALIAS;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;
    na3d::CrossParams p = cross_params(in, B, L, S, NH, NKV, doc, kv_doc, work);
    p.dq_ts = dq_token_stride; p.dk_ts = dk_token_stride; p.dv_ts = dv_token_stride;
    p.out = static_cast<uint16_t*>(const_cast<void*>(out));
    p.lse = const_cast<float*>(lse);
    p.dout = static_cast<const uint16_t*>(dout);
    p.dq = static_cast<uint16_t*>(dq);
    p.dk = static_cast<uint16_t*>(dk);
    p.dv = static_cast<uint16_t*>(dv);
    p.withhold = withhold;
    return na3d::launch_cross_bwd(int(HD), p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t na3d_cross_workspace(int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD, int backward) {
    return check_cross(B, L, S, NH, NKV, HD) == NA3D_OK ? na3d::cross_workspace(B, L, S, NH, NKV, HD, backward != 0) : -1;
}

int na3d_cross_fwd(const void* q, const void* k, const void* v, void* out, float* lse, void* work, int64_t B,
                   int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD, int64_t q_token_stride,
                   int64_t k_token_stride, int64_t v_token_stride, const int32_t* doc, const int32_t* kv_doc,
                   void* stream) {
    return cross_fwd(q, k, v, out, lse, work, B, L, S, NH, NKV, HD, q_token_stride, k_token_stride, v_token_stride, doc, kv_doc,
                     stream, false);
}

int na3d_cross_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout,
                   void* dq, void* dk, void* dv, void* work, int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV,
                   int64_t HD, int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                   int64_t dq_token_stride, int64_t dk_token_stride, int64_t dv_token_stride, const int32_t* doc,
                   const int32_t* kv_doc, void* stream) {
    return cross_bwd(q, k, v, out, lse, dout, dq, dk, dv, work, B, L, S, NH, NKV, HD, q_token_stride, k_token_stride,
                     v_token_stride, dq_token_stride, dk_token_stride, dv_token_stride, doc, kv_doc, stream, false);
}

int na3d_cross_selftest_withhold(const void* q, const void* k, const void* v, void* out, float* lse, const void* dout,
                                 void* dq, void* dk, void* dv, void* work, int64_t B, int64_t L, int64_t S, int64_t NH,
                                 int64_t NKV, int64_t HD, const int32_t* doc, const int32_t* kv_doc, void* stream) {
    if (!dout)
        return cross_fwd(q, k, v, out, lse, work, B, L, S, NH, NKV, HD, NH * HD, NKV * HD, NKV * HD, doc, kv_doc, stream, true);
    return cross_bwd(q, k, v, out, lse, dout, dq, dk, dv, work, B, L, S, NH, NKV, HD, NH * HD, NKV * HD, NKV * HD, NH * HD,
                     NKV * HD, NKV * HD, doc, kv_doc, stream, true);
}

}  // extern "C"
