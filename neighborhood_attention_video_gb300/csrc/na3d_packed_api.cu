// C entry points of the packed-batch operators: the attention with shaped
// scores and the projection with adapters, forward and backward. Argument
// checks and launches; declared in include/na3d.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "na3d.h"
#include "na3d_host.cuh"
#include "na3d_lora.cuh"
#include "na3d_scored.cuh"

namespace {

using na3d::is_pow2;
using na3d::mul_ok;
using na3d::overlaps;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// `row` values every `stride` elements: bytes spanned, or an error. The strides
// of a TMA descriptor stay below 2^40 bytes: `grid` tokens of a batch entry.
int strided_span(int64_t tokens, int64_t grid, int64_t stride, int64_t row, int64_t* bytes) {
    if (stride < row) return NA3D_ERR_SHAPE;
    if (stride % 8 != 0) return NA3D_ERR_ALIGN;
    int64_t span;
    if (stride >= (int64_t(1) << 39) / grid || !mul_ok(tokens - 1, stride, &span) || !mul_ok(span + row, 2, bytes))
        return NA3D_ERR_OVERFLOW;
    return NA3D_OK;
}

// Do two written tensors of `tokens` rows of `row` values share an element?
// Views of one fused tensor (equal strides, disjoint columns) do not.
bool written_overlap(const void* a, int64_t a_bytes, int64_t a_ts, const void* b, int64_t b_bytes, int64_t b_ts,
                     int64_t row) {
    if (!overlaps(a, a_bytes, b, b_bytes)) return false;
    if (a_ts != b_ts) return true;
    const intptr_t d = (reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / 2;
    const int64_t off = ((d % a_ts) + a_ts) % a_ts;   // column of b's rows in a's
    return off < row || off > a_ts - row;
}

struct Span {
    const void* ptr;
    int64_t bytes;
};

// Checks that the calls of both directions share; *n = B*T*H*W tokens.
int check_scored(int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD, int64_t KT, int64_t KH,
                 int64_t KW, float softcap, const float* slopes, const int32_t* doc, const int32_t* prefix,
                 int64_t* n) {
    if (const int rc = na3d::validate_shape(B, T, H, W, NH, HD, KT, KH, KW)) return rc;
    // tanh(a / c) keeps its relative precision over this range of caps
    if (HD > 128 || !(softcap == 0.f || (softcap >= 0x1p-10f && softcap <= 0x1p20f))) return NA3D_ERR_UNSUPPORTED;
    *n = B * T * H * W;
    if (*n >= (int64_t(1) << 34) / NH) return NA3D_ERR_OVERFLOW;   // rows, 16 to a unit of work
    if (!aligned(slopes, 4) || !aligned(doc, 4) || !aligned(prefix, 4)) return NA3D_ERR_ALIGN;
    return NA3D_OK;
}

}  // namespace

extern "C" {

int na3d_scored_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int64_t B, int64_t T,
                    int64_t H, int64_t W, int64_t NH, int64_t HD, int64_t KT, int64_t KH, int64_t KW,
                    int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, float softcap,
                    const float* slopes, const int32_t* doc, const int32_t* prefix, void* stream) {
    int64_t n;
    if (const int rc = check_scored(B, T, H, W, NH, HD, KT, KH, KW, softcap, slopes, doc, prefix, &n)) return rc;
    if (!q || !k || !v || !out) return NA3D_ERR_NULL;
    const int64_t row = NH * HD, ts[3] = {q_token_stride, k_token_stride, v_token_stride};
    const void* in[3] = {q, k, v};
    int64_t bytes[3];
    for (int i = 0; i < 3; ++i)
        if (const int rc = strided_span(n, T * H * W, ts[i], row, &bytes[i])) return rc;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4))
        return NA3D_ERR_ALIGN;
    const Span written[2] = {{out, n * row * 2}, {lse, n * NH * 4}};
    const Span read[6] = {{in[0], bytes[0]}, {in[1], bytes[1]}, {in[2], bytes[2]},
                          {slopes, NH * 12}, {doc, n * 4}, {prefix, B * 4}};
    for (const Span& a : written)
        for (const Span& b : read)
            if (a.ptr && b.ptr && overlaps(a.ptr, a.bytes, b.ptr, b.bytes)) return NA3D_ERR_ALIAS;
    if (lse && overlaps(out, n * row * 2, lse, n * NH * 4)) return NA3D_ERR_ALIAS;

    na3d::ScoredParams p{};
    p.B = int32_t(B); p.T = int32_t(T); p.H = int32_t(H); p.W = int32_t(W); p.NH = int32_t(NH);
    p.KT = int32_t(KT); p.KH = int32_t(KH); p.KW = int32_t(KW);
    p.q_ts = ts[0]; p.k_ts = ts[1]; p.v_ts = ts[2];
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.softcap = softcap;
    p.slopes = slopes;
    p.doc = doc;
    p.prefix = prefix;
    if (!na3d::scored_planned(int(HD), p, false)) return NA3D_ERR_UNSUPPORTED;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;
    return na3d::launch_scored_fwd(int(HD), p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK
                                                                                                       : NA3D_ERR_CUDA;
}

int64_t na3d_scored_bwd_workspace(int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH) {
    int64_t n = 8;
    const int64_t dims[5] = {B, T, H, W, NH};
    for (const int64_t d : dims)
        if (d < 1 || !mul_ok(n, d, &n)) return -1;
    return n;
}

int na3d_scored_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout,
                    void* dq, void* dk, void* dv, void* work, int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH,
                    int64_t HD, int64_t KT, int64_t KH, int64_t KW, int64_t q_token_stride, int64_t k_token_stride,
                    int64_t v_token_stride, int64_t dq_token_stride, int64_t dk_token_stride,
                    int64_t dv_token_stride, float softcap, const float* slopes, const int32_t* doc,
                    const int32_t* prefix, void* stream) {
    int64_t n;
    if (const int rc = check_scored(B, T, H, W, NH, HD, KT, KH, KW, softcap, slopes, doc, prefix, &n)) return rc;
    const void* all[10] = {q, k, v, out, lse, dout, dq, dk, dv, work};
    for (const void* p : all)
        if (!p) return NA3D_ERR_NULL;
    const int64_t row = NH * HD;
    const int64_t ts[6] = {q_token_stride, k_token_stride, v_token_stride,
                           dq_token_stride, dk_token_stride, dv_token_stride};
    int64_t bytes[6];
    for (int i = 0; i < 6; ++i)
        if (const int rc = strided_span(n, T * H * W, ts[i], row, &bytes[i])) return rc;
    for (const void* p : all)
        if (!aligned(p, p == lse ? 4 : 16)) return NA3D_ERR_ALIGN;
    const void* const grads[3] = {dq, dk, dv};
    const Span written[4] = {{dq, bytes[3]}, {dk, bytes[4]}, {dv, bytes[5]}, {work, n * NH * 8}};
    const Span read[9] = {{q, bytes[0]}, {k, bytes[1]}, {v, bytes[2]}, {out, n * row * 2}, {dout, n * row * 2},
                          {lse, n * NH * 4}, {slopes, NH * 12}, {doc, n * 4}, {prefix, B * 4}};
    for (const Span& a : written)
        for (const Span& b : read)
            if (b.ptr && overlaps(a.ptr, a.bytes, b.ptr, b.bytes)) return NA3D_ERR_ALIAS;
    for (int i = 0; i < 3; ++i) {
        if (overlaps(work, n * NH * 8, grads[i], bytes[3 + i])) return NA3D_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (written_overlap(grads[i], bytes[3 + i], ts[3 + i], grads[j], bytes[3 + j], ts[3 + j], row))
                return NA3D_ERR_ALIAS;
    }

    na3d::ScoredParams p{};
    p.B = int32_t(B); p.T = int32_t(T); p.H = int32_t(H); p.W = int32_t(W); p.NH = int32_t(NH);
    p.KT = int32_t(KT); p.KH = int32_t(KH); p.KW = int32_t(KW);
    p.q_ts = ts[0]; p.k_ts = ts[1]; p.v_ts = ts[2];
    p.dq_ts = ts[3]; p.dk_ts = ts[4]; p.dv_ts = ts[5];
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<uint16_t*>(const_cast<void*>(out));
    p.lse = const_cast<float*>(lse);
    p.dout = static_cast<const uint16_t*>(dout);
    p.dq = static_cast<uint16_t*>(dq);
    p.dk = static_cast<uint16_t*>(dk);
    p.dv = static_cast<uint16_t*>(dv);
    p.stat = static_cast<float2*>(work);
    p.softcap = softcap;
    p.slopes = slopes;
    p.doc = doc;
    p.prefix = prefix;
    if (!na3d::scored_planned(int(HD), p, true)) return NA3D_ERR_UNSUPPORTED;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;
    return na3d::launch_scored_bwd(int(HD), p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK
                                                                                                       : NA3D_ERR_CUDA;
}

}  // extern "C"

namespace {

// Sizes of one projection call; *N = 3*NH*HD, work_bytes as the workspace call.
int check_lora_sizes(int64_t M, int64_t C, int64_t NH, int64_t HD, int64_t R, int64_t n_req, int64_t n_ad, bool backward,
                     int64_t* N, int64_t* work_bytes) {
    if (M < 1 || NH < 1 || C < 1 || HD < 1 || R < 1 || n_req < 1 || n_ad < 1) return NA3D_ERR_SHAPE;
    if (!is_pow2(HD) || HD < 16) return NA3D_ERR_HEAD_DIM;
    if (C % 8 != 0 || R % 8 != 0) return NA3D_ERR_ALIGN;   // 16-byte rows
    // A tile's roles walk its requests one by one, 0.3 us for each empty one; these must not add up
    // to the seconds that a wait allows.
    if (R > 128 || n_req - M > int64_t(1) << 20) return NA3D_ERR_UNSUPPORTED;
    const int64_t lim = int64_t(1) << 31;
    int64_t b;
    if (!mul_ok(3 * NH, HD, N) || *N >= lim || M >= lim - 256 || C >= lim ||
        n_req >= lim / 128 - (M + 127) / 128 || n_ad >= lim / *N || n_ad >= lim / 128 ||
        !mul_ok(M, *N, &b) || !mul_ok(b, 2, &b) || !mul_ok(M, C, &b) || !mul_ok(b, 2, &b) ||
        !mul_ok(n_ad * 128, *N + C, &b) || !mul_ok(b, 8, &b))   // adapters, and the workspace's sums of them
        return NA3D_ERR_OVERFLOW;
    *work_bytes = na3d::lora_workspace(M, C, *N, R, n_req, n_ad, backward);
    return NA3D_OK;
}

int check_lora_buffers(const Span* written, int n_written, const Span* read, int n_read) {
    for (int i = 0; i < n_written; ++i) {
        if (!written[i].ptr) continue;
        if (!aligned(written[i].ptr, 16)) return NA3D_ERR_ALIGN;
        for (int j = 0; j < i; ++j)
            if (written[j].ptr && overlaps(written[i].ptr, written[i].bytes, written[j].ptr, written[j].bytes))
                return NA3D_ERR_ALIAS;
        for (int j = 0; j < n_read; ++j)
            if (read[j].ptr && overlaps(written[i].ptr, written[i].bytes, read[j].ptr, read[j].bytes))
                return NA3D_ERR_ALIAS;
    }
    return NA3D_OK;
}

}  // namespace

extern "C" {

int64_t na3d_lora_workspace(int64_t M, int64_t C, int64_t NH, int64_t HD, int64_t R, int64_t n_requests,
                            int64_t n_adapters, int backward) {
    int64_t N, bytes;
    return check_lora_sizes(M, C, NH, HD, R, n_requests, n_adapters, backward != 0, &N, &bytes) == NA3D_OK ? bytes : -1;
}

int na3d_lora_qkv_proj(const void* x, const void* w, const void* bias, const void* lora_a, const void* lora_b,
                       const float* scaling, const int32_t* offsets, const int32_t* adapter, void* qkv, void* work,
                       int64_t M, int64_t C, int64_t NH, int64_t HD, int64_t R, int64_t n_requests,
                       int64_t n_adapters, void* stream) {
    int64_t N, work_bytes;
    if (const int rc = check_lora_sizes(M, C, NH, HD, R, n_requests, n_adapters, false, &N, &work_bytes)) return rc;
    if (!x || !w || !lora_a || !lora_b || !scaling || !offsets || !adapter || !qkv || !work) return NA3D_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(bias, 2) ||
        !aligned(scaling, 4) || !aligned(offsets, 4) || !aligned(adapter, 4))
        return NA3D_ERR_ALIGN;
    const Span written[2] = {{qkv, M * N * 2}, {work, work_bytes}};
    const Span read[8] = {{x, M * C * 2}, {w, N * C * 2}, {bias, N * 2}, {lora_a, n_adapters * R * C * 2},
                          {lora_b, n_adapters * N * R * 2}, {scaling, n_adapters * 4},
                          {offsets, (n_requests + 1) * 4}, {adapter, n_requests * 4}};
    if (const int rc = check_lora_buffers(written, 2, read, 8)) return rc;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;

    na3d::LoraParams p{};
    p.M = int32_t(M); p.C = int32_t(C); p.N = int32_t(N); p.Nq = int32_t(NH * HD);
    p.R = int32_t(R); p.n_req = int32_t(n_requests); p.n_ad = int32_t(n_adapters);
    p.q_scale = float(1.0 / __builtin_sqrt(double(HD)));
    p.x = static_cast<const uint16_t*>(x);
    p.w = static_cast<const uint16_t*>(w);
    p.bias = static_cast<const uint16_t*>(bias);
    p.a = static_cast<const uint16_t*>(lora_a);
    p.b = static_cast<const uint16_t*>(lora_b);
    p.scaling = scaling;
    p.offsets = offsets;
    p.adapter = adapter;
    p.qkv = static_cast<uint16_t*>(qkv);
    p.work = work;
    return na3d::launch_lora_fwd(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

int na3d_lora_qkv_proj_bwd(const void* dqkv, const void* x, const void* w, const void* lora_a, const void* lora_b,
                           const float* scaling, const int32_t* offsets, const int32_t* adapter, void* dx,
                           void* dlora_a, void* dlora_b, void* work, int64_t M, int64_t C, int64_t NH, int64_t HD,
                           int64_t R, int64_t n_requests, int64_t n_adapters, void* stream) {
    int64_t N, work_bytes;
    if (const int rc = check_lora_sizes(M, C, NH, HD, R, n_requests, n_adapters, true, &N, &work_bytes)) return rc;
    if (!dqkv || !x || !w || !lora_a || !lora_b || !scaling || !offsets || !adapter || !dlora_a || !dlora_b || !work)
        return NA3D_ERR_NULL;
    if (!aligned(dqkv, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) ||
        !aligned(scaling, 4) || !aligned(offsets, 4) || !aligned(adapter, 4))
        return NA3D_ERR_ALIGN;
    const Span written[4] = {{dx, M * C * 2}, {dlora_a, n_adapters * R * C * 2}, {dlora_b, n_adapters * N * R * 2},
                             {work, work_bytes}};
    const Span read[8] = {{dqkv, M * N * 2}, {x, M * C * 2}, {w, N * C * 2}, {lora_a, n_adapters * R * C * 2},
                          {lora_b, n_adapters * N * R * 2}, {scaling, n_adapters * 4},
                          {offsets, (n_requests + 1) * 4}, {adapter, n_requests * 4}};
    if (const int rc = check_lora_buffers(written, 4, read, 8)) return rc;
    int sms;
    if (const int rc = na3d::current_device(&sms)) return rc;

    na3d::LoraParams p{};
    p.M = int32_t(M); p.C = int32_t(C); p.N = int32_t(N); p.Nq = int32_t(NH * HD);
    p.R = int32_t(R); p.n_req = int32_t(n_requests); p.n_ad = int32_t(n_adapters);
    p.q_scale = float(1.0 / __builtin_sqrt(double(HD)));
    p.dqkv = static_cast<const uint16_t*>(dqkv);
    p.x = static_cast<const uint16_t*>(x);
    p.w = static_cast<const uint16_t*>(w);
    p.a = static_cast<const uint16_t*>(lora_a);
    p.b = static_cast<const uint16_t*>(lora_b);
    p.scaling = scaling;
    p.offsets = offsets;
    p.adapter = adapter;
    p.dx = static_cast<uint16_t*>(dx);
    p.da = static_cast<uint16_t*>(dlora_a);
    p.db = static_cast<uint16_t*>(dlora_b);
    p.work = work;
    return na3d::launch_lora_bwd(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NA3D_OK : NA3D_ERR_CUDA;
}

}  // extern "C"
