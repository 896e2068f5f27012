// Host helpers that the C entry points share: argument checks, the current
// device's properties and 2-D TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "na3d.h"

namespace na3d {

// ------------------------------------------------------------------ validation

inline bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

inline int validate_shape(int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD, int64_t KT,
                   int64_t KH, int64_t KW) {
    if (B < 1 || NH < 1 || T < 1 || H < 1 || W < 1 || HD < 1) return NA3D_ERR_SHAPE;
    const int64_t ks[3] = {KT, KH, KW}, ns[3] = {T, H, W};
    for (int a = 0; a < 3; ++a)
        if (ks[a] < 1 || (ks[a] & 1) == 0 || ks[a] > ns[a]) return NA3D_ERR_KERNEL;
    if (!is_pow2(HD) || HD < 16) return NA3D_ERR_HEAD_DIM;
    // element count and byte size of one tensor must fit int64; TMA limits:
    // every global dimension < 2^32, every stride < 2^40 bytes.
    int64_t n = 1;
    const int64_t dims[6] = {B, T, H, W, NH, HD};
    for (int i = 0; i < 6; ++i)
        if (!mul_ok(n, dims[i], &n)) return NA3D_ERR_OVERFLOW;
    if (!mul_ok(n, 2, &n)) return NA3D_ERR_OVERFLOW;
    // a head's column offset is a signed 32-bit TMA coordinate
    if (NH * HD >= (int64_t(1) << 31) || W >= (int64_t(1) << 31) || H >= (int64_t(1) << 31) ||
        T >= (int64_t(1) << 31) || B >= (int64_t(1) << 31))
        return NA3D_ERR_OVERFLOW;
    if (n / dims[0] >= (int64_t(1) << 40)) return NA3D_ERR_OVERFLOW;  // batch stride in bytes
    return NA3D_OK;
}

// Do the byte ranges [a, a + a_bytes) and [b, b + b_bytes) intersect?
inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + uintptr_t(b_bytes) && y < x + uintptr_t(a_bytes);
}

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// `row` values every `stride` elements: bytes spanned, or an error. The strides
// of a TMA descriptor stay below 2^40 bytes: `grid` tokens of a batch entry.
inline int strided_span(int64_t tokens, int64_t grid, int64_t stride, int64_t row, int64_t* bytes) {
    if (stride < row) return NA3D_ERR_SHAPE;
    if (stride % 8 != 0) return NA3D_ERR_ALIGN;
    int64_t span;
    if (stride >= (int64_t(1) << 39) / grid || !mul_ok(tokens - 1, stride, &span) || !mul_ok(span + row, 2, bytes))
        return NA3D_ERR_OVERFLOW;
    return NA3D_OK;
}

// Do two written tensors of `tokens` rows of `row` values share an element?
// Views of one fused tensor (equal strides, disjoint columns) do not.
inline bool written_overlap(const void* a, int64_t a_bytes, int64_t a_ts, const void* b, int64_t b_bytes, int64_t b_ts,
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

// NA3D_OK where the current device is a GB300, with its number of SMs.
inline int current_device(int* sms) {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return NA3D_ERR_CUDA;
    return major == 10 && minor == 3 ? NA3D_OK : NA3D_ERR_ARCH;
}

// ------------------------------------------------------------------ TMA descriptors

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// The (B,T,H,W,NH,HD) tensor viewed as 5-D (NH*HD, W, H, T, B), with
// `token_stride` elements between consecutive grid positions: a box of
// {hd_box, bx, by, bz, 1} at x = head*HD + column picks one head's rows.
inline bool encode_map(CUtensorMap* m, const void* ptr, int64_t B, int64_t T, int64_t H, int64_t W,
                int64_t NH, int64_t HD, int64_t token_stride, int hd_box, int bx, int by, int bz) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[5] = {cuuint64_t(NH * HD), cuuint64_t(W), cuuint64_t(H), cuuint64_t(T),
                                cuuint64_t(B)};
    const cuuint64_t row = cuuint64_t(token_stride * 2);
    const cuuint64_t strides[4] = {row, row * W, row * W * H, row * W * H * T};
    const cuuint32_t box[5] = {cuuint32_t(hd_box), cuuint32_t(bx), cuuint32_t(by), cuuint32_t(bz), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUtensorMapSwizzle swz = hd_box == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                   : hd_box == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                  : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major (outer, inner) bf16 matrix as a 2-D tensor map with a
// (box_inner, box_outer) box and the 128-byte swizzle (box_inner = 64).
inline bool encode_map_2d(CUtensorMap* m, const void* ptr, int64_t inner, int64_t outer, int box_inner,
                   int box_outer) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
    const cuuint64_t strides[1] = {cuuint64_t(inner * 2)};
    const cuuint32_t box[2] = {cuuint32_t(box_inner), cuuint32_t(box_outer)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace na3d
