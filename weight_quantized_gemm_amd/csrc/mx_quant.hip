// mx_quant.hip -- MXFP4 (microscaled 4-bit floats) conversions: float rows ->
// E2M1 codes and E8M0 scales, codes -> values, and the canonical -> packed
// permutation of weights.
//
// Block of 32 elements with largest magnitude m (OCP Microscaling Formats
// v1.0, conversion to MXFP4): the shared exponent is floor(log2 m) - 2 (2 is
// the exponent of E2M1's largest value), limited to [-127, 127]; every
// element is divided by 2^e (exact) and rounded to the nearest E2M1 value,
// ties to even, at most 6. The exponent comes from the bits of m as an fp32
// number: its biased exponent E gives the scale byte max(E - 2, 0), because
// byte = (E - 127) - 2 + 127 and everything with E <= 2 (subnormal fp32
// numbers too) is limited to byte 0. gfx950 converts two elements to codes in
// one instruction that takes the scale as an fp32 operand; it divides,
// rounds to nearest even and saturates as the rule above says (compared code
// by code in the tests).
//
// All kernels here are bound by memory: 4 lanes share a block (8 elements, one
// code word each), so the block's maximum costs two exchanges among
// neighbouring lanes and nothing goes through LDS. Loads and stores are in
// order across a wave. 4096 x 4096, inputs and outputs rotated past the
// last-level cache: fp32 quantise 15.3 us, dequantise 21.7 (76 MB each: 5.0 and
// 3.5 TB/s; 14.6 and 14.3 where the same buffers are used again), fp16 10.3 and
// 10.8, bf16 10.4 and 10.7 (4 TB/s); one row costs a launch, 1.8 us.
#include "kernels_common.h"
#include "mx_common.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGrid = 4096;      // workgroups: sixteen per CU, then each walks on

// Where a block's codes and scale byte go.
enum Layout { CANON = 0, ACT = 1, PACKED = 2 };

struct Walk {            // a thread's position: row r, 8-element chunk c of it
    unsigned chunks;     // chunks per row
    unsigned dr, dc;     // one step of the whole grid, as rows and chunks
};

// 8 elements of type T at p (16-byte aligned) as fp32.
template <int T>
__device__ __forceinline__ void load8(const void *p, float (&v)[8]) {
    if constexpr (T == QGEMM_TYPE_F32) {
        const f4_t a = static_cast<const f4_t *>(p)[0], b = static_cast<const f4_t *>(p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else if constexpr (T == QGEMM_TYPE_F16) {
        const h8_t a = *static_cast<const h8_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    } else {
        const u4_t a = *static_cast<const u4_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
}

template <int T> struct ElemSize { static constexpr int value = T == QGEMM_TYPE_F32 ? 4 : 2; };

// `rows` rows of the output; those from R on (packed padding) and the chunks
// from K on (padding of the activation and packed layouts) are zeros.
template <int T, int L>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(size_t R, size_t rows, int K, Walk w,
                                                               const char *__restrict__ X, size_t ldx,
                                                               uint8_t *__restrict__ q,
                                                               uint8_t *__restrict__ scales) {
    const unsigned i0 = blockIdx.x * kThreads + threadIdx.x;
    size_t r = i0 / w.chunks;
    unsigned c = i0 % w.chunks;
    const unsigned kc = (unsigned)K >> 3;         // chunks that hold elements
    const unsigned n64 = (unsigned)K >> 6, n256 = ((unsigned)K + 255) >> 8;
    // chunks is a multiple of 4, so the four lanes of a block walk together
    while (r < rows) {
        unsigned word = 0, byte = 0;
        if (r < R && c < kc) {
            float v[8];
            load8<T>(X + (r * ldx + 8 * (size_t)c) * ElemSize<T>::value, v);
            unsigned top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
            word = mx_encode8(v, top, &byte);
        }
        if constexpr (L == CANON) {
            reinterpret_cast<unsigned *>(q)[r * kc + c] = word;
            if ((c & 3) == 0) scales[r * (kc >> 2) + (c >> 2)] = (uint8_t)byte;
        } else if constexpr (L == ACT) {
            reinterpret_cast<unsigned *>(q)[r * w.chunks + c] = word;
            if ((c & 3) == 0) scales[mx_act_scale(r, c >> 3, (c >> 2) & 1, n256)] = (uint8_t)byte;
        } else {
            const unsigned b = c >> 3, h = (c >> 2) & 1;
            if (c < kc)
                reinterpret_cast<unsigned *>(q + ((r >> 5) * n64 + b) * 1024)[(32 * h + (unsigned)(r & 31)) * 4 + (c & 3)] = word;
            if ((c & 3) == 0) scales[mx_weight_scale(r, b, h, n256)] = (uint8_t)byte;
        }
        r += w.dr;
        c += w.dc;
        if (c >= w.chunks) c -= w.chunks, ++r;
    }
}

template <int T>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(size_t R, int K, Walk w,
                                                                 const uint8_t *__restrict__ q,
                                                                 const uint8_t *__restrict__ scales,
                                                                 char *__restrict__ Y, size_t ldy) {
    const unsigned i0 = blockIdx.x * kThreads + threadIdx.x;
    size_t r = i0 / w.chunks;
    unsigned c = i0 % w.chunks;
    while (r < R) {
        const unsigned word = reinterpret_cast<const unsigned *>(q)[r * w.chunks + c];
        const float s = mx_scale(scales[r * (w.chunks >> 2) + (c >> 2)]);
        char *p = Y + (r * ldy + 8 * (size_t)c) * ElemSize<T>::value;
        if constexpr (T == QGEMM_TYPE_F32) {
            const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 0);
            const f2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 1);
            const f2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 2);
            const f2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 3);
            reinterpret_cast<f4_t *>(p)[0] = f4_t{a.x, a.y, b.x, b.y};
            reinterpret_cast<f4_t *>(p)[1] = f4_t{d.x, d.y, e.x, e.y};
        } else if constexpr (T == QGEMM_TYPE_F16) {
            *reinterpret_cast<h8_t *>(p) = mx_decode8(word, s);
        } else {
            u4_t o;
            o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, s, 0));
            o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, s, 1));
            o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, s, 2));
            o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, s, 3));
            *reinterpret_cast<u4_t *>(p) = o;
        }
        r += w.dr;
        c += w.dc;
        if (c >= w.chunks) c -= w.chunks, ++r;
    }
}

// One thread per 16-byte piece of a packed record (32 codes of a channel) and
// its scale byte; blockIdx.y is the weight. Blocks from n64 on (K is a
// multiple of 64, the scale records cover 256) write zero scales only.
__global__ __launch_bounds__(kThreads) void mx_pack_kernel(int K, int N, unsigned tiles,
                                                           const uint8_t *__restrict__ q,
                                                           const uint8_t *__restrict__ scales,
                                                           uint8_t *__restrict__ wp,
                                                           uint8_t *__restrict__ sp, size_t w_bytes,
                                                           size_t s_bytes) {
    const unsigned n64 = (unsigned)K >> 6, n256 = ((unsigned)K + 255) >> 8;
    const size_t e = blockIdx.y;
    q += e * N * (K / 2);
    scales += e * N * (K / 32);
    wp += e * w_bytes;
    sp += e * s_bytes;
    const size_t pieces = (size_t)tiles * n256 * 4 * 64;
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += (size_t)gridDim.x * kThreads) {
        const unsigned lane = i & 63;
        const size_t rec = i >> 6;
        const unsigned t = (unsigned)(rec / (n256 * 4)), b = (unsigned)(rec % (n256 * 4));
        const unsigned c = lane & 31, h = lane >> 5;
        const size_t n = (size_t)32 * t + c;
        const bool live = n < (size_t)N && b < n64;
        if (b < n64) {
            u4_t v = {0u, 0u, 0u, 0u};
            if (live) v = *reinterpret_cast<const u4_t *>(q + n * (K / 2) + 32 * (size_t)b + 16 * h);
            reinterpret_cast<u4_t *>(wp + ((size_t)t * n64 + b) * 1024)[lane] = v;
        }
        sp[mx_weight_scale(n, b, h, n256)] = live ? scales[n * (K / 32) + 2 * b + h] : 0;
    }
}

Walk make_walk(size_t rows, unsigned chunks, unsigned *grid) {
    const size_t items = rows * chunks;
    size_t g = (items + kThreads - 1) / kThreads;
    if (g > kMaxGrid) g = kMaxGrid;
    *grid = (unsigned)g;
    const unsigned step = (unsigned)g * kThreads;
    return Walk{chunks, step / chunks, step % chunks};
}

template <int L>
hipError_t quantize(size_t R, size_t rows, int K, unsigned chunks, int t, const void *X, size_t ldx,
                    uint8_t *q, uint8_t *scales, hipStream_t s) {
    unsigned grid = 0;
    const Walk w = make_walk(rows, chunks, &grid);
    auto kernel = t == QGEMM_TYPE_F32   ? mx_quantize_kernel<QGEMM_TYPE_F32, L>
                  : t == QGEMM_TYPE_F16 ? mx_quantize_kernel<QGEMM_TYPE_F16, L>
                                        : mx_quantize_kernel<QGEMM_TYPE_BF16, L>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, R, rows, K, w, static_cast<const char *>(X),
                       ldx, q, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int R, int K, int t, const void *X, size_t ldx, uint8_t *q, uint8_t *scales,
                              hipStream_t s) {
    return quantize<CANON>(R, R, K, (unsigned)K / 8, t, X, ldx, q, scales, s);
}

hipError_t launch_mx_quantize_act(int R, int K, const void *A, uint8_t *q, uint8_t *scales, hipStream_t s) {
    return quantize<ACT>(R, R, K, (unsigned)round_up(K, 256) / 8, QGEMM_TYPE_F16, A, K, q, scales, s);
}

hipError_t launch_mx_quantize_pack(int K, int N, const float *W, void *Bq, void *scales, hipStream_t s) {
    return quantize<PACKED>(N, round_up(N, 32), K, (unsigned)round_up(K, 256) / 8, QGEMM_TYPE_F32, W, K,
                            static_cast<uint8_t *>(Bq), static_cast<uint8_t *>(scales), s);
}

hipError_t launch_mx_dequantize(int R, int K, const uint8_t *q, const uint8_t *scales, int t, void *Y,
                                size_t ldy, hipStream_t s) {
    unsigned grid = 0;
    const Walk w = make_walk(R, (unsigned)K / 8, &grid);
    auto kernel = t == QGEMM_TYPE_F32   ? mx_dequantize_kernel<QGEMM_TYPE_F32>
                  : t == QGEMM_TYPE_F16 ? mx_dequantize_kernel<QGEMM_TYPE_F16>
                                        : mx_dequantize_kernel<QGEMM_TYPE_BF16>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, (size_t)R, K, w, q, scales,
                       static_cast<char *>(Y), ldy);
    return hipGetLastError();
}

hipError_t launch_mx_pack(int K, int N, int E, const uint8_t *q, const uint8_t *scales, void *wp, void *sp,
                          size_t w_bytes, size_t s_bytes, hipStream_t s) {
    const unsigned tiles = (unsigned)div_up(N, 32);
    const size_t pieces = (size_t)tiles * (round_up(K, 256) / 64) * 64;
    const size_t grid = (pieces + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(mx_pack_kernel, dim3((unsigned)(grid > kMaxGrid ? kMaxGrid : grid), (unsigned)E),
                       dim3(kThreads), 0, s, K, N, tiles, q, scales, static_cast<uint8_t *>(wp),
                       static_cast<uint8_t *>(sp), w_bytes, s_bytes);
    return hipGetLastError();
}

}  // namespace qg
