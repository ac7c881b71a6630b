// mx_gemm.hip -- products with MXFP4 weights, dense (qgemm_run*) and grouped
// by expert (qgemm_run_grouped): C[s] = act(A[row(s)] x deq(B_e) + bias_e +
// residual[s]) for the slots s of every group e; the dense product is the
// one-group case with row(s) = s.
//
// deq(B)[k][n] = 2^(scale[n][k / 32] - 127) E2M1(q[n][k]). With fp16
// activations the weight is formed in fp16 by gfx950's scaled conversion (two
// codes an instruction, one rounding, exact for scales 2^-23 .. 2^13) and
// meets A in v_mfma_f32_32x32x16_f16. With MXFP4 activations both operands
// go to v_mfma_scale_f32_32x32x64_f8f6f4 as codes and scale bytes: the 32
// codes a lane feeds are exactly one scaled block, and a packed 1 KiB record
// is one operand.
#include "mx_common.h"

namespace qg {
namespace {

typedef int i8v_t __attribute__((ext_vector_type(8)));

// The 32 codes of a lane as a scaled-MFMA operand (the FP4 form reads the
// first four registers).
__device__ __forceinline__ i8v_t mx_operand(u4_t c) {
    return i8v_t{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

constexpr int kFp4 = 4;      // operand type of the scaled MFMA

__device__ __forceinline__ f16_t mfma_fp4(u4_t a, u4_t b, f16_t c, unsigned sa, unsigned sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, kFp4, kFp4, 0,
                                                           (int)sa, 0, (int)sb);
}

// One wave per 32 x 32 tile of C, operands straight from memory.
template <bool A4>
__global__ __launch_bounds__(256) void mx_gemm_kernel(MxArgs p) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int tile_m = blockIdx.x / p.tiles_n, tn = blockIdx.x % p.tiles_n;
    const RowTile rt = find_row_tile(p.offsets, p.E, p.S, 32, tile_m);
    if (rt.e < 0) return;
    const int n64 = p.K >> 6, n256 = (p.K + 255) >> 8;
    const int t = min(tn * 4 + wave, (p.N + 31) / 32 - 1);
    const uint8_t *W = p.W + (size_t)rt.e * p.w_bytes + (size_t)t * n64 * 1024 + lane * 16;
    const uint8_t *Ws = p.Ws + (size_t)rt.e * p.s_bytes + (size_t)t * n256 * 256 + lane * 4;
    const int slot = rt.s0 + min(r, rt.n - 1);
    const size_t arow = p.rows ? (size_t)min(max(p.rows[slot], 0), p.a_rows - 1) : (size_t)slot;

    f16_t acc = {};
    if constexpr (A4) {
        const uint8_t *a = p.Aq + arow * n256 * 128 + 16 * h;
        const uint8_t *as = p.As + (arow * n256 * 2 + h) * 4;
        for (int b = 0; b < n64; ++b)
            acc = mfma_fp4(*reinterpret_cast<const u4_t *>(a + 32 * b),
                           *reinterpret_cast<const u4_t *>(W + (size_t)b * 1024), acc,
                           as[(b >> 2) * 8 + (b & 3)], Ws[(b >> 2) * 256 + (b & 3)]);
    } else {
        const _Float16 *a = static_cast<const _Float16 *>(p.A) + arow * p.K + 32 * h;
        for (int b = 0; b < n64; ++b) {
            const u4_t w = *reinterpret_cast<const u4_t *>(W + (size_t)b * 1024);
            const float s = mx_scale(Ws[(b >> 2) * 256 + (b & 3)]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                    *reinterpret_cast<const h8_t *>(a + 64 * b + 8 * i), mx_decode8(w[i], s), acc, 0, 0, 0);
        }
    }
    const int n = (tn * 4 + wave) * 32 + r;
    if (n >= p.N) return;
    Epilogue epi = p.epi;
    if (epi.bias) epi.bias += (size_t)rt.e * p.N;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int m = 8 * (j >> 2) + 4 * h + (j & 3);
        if (m < rt.n) epi_put(epi, p.C, rt.s0 + m, n, p.N, acc[j]);
    }
}

}  // namespace

hipError_t launch_mx_gemm(qgemm_format f, const MxArgs &args, void *ws, hipStream_t s) {
    MxArgs p = args;
    p.tiles_n = div_up(p.N, 128);
    const dim3 grid((unsigned)mx_grid(p.S, p.offsets ? p.E : 1, p.N));
    if (f == QGEMM_MXFP4_A4) {
        const MxWorkspace w = mx_workspace(f, p.a_rows, p.K);
        uint8_t *base = static_cast<uint8_t *>(ws);
        const hipError_t e = launch_mx_quantize_act(p.a_rows, p.K, p.A, base, base + w.s_off, s);
        if (e != hipSuccess) return e;
        p.Aq = base;
        p.As = base + w.s_off;
        hipLaunchKernelGGL(mx_gemm_kernel<true>, grid, dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL(mx_gemm_kernel<false>, grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace qg
