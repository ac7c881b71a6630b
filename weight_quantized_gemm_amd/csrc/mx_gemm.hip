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
#include <type_traits>

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

// c += a x b with byte s (a constant once unrolled) of the scale words.
__device__ __forceinline__ f16_t mfma_fp4(u4_t a, u4_t b, f16_t c, unsigned sa, unsigned sb, int s) {
#define QG_MFMA(S)                                                                                         \
    __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, kFp4, kFp4, S, (int)sa, \
                                                    S, (int)sb)
    switch (s) {
    case 0: return QG_MFMA(0);
    case 1: return QG_MFMA(1);
    case 2: return QG_MFMA(2);
    default: return QG_MFMA(3);
    }
#undef QG_MFMA
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, void *lds, unsigned voff, unsigned soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, (int)voff,
                                             (int)soff, 0, 0);
#endif
}
__device__ __forceinline__ u4_t load16(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff) {
    return __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}
// The same, past the caches, for bytes that no other workgroup wants.
__device__ __forceinline__ u4_t load16_once(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff) {
    return __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 2));
}
__device__ __forceinline__ unsigned load4(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff) {
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, (int)soff, 0));
}
__device__ __forceinline__ unsigned load1(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff) {
    return __builtin_amdgcn_raw_buffer_load_b8(r, (int)voff, (int)soff, 0);
}

// A's row of a slot: through the index, limited to A's rows, or the slot.
__device__ __forceinline__ int a_row(const MxArgs &p, int slot) {
    return p.rows ? min(max(p.rows[slot], 0), p.a_rows - 1) : slot;
}

// A workgroup barrier without __syncthreads' release fence, which would also
// wait for the loads in flight; LDS reads before it have been consumed, and
// the fence keeps later ones behind it.
__device__ __forceinline__ void stage_barrier() {
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Orders one wave's LDS writes before its later reads of them (and the other
// way round) for the compiler; the hardware keeps a wave's LDS operations in
// order.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The library's activations. SiLU x / (1 + e^-x) without the full-range
// exponential and division, which cost more than the rest of a prefill
// epilogue (2048 x 11008 outputs: 24 us of vector instructions against 6):
// e^-x = 2^t (1 + c) with t = -x log2 e in one rounding and c its error times
// ln 2 (two fused multiply-adds, log2 e in two parts), so the hardware's
// 2^t and 1 / d leave about two units. x is limited to [-88.5, 100] in the
// exponent: above, the result is x itself; below about -87.3 the reciprocal is
// a subnormal number, which the hardware returns as zero, so the result is -0
// however far x lies out (its value is less than 1.2e-36 in size), and NaN at
// -infinity as from the division.
// For an fp16 result the first rounding alone (a few 2^-24 of the value) is
// far below the result's own.
__device__ __forceinline__ float silu16(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269502f));
}
__device__ __forceinline__ float silu32(float v) {
    const float x = __builtin_amdgcn_fmed3f(v, -88.5f, 100.0f);
    const float t = x * -1.44269502f;                             // log2 e = 1.44269502 + 1.92596303e-8
    const float c = fmaf(x, -1.92596303e-8f, fmaf(x, -1.44269502f, -t));
    float p = __builtin_amdgcn_exp2f(t);
    p = fmaf(p, c * 0.693147181f, p);
    return v * __builtin_amdgcn_rcpf(1.0f + p);
}

// The epilogue of a lane that holds columns n .. n + 3 (n a multiple of 4) of
// several rows: its bias is loaded once, before any store (a wait for a load
// waits for the stores issued before it as well), rows are handled B at a
// time, a batch's loads all requested before the first use. VEC: N is a
// multiple of 4, so four columns are one vector in every row; otherwise rows
// of C (and of bias and residual) start anywhere.
template <bool VEC>
struct ColumnEpilogue {
    Epilogue epi;
    void *C;
    int n, N;
    f4_t bias;

    __device__ __forceinline__ ColumnEpilogue(const Epilogue &e, void *C_, int n_, int N_)
        : epi(e), C(C_), n(n_), N(N_), bias{0.f, 0.f, 0.f, 0.f} {
        if (e.bias) {
            if constexpr (VEC) {
                bias = *reinterpret_cast<const f4_t *>(e.bias + min(n, N - 4));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) bias[i] = e.bias[min(n + i, N - 1)];
            }
        }
        asm volatile("" : "+v"(bias));     // here, not in the loops of rows
    }

    template <int B>
    __device__ __forceinline__ void activate(f4_t (&v)[B]) const {
        if (epi.act == QGEMM_ACT_NONE) return;
        if (epi.act == QGEMM_ACT_SILU) {
            if (epi.f16) {
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = silu16(v[i][c]);
            } else {
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = silu32(v[i][c]);
            }
        } else if (epi.act == QGEMM_ACT_RELU) {
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = v[i][c] > 0.f ? v[i][c] : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const float x = epi_act(v[i][0], QGEMM_ACT_GELU);
                    v[i] = f4_t{v[i][1], v[i][2], v[i][3], x};
                }
        }
    }

    // rows m, m + step, ... of the `rows` (at least one) from slot0 on, with
    // values v; those past the last are left out
    template <int B>
    __device__ __forceinline__ void put(size_t slot0, int m, int step, int rows, f4_t (&v)[B]) const {
        if (n >= N) return;
        size_t at[B];
#pragma unroll
        for (int i = 0; i < B; ++i) at[i] = (slot0 + min(m + i * step, rows - 1)) * N + n;
        if (epi.residual) {
            // (a row past the last re-reads that one, to keep the loads together)
            f4_t res[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if constexpr (VEC) {
                    if (epi.f16) {
                        const h4_t x = *reinterpret_cast<const h4_t *>(static_cast<const _Float16 *>(epi.residual) + at[i]);
                        res[i] = f4_t{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
                    } else {
                        res[i] = *reinterpret_cast<const f4_t *>(static_cast<const float *>(epi.residual) + at[i]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const size_t k = at[i] + min(c, N - 1 - n);
                        res[i][c] = epi.f16 ? (float)static_cast<const _Float16 *>(epi.residual)[k]
                                            : static_cast<const float *>(epi.residual)[k];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) v[i] = (v[i] + bias) + res[i];
        } else {
#pragma unroll
            for (int i = 0; i < B; ++i) v[i] = v[i] + bias;
        }
        activate(v);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (m + i * step >= rows) continue;
            if constexpr (VEC) {
                if (epi.f16)
                    *reinterpret_cast<h4_t *>(static_cast<_Float16 *>(C) + at[i]) =
                        h4_t{(_Float16)v[i][0], (_Float16)v[i][1], (_Float16)v[i][2], (_Float16)v[i][3]};
                else
                    *reinterpret_cast<f4_t *>(static_cast<float *>(C) + at[i]) = v[i];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n + c < N) epi_store(epi, C, at[i] + c, v[i][c]);
            }
        }
    }
};

// s_waitcnt operand: at most n vector memory loads outstanding, and no LDS read.
constexpr int stage_wait(int n) { return vm_wait(n) & ~0xF00; }

// ---------------------------------------------------------------------------
// Tiled product
// ---------------------------------------------------------------------------
template <bool A4_, int RF_, int CF_, int WM_, int WN_, int WK_, int NS_, int BR_, int MINW_ = 1>
struct Tile {
    static constexpr bool A4 = A4_;
    static constexpr int RF = RF_, CF = CF_, WM = WM_, WN = WN_, WK = WK_, NS = NS_, BR = BR_, MINW = MINW_;
    static constexpr int BM = 32 * RF * WM, BN = 32 * CF * WN;
    static constexpr int GW = WM * WN;                    // waves of a K group
    static constexpr int THREADS = 64 * GW * WK;
    static constexpr int SLOT = BM * 128;                 // bytes of A per stage
    static constexpr int D = BM / 8 / GW;                 // DMA instructions per wave and stage
    static constexpr int NREC = A4 ? 4 : 1;               // weight records per stage and column fragment
    static constexpr int NB = CF * NREC + CF;             // other loads per wave and stage
    // scales of the tile's rows (MXFP4 activations): 8 bytes a stage, the NS
    // stages of an unrolled turn in one of two slots; in DMA instructions of
    // RPI rows
    static constexpr int PPR = NS / 2;                    // 16-byte pieces per row
    static constexpr int RPI = 64 / PPR;
    static constexpr int ASC = A4 ? (BM + RPI - 1) / RPI * 1024 : 0;          // bytes of a slot
    static constexpr int DS = A4 ? ((BM + RPI - 1) / RPI + GW - 1) / GW : 0;
    // register slots of the weights' scales: MXFP4 activations take a stage's
    // codes step by step, and scales fetched no earlier than its last codes
    // would be what its first step waits for
    static constexpr int SR = A4 ? NS : BR;
    // loads issued since the DMA of the next stage when a wave waits for it
    // (the weights' and scales' of that stage, everything of NS - 2 more)
    static constexpr int WAIT = NB + (NS - 2) * (D + NB);
    // MFMA steps that A is read from LDS ahead of its use: a step of one or two
    // matrix instructions is much shorter than a read (128 x 4096 x 4096 in
    // 64 x 128 tiles 21.9 us one step ahead, 20.7 three), a long one with four
    // or eight gains from two with fp16 activations (512 x 4096 x 4096 in 64 x
    // 256 tiles 41.4 -> 39.7) but not with MXFP4 ones, which lack the registers
    static constexpr int PD = RF * CF <= 2 ? 3 : A4 ? 1 : 2;
    // loads issued after the prologue's DMA
    static constexpr int PRO = A4 ? BR * 4 * CF + SR * CF : BR * NB;
    // floats per row of a wave's C block in LDS: rows 4 apart, which one
    // instruction writes, fall into different halves of the banks
    static constexpr int PITCH = 32 * CF + 8;
    static constexpr int LDS_A = WK * (NS * SLOT + 2 * ASC);
    static constexpr int LDS_C = WK > 1 ? WK * BM * BN * 4 : GW * 32 * PITCH * 4;
    static constexpr int LDS = LDS_A > LDS_C ? LDS_A : LDS_C;
    static_assert(D * 8 * GW == BM, "whole DMA instructions");
    static_assert(!A4 || NS == 2 || NS == 4, "whole pieces of scales");
    static_assert(NS % SR == 0 && NS % BR == 0, "register slots repeat within an unrolled turn");
    static_assert(WAIT <= 63 && PRO <= 63, "vmcnt range");
    static_assert(LDS <= 160 * 1024, "LDS of a workgroup");
};

template <class T>
__global__ __launch_bounds__(T::THREADS, T::MINW) void mx_tile_kernel(MxArgs p) {
    constexpr bool A4 = T::A4;
    constexpr int RF = T::RF, CF = T::CF, NS = T::NS, BR = T::BR, D = T::D, WK = T::WK;
    __shared__ __align__(16) unsigned char lds[T::LDS];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int kg = wave / T::GW, gw = wave % T::GW, wm = gw / T::WN, wn = gw % T::WN;
    RowTile rt = find_tile(p.offsets, p.E, p.S, T::BM, p.tiles_n, blockIdx.x);
    if (rt.e < 0) return;
    // scalars: the buffer resources built from them must be
    rt = RowTile{uniform(rt.e), uniform(rt.s0), uniform(rt.n), uniform(rt.tn)};
    const int tn = rt.tn;
    const int n64 = p.K >> 6, n256 = (p.K + 255) >> 8;
    // this slice's stages, and of those this K group's
    const int nall = A4 ? n256 : n64;
    // (of whole pairs with MXFP4 activations, whose scales come in pairs)
    constexpr int U = A4 ? 2 : 1;
    int lo = 0, units = (nall + U - 1) / U;
    if (gridDim.y > 1) {
        lo = (int)blockIdx.y * units / (int)gridDim.y;
        units = ((int)blockIdx.y + 1) * units / (int)gridDim.y - lo;
    }
    const int st0 = U * (lo + kg * units / WK), nst = min(U * (lo + (kg + 1) * units / WK), nall) - st0;
    const int nmax = U * ((units + WK - 1) / WK);      // of the longest K group, at most
    const int last = max(nst - 1, 0);

    // A: gathered rows from the array's start, others from the tile's first row
    const unsigned row_bytes = A4 ? (unsigned)n256 * 128u : (unsigned)p.K * 2u;
    const size_t first = p.rows ? 0 : (size_t)rt.s0;
    const uint8_t *Ab = (A4 ? p.Aq : static_cast<const uint8_t *>(p.A)) + first * row_bytes;
    const __amdgpu_buffer_rsrc_t a_rs = byte_rsrc(Ab, 0xFFFFFFFFu);
    unsigned a_off[D];
#pragma unroll
    for (int i = 0; i < D; ++i) {
        const int row = 8 * (gw + T::GW * i) + (lane >> 3);
        a_off[i] = (unsigned)(a_row(p, rt.s0 + min(row, rt.n - 1)) - (int)first) * row_bytes +
                   16u * ((lane & 7) ^ (lane >> 3));
    }
    // scales: 16-byte piece x (two stages) of a row stands at x ^ (row / 8 %
    // 2), so that the 32 rows one instruction reads spread over the banks;
    // lane l of an instruction brings piece l % PPR of row l / PPR
    const unsigned as_bytes = mx_act_groups(n256) * 8u;
    const __amdgpu_buffer_rsrc_t as_rs = byte_rsrc(A4 ? p.As + first * as_bytes : p.As, 0xFFFFFFFFu);
    unsigned as_off[A4 ? T::DS : 1];
    if constexpr (A4) {
#pragma unroll
        for (int i = 0; i < T::DS; ++i) {
            const int row = min(T::RPI * (gw + T::GW * i) + lane / T::PPR, T::BM - 1);
            as_off[i] = (unsigned)(a_row(p, rt.s0 + min(row, rt.n - 1)) - (int)first) * as_bytes +
                        16u * (T::PPR == 1 ? 0u : (lane ^ (row >> 3)) & 1u);
        }
    }
    // B: the records and scales of this wave's column fragments
    const int ntiles = (p.N + 31) / 32;
    __amdgpu_buffer_rsrc_t b_rs[CF], bs_rs[CF];
#pragma unroll
    for (int cf = 0; cf < CF; ++cf) {
        const int t = min((tn * T::WN + wn) * CF + cf, ntiles - 1);
        b_rs[cf] = byte_rsrc(p.W + (size_t)rt.e * p.w_bytes + (size_t)t * n64 * 1024, (unsigned)n64 * 1024u);
        bs_rs[cf] = byte_rsrc(p.Ws + (size_t)rt.e * p.s_bytes + (size_t)t * n256 * 256, (unsigned)n256 * 256u);
    }

    unsigned char *const mine = lds + (size_t)kg * (NS * T::SLOT + 2 * T::ASC);
    unsigned char *const mine_s = mine + NS * T::SLOT;
    auto dma = [&](int slot, int st) {
        const unsigned so = (unsigned)(st0 + min(st, last)) * 128u;
#pragma unroll
        for (int i = 0; i < D; ++i)
            dma16(a_rs, mine + slot * T::SLOT + (gw + T::GW * i) * 1024, a_off[i], so);
    };
    // the scales of turn c (stages NS c ..) into slot c % 2
    auto dma_scales = [&](int c) {
        const unsigned so = (unsigned)(st0 + min(NS * c, last / NS * NS)) * 8u;
#pragma unroll
        for (int i = 0; i < T::DS; ++i)
            if (T::DS * T::GW * T::RPI == T::BM || T::RPI * (gw + T::GW * i) < T::BM)
                dma16(as_rs, mine_s + (c & 1) * T::ASC + (gw + T::GW * i) * 1024, as_off[i], so);
    };
    // MXFP4 activations: a record per step, reloaded for the next stage as
    // soon as its step has run, and the stage's scale words in two slots.
    // fp16 activations: one record and scale byte for the whole stage.
    u4_t bc[BR][CF][T::NREC];
    unsigned bs[T::SR][CF], as[2][RF];
    auto load_codes = [&](int j, int rec, int st) {
        const int k = (st0 + min(st, last)) * T::NREC + rec;
#pragma unroll
        for (int cf = 0; cf < CF; ++cf)
            bc[j][cf][rec] = load16(b_rs[cf], lane * 16u, (unsigned)min(k, n64 - 1) * 1024u);
    };
    auto load_scales = [&](int j, int st) {
        const int k = st0 + min(st, last);
#pragma unroll
        for (int cf = 0; cf < CF; ++cf)
            bs[j][cf] = A4 ? load4(bs_rs[cf], lane * 4u, (unsigned)k * 256u)
                           : load1(bs_rs[cf], lane * 4u, (unsigned)(k >> 2) * 256u + (k & 3));
    };
    // the words of a turn's stage u
    auto read_scales = [&](int j, int c, int u) {
        if constexpr (A4) {
            const unsigned char *src = mine_s + (c & 1) * T::ASC + (32 * RF * wm + r) * (16 * T::PPR) +
                                       16 * (T::PPR == 1 ? 0 : (u >> 1 ^ r >> 3) & 1) + 8 * (u & 1) + 4 * h;
#pragma unroll
            for (int rf = 0; rf < RF; ++rf)
                as[j][rf] = *reinterpret_cast<const unsigned *>(src + rf * 32 * (16 * T::PPR));
        }
    };

    f16_t acc[RF][CF];
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < CF; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    // operands of one MFMA step: s of the stage in LDS slot `slot` and register slot j
    // (A's PD steps ahead)
    constexpr int PD = T::PD, AR = PD == 1 ? 2 : 4;
    u4_t a[AR][RF];
    h8_t b[2][CF];
    const unsigned char *const a_lds = mine + (32 * RF * wm + r) * 128;
    auto read_a = [&](u4_t (&dst)[RF], int slot, int s) {
#pragma unroll
        for (int rf = 0; rf < RF; ++rf)
            dst[rf] = *reinterpret_cast<const u4_t *>(a_lds + slot * T::SLOT + rf * 4096 +
                                                      16 * ((A4 ? 2 * s + h : 4 * h + s) ^ (r & 7)));
    };
    auto decode_b = [&](h8_t (&dst)[CF], int j, int s) {
        if constexpr (!A4) {
#pragma unroll
            for (int cf = 0; cf < CF; ++cf) {
                dst[cf] = mx_decode8(bc[j][cf][0][s], mx_scale(bs[j % T::SR][cf]));
                asm volatile("" : "+v"(dst[cf]));      // formed here, not next to its use
            }
        }
    };
    auto multiply = [&](int x, int z, int j, int y, int s) {
#pragma unroll
        for (int rf = 0; rf < RF; ++rf)
#pragma unroll
            for (int cf = 0; cf < CF; ++cf) {
                if constexpr (A4)
                    acc[rf][cf] = mfma_fp4(a[x][rf], bc[y][cf][s], acc[rf][cf], as[j & 1][rf], bs[j][cf], s);
                else
                    acc[rf][cf] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8_t, a[x][rf]), b[z][cf],
                                                                         acc[rf][cf], 0, 0, 0);
            }
        if constexpr (A4) {
#pragma unroll
            for (int i = 0; i < RF; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, CF, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RF; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int i = 0; i < RF * CF; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, (6 + RF - 1) / RF, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    if constexpr (A4) dma_scales(0);
#pragma unroll
    for (int d = 0; d < NS; ++d) dma(d, d);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < T::SR || d < BR; ++d) {
        if (d < BR) {
#pragma unroll
            for (int k = 0; k < T::NREC; ++k) load_codes(d, k, d);
        }
        if (d < T::SR) load_scales(d, d);
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(vm_wait(T::PRO));
    stage_barrier();
    read_scales(0, 0, 0);
#pragma unroll
    for (int s = 0; s < PD; ++s) read_a(a[s], 0, s);
    decode_b(b[0], 0, 0);

    auto stage = [&](int base, int u) {
        const int i = base + u;
        const int j = u % T::SR, y = u % BR;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s == 4 - PD) {
                // The reads of this stage are done, and the next ones are
                // the next stage's. (No branch here: the optimiser would
                // move the matrix instructions above into the block
                // behind it, past the loads.)
                __builtin_amdgcn_s_waitcnt(stage_wait(T::WAIT));
                stage_barrier();
                dma(u, i + NS);
                // (the other slot's scales, of the turn before, have been read)
                if constexpr (A4) {
                    if (u == 0) dma_scales(base / NS + 1);
                }
                __builtin_amdgcn_sched_barrier(0);
                read_scales((u + 1) & 1, base / NS + (u + 1) / NS, (u + 1) % NS);
            }
            if (s + PD < 4) read_a(a[(s + PD) % AR], u, s + PD);
            else read_a(a[(s + PD) % AR], (u + 1) % NS, s + PD - 4);
            if (s < 3) {
                decode_b(b[(s + 1) & 1], j, s + 1);
            } else {
                if constexpr (!A4) {
                    load_codes(j, 0, i + BR);
                    load_scales(j, i + BR);
                    __builtin_amdgcn_sched_barrier(0);
                }
                decode_b(b[0], (u + 1) % T::SR, 0);
            }
            multiply(s % AR, s & 1, j, y, s);
            if constexpr (A4) {
                load_codes(y, s, i + BR);
                if (s == 3) load_scales(j, i + T::SR);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // Whole turns, then the stages that are left: with a way out of the middle
    // of a turn the compiler takes it for a way back to the top as well, and
    // waits there, every turn, for all loads in flight.
    int base = 0;
    for (; base + NS <= nst; base += NS) {
#pragma unroll
        for (int u = 0; u < NS; ++u) stage(base, u);
    }
#pragma unroll
    for (int u = 0; u < NS - 1; ++u) {
        if (base + u >= nst) break;            // wave-uniform
        stage(base, u);
    }

    // every wave of the workgroup meets as many barriers
    if constexpr (WK > 1) {
        for (int i = nst; i < nmax; ++i) stage_barrier();
    }

    // ---- C goes through LDS so that a lane holds four neighbouring columns
    //      of a row: whole vectors of bias, residual and C, and the epilogue's
    //      code once, in rolled loops (written out per accumulator register
    //      it left the instruction cache and waited for each bias load) ----
    Epilogue epi = p.epi;
    if (epi.bias) epi.bias += (size_t)rt.e * p.N;
    const int n0 = tn * T::BN;
    __builtin_amdgcn_s_waitcnt(vm_wait(0));      // no DMA in flight into what follows
    __syncthreads();
    float *const out = reinterpret_cast<float *>(lds);
    // (slice y of a split K: its partial tiles; one slice is C itself)
    void *const C = static_cast<float *>(p.C) + (size_t)blockIdx.y * p.S * p.N;
    auto store = [&](auto vec) {
        using CE = ColumnEpilogue<decltype(vec)::value>;
        if constexpr (WK > 1) {
            // the K groups' partial tiles, added in the order of K
            constexpr int TPR = T::BN / 4, STEP = T::THREADS / TPR;      // threads per row, rows per turn
            static_assert(T::THREADS % TPR == 0, "a thread keeps its columns");
            const int col = 4 * (threadIdx.x % TPR);
            const CE ce(epi, C, n0 + col, p.N);
            const float *src = out + (threadIdx.x / TPR) * T::BN + col;
#pragma unroll 1
            for (int m = threadIdx.x / TPR; m < rt.n; m += STEP, src += STEP * T::BN) {
                f4_t v[1] = {*reinterpret_cast<const f4_t *>(src)};
#pragma unroll
                for (int g = 1; g < WK; ++g) v[0] += *reinterpret_cast<const f4_t *>(src + g * T::BM * T::BN);
                ce.put(rt.s0, m, STEP, rt.n, v);
            }
        } else {
            // each wave by itself, 32 rows of its columns at a time
            constexpr int LPR = 8 * CF, STEP = 64 / LPR;      // lanes per row, rows per turn
            float *const own = out + wave * 32 * T::PITCH;
            const int col = 4 * (lane % LPR);
            const CE ce(epi, C, n0 + 32 * CF * wn + col, p.N);
#pragma unroll
            for (int rf = 0; rf < RF; ++rf) {
                const int m0 = 32 * (RF * wm + rf);
                if (m0 >= rt.n) break;               // wave-uniform
#pragma unroll
                for (int cf = 0; cf < CF; ++cf)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        own[(8 * (j >> 2) + 4 * h + (j & 3)) * T::PITCH + 32 * cf + r] = acc[rf][cf][j];
                wave_lds_sync();
#pragma unroll 1
                for (int m = lane / LPR; m < 32; m += 4 * STEP) {
                    f4_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = *reinterpret_cast<const f4_t *>(own + (m + i * STEP) * T::PITCH + col);
                    ce.put(rt.s0, m0 + m, STEP, rt.n, v);
                }
                wave_lds_sync();
            }
        }
    };
    if constexpr (WK > 1) {
#pragma unroll
        for (int rf = 0; rf < RF; ++rf)
#pragma unroll
            for (int cf = 0; cf < CF; ++cf)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    out[(kg * T::BM + 32 * (RF * wm + rf) + 8 * (j >> 2) + 4 * h + (j & 3)) * T::BN +
                        32 * (CF * wn + cf) + r] = acc[rf][cf][j];
        __syncthreads();
    }
    if ((p.N & 3) == 0) store(std::true_type{});
    else store(std::false_type{});
}

// ---------------------------------------------------------------------------
// Few rows (decode): a row tile of RT (2 or 8) rows against 32 channels and
// all of K, for which the weights are the bytes that matter. Eight waves share
// K in groups of 256 elements, taken in turn (one group: four 1 KiB weight
// records, one 256-byte scale record, 512 bytes of every row), each group's
// loads all requested at once. The rows go through LDS, wave by wave without
// a barrier: fp16 as they are, or quantised to MXFP4 on the way (a 32-element
// block is what four neighbouring lanes loaded, so no pass over A of its own
// is needed). The matrix cores run 32 rows wide and the lanes past RT repeat
// real rows: at 1 x 4096 x 11008 that is 1.2 us of matrix work spread over
// the chip beside 4.7 us of memory. The waves' partial sums are added in wave
// order. ONCE (the dense product, whose weights one workgroup reads): weight
// loads past the caches.
// Measured (us): 1 x 4096 x 11008 8.2 (12.7 in 32 x 64 tiles; 8.8 through the
// caches; 8.7 with RT = 8; two groups at once 8.4; 16 waves 8.2, 4 waves 9.1),
// 8 x 4096 x 11008 9.6 (12.9), 1 x 9728 x 2560 8.5 (16.5 in 32 x 32 tiles; 16
// waves 7.6, but 10 experts-grouped rows go from 19 to 27), MXFP4 activations
// 1 x 4096 x 11008 8.0 (11.2 with the separate quantiser and tiles).
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;

template <bool A4, int RT, bool ONCE>
__global__ __launch_bounds__(64 * kDecodeWaves) void mx_decode_kernel(MxArgs p) {
    constexpr int AL = RT / 2;                             // 16-byte loads of A per lane and group
    constexpr int PITCH = A4 ? 144 : 528;                  // bytes per row in LDS (4 banks more than a power of two)
    constexpr int GROUP = RT * PITCH + (A4 ? RT * 8 : 0);  // bytes of a group: the rows, then their scales
    static_assert(GROUP % 16 == 0 && RT <= 8, "aligned groups; C in registers 0 .. 3");
    __shared__ __align__(16) unsigned char rows_lds[kDecodeWaves * GROUP];
    __shared__ __align__(16) float sums[kDecodeWaves * RT * 32];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    RowTile rt = find_tile(p.offsets, p.E, p.S, RT, p.tiles_n, blockIdx.x);
    if (rt.e < 0) return;
    rt = RowTile{uniform(rt.e), uniform(rt.s0), uniform(rt.n), uniform(rt.tn)};
    const int n64 = p.K >> 6, n256 = (p.K + 255) >> 8;
    const __amdgpu_buffer_rsrc_t b_rs =
        byte_rsrc(p.W + (size_t)rt.e * p.w_bytes + (size_t)rt.tn * n64 * 1024, (unsigned)n64 * 1024u);
    const __amdgpu_buffer_rsrc_t bs_rs =
        byte_rsrc(p.Ws + (size_t)rt.e * p.s_bytes + (size_t)rt.tn * n256 * 256, (unsigned)n256 * 256u);
    // this lane's rows of A: half a wave loads the 256 elements of one
    const _Float16 *a_src[AL];
#pragma unroll
    for (int i = 0; i < AL; ++i)
        a_src[i] = static_cast<const _Float16 *>(p.A) + (size_t)a_row(p, rt.s0 + min(2 * i + h, rt.n - 1)) * p.K;
    unsigned char *const mine = rows_lds + wave * GROUP, *const mine_s = mine + RT * PITCH;

    f16_t acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    for (int g = wave; g < n256; g += kDecodeWaves) {
        h8_t a[AL];
        u4_t w[4];
        // elements past K (of the last group) re-read the row's first ones,
        // for records that are not used
        const int k = 256 * g + 8 * r < p.K ? 256 * g + 8 * r : 0;
#pragma unroll
        for (int i = 0; i < AL; ++i) a[i] = *reinterpret_cast<const h8_t *>(a_src[i] + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned at = (unsigned)min(4 * g + j, n64 - 1) * 1024u;
            w[j] = ONCE ? load16_once(b_rs, lane * 16u, at) : load16(b_rs, lane * 16u, at);
        }
        const unsigned ws = load4(bs_rs, lane * 4u, (unsigned)g * 256u);
#pragma unroll
        for (int i = 0; i < AL; ++i) {
            const int row = 2 * i + h;
            if constexpr (A4) {
                float v[8];
                unsigned top = 0, byte = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = (float)a[i][e];
                    top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
                }
                *reinterpret_cast<unsigned *>(mine + row * PITCH + 4 * r) = mx_encode8(v, top, &byte);
                // block r / 4 of the eight: half r / 4 % 2 of 64-block r / 8
                if ((r & 3) == 0) mine_s[row * 8 + 4 * (r >> 2 & 1) + (r >> 3)] = (uint8_t)byte;
            } else {
                *reinterpret_cast<h8_t *>(mine + row * PITCH + 16 * r) = a[i];
            }
        }
        wave_lds_sync();
        const unsigned char *const src = mine + (r % RT) * PITCH;
        const unsigned as = A4 ? *reinterpret_cast<const unsigned *>(mine_s + (r % RT) * 8 + 4 * h) : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (4 * g + j >= n64) break;                   // wave-uniform
            if constexpr (A4) {
                acc = mfma_fp4(*reinterpret_cast<const u4_t *>(src + 32 * j + 16 * h), w[j], acc, as, ws, j);
            } else {
                const float s = mx_scale(ws >> (8 * j) & 255u);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        *reinterpret_cast<const h8_t *>(src + 128 * j + 64 * h + 16 * e), mx_decode8(w[j][e], s), acc, 0,
                        0, 0);
            }
        }
        wave_lds_sync();
    }
    // rows 0 .. 7 of C: registers 0 .. 3 of both halves
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (4 * h + j < RT) sums[(wave * RT + 4 * h + j) * 32 + r] = acc[j];
    __syncthreads();
    const int m = threadIdx.x >> 3, col = 4 * (threadIdx.x & 7);
    if (m >= rt.n) return;
    Epilogue epi = p.epi;
    if (epi.bias) epi.bias += (size_t)rt.e * p.N;
    f4_t v[1] = {*reinterpret_cast<const f4_t *>(sums + m * 32 + col)};
#pragma unroll
    for (int k = 1; k < kDecodeWaves; ++k) v[0] += *reinterpret_cast<const f4_t *>(sums + (k * RT + m) * 32 + col);
    if ((p.N & 3) == 0) ColumnEpilogue<true>(epi, p.C, 32 * rt.tn + col, p.N).put(rt.s0, m, 1, rt.n, v);
    else ColumnEpilogue<false>(epi, p.C, 32 * rt.tn + col, p.N).put(rt.s0, m, 1, rt.n, v);
}

}  // namespace

namespace {

// ---------------------------------------------------------------------------
// Which kernel runs. Large tiles move fewer bytes into a CU for each matrix
// instruction; small ones, and more K groups in a workgroup, keep 256 CUs busy
// when C is small. Measured on an MI355X (us, M x K x N, the number of tiles
// in brackets; "64x128/4" is a tile with four K groups):
//   dense, fp16 activations  128x256     64x256      64x128/4    32x64/4     32x32/8
//   4096 x 4096 x 4096       110 [512]   122         173
//   2048 x 4096 x 4096       64.1 [256]  65.7 [512]  90.1
//   2048 x 9728 x 2560       118 [160]   115 [320]   129
//   512 x 4096 x 4096        53.5        40.0 [128]  25.4 [256]  35.8
//   128 x 2560 x 9728                    28.2        18.1 [152]  21.7 [608]  36.0
//   128 x 4096 x 4096                    37.2        19.6 [64]   12.3 [256]  18.8
//   32 x 2560 x 9728                                 14.5        10.8 [152]  16.2 [304]
//   64 x 4096 x 4096                                 18.8        11.8 [128]  10.2 [256]
//   dense, MXFP4 activations                         64x128/2
//   2048 x 9728 x 2560       59.2 [160]  70.5        69.2
//   512 x 4096 x 4096        28.2 [64]   22.0        17.3 [256]
// (a stage of the 128 x 256 tile takes more than twice as long with fp16
// activations, so a second round of such tiles costs more there. Not kept:
// 96 x 256 tiles, 2048 x 4096 x 11008 with MXFP4 activations 74.3 as with 128
// x 256, 16384 rows over 32 experts 144 against 132.)
//   32 experts of 2560 x 4096, fp16: rows of the average expert
//                            128x256     64x256      32x256      32x128/2    8 rows (decode)
//   512                      316         314         362         430
//   32                       75.3        54.3        53.3        55.9
//   16                       63.8        45.1        41.6        41.9
//   4                        52.5        34.8        28.2        24.8        41.9
//   1                        35.2        25.0        22.6        16.7        18.8
//   the same, MXFP4 activations
//   512                      152         174         221         289
//   128                      68.1        67.3        81.2        101
//   16                       41.5        35.9        36.9        37.4
//   8                        38.4        34.8        31.2        31.9        61.7
//   1                        18.6        16.3        15.8        16.0        18.5
// 32 x 256 tiles, one K group of four waves each, need two on a CU: 800 rows
// over 64 experts of 2560 x 640, 180 such tiles 24.1, 300 of 32 x 128 17.5 (18.0
// and 16.6 with MXFP4 activations); 300 rows over 16 of 9728 x 2560 73.5
// [170], 57.6. Over 37 layers of 2 to 256 experts the rules' choice is 2 %
// (MXFP4 activations: 1 %) above the best tile on average, 24 % at most.
// One token's 8 of 64 experts of 2560 x 2048: 8 rows (decode) 8.2, 2 rows 7.9.
// Split K (dense, few tiles) multiplies the workgroups by the slices of K; a
// second launch adds the slices up in their order and applies the epilogue.
// ---------------------------------------------------------------------------
template <MxShape SHAPE, class T>
hipError_t launch_tile(MxArgs p, hipStream_t s) {
    static_assert(T::BM == kMxTileRows[SHAPE] && T::BN == kMxTileCols[SHAPE] &&
                      T::THREADS == kMxTileThreads[T::A4][SHAPE],
                  "the shape the host counts with");
    p.tiles_n = div_up(p.N, T::BN);
    const long long grid = mx_row_tiles(p.S, p.offsets ? p.E : 1, T::BM) * p.tiles_n;
    hipLaunchKernelGGL(mx_tile_kernel<T>, dim3((unsigned)((grid + 7) / 8 * 8), (unsigned)p.nsplit), dim3(T::THREADS), 0,
                       s, p);
    return hipGetLastError();
}

template <bool A4, int RT, bool ONCE>
hipError_t launch_decode_rows(MxArgs p, hipStream_t s) {
    p.tiles_n = div_up(p.N, 32);
    const long long grid = mx_row_tiles(p.S, p.offsets ? p.E : 1, RT) * p.tiles_n;
    hipLaunchKernelGGL((mx_decode_kernel<A4, RT, ONCE>), dim3((unsigned)((grid + 7) / 8 * 8)),
                       dim3(64 * kDecodeWaves), 0, s, p);
    return hipGetLastError();
}

// Up to two rows a group (as far as the host can know): tiles of two rows.
template <bool A4>
hipError_t launch_decode(const MxArgs &p, hipStream_t s) {
    if (!p.offsets)
        return p.S <= 2 ? launch_decode_rows<A4, 2, true>(p, s) : launch_decode_rows<A4, 8, true>(p, s);
    return 4LL * p.S <= p.E ? launch_decode_rows<A4, 2, false>(p, s) : launch_decode_rows<A4, 8, false>(p, s);
}

template <bool A4>
hipError_t launch_shape(MxShape shape, const MxArgs &p, hipStream_t s) {
    switch (shape) {
    //                                       RF CF WM WN WK NS BR waves a SIMD
    case T128x256: return launch_tile<T128x256, Tile<A4, 4, 2, 1, 4, 1, 4, 2, 2>>(p, s);
    case T64x256:  return launch_tile<T64x256, Tile<A4, 2, 2, 1, 4, 1, 4, 2, 2>>(p, s);
    case T64x128:  return launch_tile<T64x128, Tile<A4, 2, 1, 1, 4, A4 ? 2 : 4, 4, 2, A4 ? 2 : 4>>(p, s);
    case T32x256:  return launch_tile<T32x256, Tile<A4, 1, 2, 1, 4, 1, 4, 2, 2>>(p, s);
    case T32x128:  return launch_tile<T32x128, Tile<A4, 1, 1, 1, 4, 2, 4, 2, 2>>(p, s);
    case T32x64:   return launch_tile<T32x64, Tile<A4, 1, 1, 1, 2, 4, 4, 2, 2>>(p, s);
    default:       return launch_tile<T32x32, Tile<A4, 1, 1, 1, 1, 8, 4, 2, 1>>(p, s);
    }
}

template <bool A4>
hipError_t launch_tiles(const MxArgs &args, hipStream_t s) {
    if (args.nsplit > 1) {
        MxArgs p = args;
        p.C = args.part;
        p.epi = Epilogue{nullptr, nullptr, QGEMM_ACT_NONE, 0, true};
        const hipError_t e = launch_shape<A4>(mx_dense_plan(A4, p.S, p.K, p.N).shape, p, s);
        return e != hipSuccess ? e : launch_splitk_reduce_f32(args.part, args.nsplit, p.S, p.N, args.C, args.epi, s);
    }
    return launch_shape<A4>(args.offsets ? mx_grouped_shape(A4, args.S, args.E, args.N)
                                         : mx_dense_plan(A4, args.S, args.K, args.N).shape,
                            args, s);
}

}  // namespace

hipError_t launch_mx_gemm(qgemm_format f, const MxArgs &args, bool decode, void *ws, hipStream_t s) {
    MxArgs p = args;
    if (f != QGEMM_MXFP4_A4) return decode ? launch_decode<false>(p, s) : launch_tiles<false>(p, s);
    if (decode) return launch_decode<true>(p, s);
    const MxWorkspace w = mx_workspace(f, p.a_rows, p.K);
    uint8_t *base = static_cast<uint8_t *>(ws);
    const hipError_t e = launch_mx_quantize_act(p.a_rows, p.K, p.A, base, base + w.s_off, s);
    if (e != hipSuccess) return e;
    p.Aq = base;
    p.As = base + w.s_off;
    return launch_tiles<true>(p, s);
}

}  // namespace qg
