// mx_common.h -- MXFP4 device helpers shared by the conversions and the
// products.
#pragma once

#include "kernels_common.h"

namespace qg {

// E8M0 byte -> fp32: 2^(byte - 127), where byte 0 is the subnormal 2^-127 and
// byte 255 is NaN.
__device__ __forceinline__ float mx_scale(unsigned byte) {
    const unsigned u = byte << 23;
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : u);
}

// Eight codes (one word, ascending, low nibble first) x scale as fp16, each
// rounded once to nearest even (exact for scales from 2^-23 to 2^13).
__device__ __forceinline__ h8_t mx_decode8(unsigned word, float s) {
    const h2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, s, 0);
    const h2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, s, 1);
    const h2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, s, 2);
    const h2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, s, 3);
    return h8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// This lane's 8 elements of a 32-element block that four neighbouring lanes
// (of one aligned group of four) hold, to a code word; `top` is the largest
// magnitude of the eight as fp32 bits (an infinity or NaN is largest of all).
// *byte gets the block's scale byte. All four lanes must be active.
__device__ __forceinline__ unsigned mx_encode8(const float (&v)[8], unsigned top, unsigned *byte) {
    top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true));   // lane ^ 2
    const unsigned E = top >> 23;
    const unsigned b = E == 255 ? 255u : E > 2 ? E - 2 : 0u;
    *byte = b;
    const float s = mx_scale(b == 255 ? 127u : b);
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    return b == 255 ? 0u : w;
}

// ---------------------------------------------------------------------------
// Groups of rows. A product's slots [0, S) fall into E consecutive groups
// (offsets[0 .. E]); a row tile holds up to BM slots of one group, and the
// tiles are numbered through all groups. offsets == nullptr: one group of all
// S rows. Every offset is limited to [0, S], whatever the array holds.
// ---------------------------------------------------------------------------
struct RowTile {
    int e;        // group; -1 past the last tile
    int s0, n;    // first slot and number of slots
};

// Row tile `tile`, found by the whole wave (every wave of a workgroup does so
// for itself): each lane counts one group's tiles, a scan over the lanes adds
// them up, 64 groups at a time.
__device__ __forceinline__ RowTile find_row_tile(const int32_t *__restrict__ offsets, int E, int S, int BM,
                                                 int tile) {
    if (!offsets) {
        const int s0 = tile * BM;
        return s0 < S ? RowTile{0, s0, min(BM, S - s0)} : RowTile{-1, 0, 0};
    }
    const int lane = threadIdx.x & 63;
    int before = 0;                       // tiles of the groups already passed
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < E) {
            lo = min(max(offsets[e], 0), S);
            hi = min(max(offsets[e + 1], lo), S);
        }
        const int nt = (hi - lo + BM - 1) / BM;
        int upto = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(upto, d);
            if (lane >= d) upto += x;
        }
        const unsigned long long past = __ballot(before + upto > tile);
        if (past) {
            const int src = __ffsll((long long)past) - 1;
            const int first = before + __shfl(upto - nt, src);     // tiles before group src
            const int s0 = __shfl(lo, src) + (tile - first) * BM;
            return RowTile{uniform(e0 + src), uniform(s0), uniform(min(BM, __shfl(hi, src) - s0))};
        }
        before += __shfl(upto, 63);
    }
    return RowTile{-1, 0, 0};
}

}  // namespace qg
