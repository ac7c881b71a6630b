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
// (offsets[0 .. E]); a row tile holds up to BM slots of one group. offsets ==
// nullptr: one group of all S rows. Every offset is limited to [0, S],
// whatever the array holds.
//
// Order of the output tiles: group by group; within a group by bands of up to
// kBand row tiles, in a band column by column, the band's row tiles of one
// column in a row. The hardware deals workgroups to the eight XCDs in turn,
// and each XCD has its own L2; XCD x takes the x-th eighth of that order, so
// the workgroups that run on it together read the same few weight columns and
// the same rows, and each weight is fetched by one XCD. (The eighths are of
// the tiles that exist, which only the GPU knows.) Measured against plain
// order with MXFP4 activations: 2048 x 4096 x 11008 in 64 x 256 tiles 134 ->
// 102 us; bands of 1, 4 and 16: 128, 105, 101 us there, and 4096^3 with fp16
// activations 120, 117, 120 us.
// ---------------------------------------------------------------------------
struct RowTile {
    int e;        // group; -1: nothing to do
    int s0, n;    // first slot and number of slots
    int tn;       // column tile
};

constexpr int kBand = 4;

// Tile i of a group of slots [lo, hi), as above.
__device__ __forceinline__ RowTile tile_of_group(int e, int lo, int hi, int BM, int tiles_n, int i) {
    const int cnt = (hi - lo + BM - 1) / BM;
    const int band = i / (kBand * tiles_n), rest = i - band * (kBand * tiles_n);
    const int rows = min(kBand, cnt - band * kBand);
    const int tn = rest / rows, s0 = lo + (band * kBand + rest - tn * rows) * BM;
    return RowTile{e, s0, min(BM, hi - s0), tn};
}

// Inclusive sum over the 64 lanes: within rows of 16 lanes, then row 0's (and
// 2's) total into the next row, then the lower half's into the upper. (With
// shuffles through LDS, dependent round trips, finding its tile took a
// workgroup 2.0 us at 16384 rows over 32 groups; so it takes 1.2.)
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);     // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);     // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);     // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);     // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);     // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);     // row_bcast:31 into rows 2 and 3
    return v;
}

// The tile of workgroup L of a launch of 8 * per-XCD workgroups, found by the
// whole wave (every wave of a workgroup does so for itself): each lane counts
// one group's row tiles, a scan over the lanes adds them up, 64 groups at a
// time.
__device__ __forceinline__ RowTile find_tile(const int32_t *__restrict__ offsets, int E, int S, int BM, int tiles_n,
                                             int L) {
    const int x = L & 7, idx = L >> 3;
    if (!offsets) {
        const int total = (S + BM - 1) / BM * tiles_n, per = (total + 7) >> 3, q = x * per + idx;
        return idx < per && q < total ? tile_of_group(0, 0, S, BM, tiles_n, q) : RowTile{-1, 0, 0, 0};
    }
    const int lane = threadIdx.x & 63;
    int lo, hi, nt, upto;                 // of group e0 + lane; row tiles of groups e0 .. e0 + lane
    auto count = [&](int e0) {
        const int e = min(e0 + lane, E - 1);
        lo = min(max(offsets[e], 0), S);
        hi = min(max(offsets[e + 1], lo), S);
        nt = e0 + lane < E ? (hi - lo + BM - 1) / BM : 0;
        upto = wave_scan(nt);
    };
    int all = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        count(e0);
        all += __builtin_amdgcn_readlane(upto, 63);
    }
    const int total = all * tiles_n, per = (total + 7) >> 3, q = x * per + idx;
    if (idx >= per || q >= total) return RowTile{-1, 0, 0, 0};
    int before = 0;                       // row tiles of the groups already passed
    for (int e0 = 0; e0 < E; e0 += 64) {
        if (E > 64) count(e0);
        const unsigned long long past = __ballot((before + upto) * tiles_n > q);
        if (past) {
            const int src = __ffsll((long long)past) - 1;
            const int first = before + __builtin_amdgcn_readlane(upto - nt, src);     // row tiles before group src
            const int i = q - first * tiles_n;
            // (offsets that fall can make the sums above pass 32 bits; one group's tiles do not)
            if (i < 0 || i >= __builtin_amdgcn_readlane(nt, src) * tiles_n) return RowTile{-1, 0, 0, 0};
            return tile_of_group(e0 + src, __builtin_amdgcn_readlane(lo, src), __builtin_amdgcn_readlane(hi, src), BM,
                                 tiles_n, i);
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return RowTile{-1, 0, 0, 0};
}

}  // namespace qg
