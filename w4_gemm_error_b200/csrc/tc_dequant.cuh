// Dequantising warps of the tcgen05 kernels with an epilogue (tc_pair.cu and
// tc_tile.cu): 4-bit codes from global memory into registers, from there as
// bf16 (form kEpi) or e4m3 (kQ8) into a 128-row, 128-byte-wide K-major operand
// tile with the 128-byte swizzle.  Four warps take a stage (32 rows each).
#pragma once
#include <cstdint>

#include "device_utils.cuh"
#include "epilogue.cuh"

namespace spear {

constexpr int kTcRowBytes = 128;   // a stage's k of one row of either operand
// k per stage: 64 bf16 or (form kQ8) 128 e4m3 values; stages per tiled block of 256 k
__host__ __device__ constexpr int tc_stage_k(int form) { return form == kQ8 ? 128 : 64; }
__host__ __device__ constexpr int tc_stages_per_block(int form) { return 256 / tc_stage_k(form); }

// A thread's share of a stage: kPieces 16-byte pieces (32 codes) of as many
// rows, the lanes of a row side by side so that a warp's load is whole sectors.
// Form kQ8 (64 bytes a row): piece lane % 4 of rows lane / 4 + 8 j; kEpi
// (32 bytes a row): piece lane % 2 of rows lane / 2 + 16 j.
template <int FORM>
struct TcDequant {
    static constexpr int kLanes = FORM == kQ8 ? 4 : 2;    // lanes a row
    static constexpr int kPieces = FORM == kQ8 ? 4 : 2;   // pieces (rows) a thread
    static constexpr int kOut = FORM == kQ8 ? 2 : 4;      // 16-byte operand pieces of 32 codes
    static constexpr int kRowStep = 32 / kLanes;          // rows between a thread's pieces

    int piece, r0;                          // this thread's piece and first row (of the 128)
    uint32_t mul[kPieces], neg[kPieces];    // kQ8: nibble mask; kEpi: factor and bias of a row's pairs
    uint4 codes[kPieces];
    uint4 out[kPieces][kOut];

    __device__ __forceinline__ TcDequant(int warp4, int lane) : piece(lane % kLanes), r0(32 * warp4 + lane / kLanes) {}

    // The rows n0 .. n0 + 127.  A row whose s is 0 has weights 0, whatever its
    // codes (the epilogue scales it by 1).
    __device__ __forceinline__ void set_rows(const float *s, const uint8_t *z, int64_t n0, int64_t Np)
    {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int64_t n = n0 + r0 + j * kRowStep;
            const bool live = n < Np && __ldg(s + n) != 0.0f;
            if constexpr (FORM == kQ8) {
                mul[j] = live ? 0x0F0F0F0Fu : 0u;
            } else {
                mul[j] = live ? 0x3F803F80u : 0u;
                neg[j] = live ? dequant_bias<false>(__ldg(z + n)) : 0u;
            }
        }
    }

    // Byte offset of this thread's codes in a 64-row block row of the tiled codes.
    __device__ __forceinline__ int64_t offset() const { return (int64_t)(r0 & 63) * 128 + piece * 16; }

    // The codes of stage st; src: this thread's place in its 64-row block row (null: zeros).
    __device__ __forceinline__ void fetch(const uint8_t *src, int st)
    {
        constexpr int SUB = tc_stages_per_block(FORM);
        const uint8_t *at = src + (int64_t)(st / SUB) * 8192 + (st % SUB) * (tc_stage_k(FORM) / 2);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            codes[j] = src ? ld_stream(at + j * kRowStep * 128) : make_uint4(0u, 0u, 0u, 0u);
    }

    __device__ __forceinline__ void convert()
    {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const uint32_t words[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
            if constexpr (FORM == kQ8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    nibbles_to_e4m3(words[2 * h], mul[j], out[j][h].x, out[j][h].y);
                    nibbles_to_e4m3(words[2 * h + 1], mul[j], out[j][h].z, out[j][h].w);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    out[j][h].x = dequant_pair_mul(words[h], mul[j], neg[j]);
                    out[j][h].y = dequant_pair_mul(words[h] >> 4, mul[j], neg[j]);
                    out[j][h].z = dequant_pair_mul(words[h] >> 8, mul[j], neg[j]);
                    out[j][h].w = dequant_pair_mul(words[h] >> 12, mul[j], neg[j]);
                }
            }
        }
    }

    // Into the operand tile at `at` (conflict-free: eight lanes cover the eight
    // 16-byte places of a 128-byte line).
    __device__ __forceinline__ void store(uint8_t *at) const
    {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int row = r0 + j * kRowStep;
#pragma unroll
            for (int h = 0; h < kOut; ++h)
                *reinterpret_cast<uint4 *>(at + row * kTcRowBytes + (((kOut * piece + h) ^ (row & 7)) << 4)) =
                    out[j][h];
        }
    }
};

}  // namespace spear
