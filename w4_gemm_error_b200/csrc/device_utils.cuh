// Small device helpers shared by the kernels of libspear_w4ec (sm_100a).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace spear {

// Sticky status bits written by kernels into the handle's device status word.
enum : int { kStatusNonFinite = 1, kStatusTimeout = 2 };

__device__ __forceinline__ uint32_t lop3_and_or(uint32_t a, uint32_t b, uint32_t c)
{
    // (a & b) | c
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// d = a * b + c on bf16x2 (round to nearest); exact when the result is a small integer.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Stored nibble order of a code word (the tiled layout on the device): the
// codes of k = 8j + {0, 2, 4, 6} sit in nibbles 0..3 and those of k = 8j +
// {1, 3, 5, 7} in nibbles 4..7, so that the nibble pair (m, m + 4), 16 bits
// apart, is the consecutive pair k = 8j + 2m, 8j + 2m + 1.  Bit offset of the
// code of k = 8j + i:
__host__ __device__ constexpr int nibble_shift(int i) { return 4 * ((i & 1) * 4 + (i >> 1)); }

// Two int4 codes, the nibbles at bit positions `sh` and `sh + 16` of w, as a
// bf16x2 pair of exact integers (q_lo - zp, q_hi - zp).  The nibble is placed
// in the low mantissa bits of 128.0 (0x4300), giving 128 + q exactly; the fma
// then subtracts 128 + zp, which is exact because the result is an integer
// of magnitude <= 15.  neg_bias = bf16x2(-(128 + zp), -(128 + zp)).
__device__ __forceinline__ uint32_t dequant_pair(uint32_t w_shifted, uint32_t neg_bias)
{
    const uint32_t t = lop3_and_or(w_shifted, 0x000F000Fu, 0x43004300u);
    return fma_bf16x2(t, 0x3F803F80u /* (1.0, 1.0) */, neg_bias);
}

// As dequant_pair with a per-row multiplier: mul = bf16x2(1, 1) with neg_bias
// as above, or mul = neg_bias = 0 for a row whose scale is 0 (its weights are
// 0 whatever its codes say), for a kernel that applies a stand-in scale of 1
// to such rows after accumulating.
__device__ __forceinline__ uint32_t dequant_pair_mul(uint32_t w_shifted, uint32_t mul, uint32_t neg_bias)
{
    const uint32_t t = lop3_and_or(w_shifted, 0x000F000Fu, 0x43004300u);
    return fma_bf16x2(t, mul, neg_bias);
}

// The eight codes of a stored word as e4m3, k = 8j + {0..3} in lo and + {4..7}
// in hi (one code a byte).  No arithmetic is needed: e4m3 counts linearly from
// zero in steps of 2^-9 up to 2^-5 (its subnormals and its first binade have
// the same spacing), so the byte 0x0q IS the value 2^-9 q.  nib = 0x0F0F0F0F,
// or 0 for a row whose weights are all 0.
__device__ __forceinline__ void nibbles_to_e4m3(uint32_t w, uint32_t nib, uint32_t &lo, uint32_t &hi)
{
    const uint32_t a = w & nib, b = (w >> 4) & nib;   // bytes: codes 0, 4, 1, 5 and 2, 6, 3, 7
    lo = prmt(a, b, 0x6420);
    hi = prmt(a, b, 0x7531);
}

// D (16x8 fp32) += A (16x16 bf16, row) * B (16x8 bf16, col).  Not volatile: its
// only effect is on d, so the compiler may interleave independent MMAs.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with f16 operands.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As dequant_pair, in f16: the nibble in the low mantissa bits of 1024.0
// (0x6400) is 1024 + q, and subtracting 1024 + zp is exact.
__device__ __forceinline__ uint32_t dequant_pair_f16(uint32_t w_shifted, uint32_t neg_bias)
{
    const uint32_t t = lop3_and_or(w_shifted, 0x000F000Fu, 0x64006400u);
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(t), "r"(neg_bias));
    return d;
}

// The three of them in the type of the activations' pairs: f16 (F16) or bf16.
template <bool F16>
__device__ __forceinline__ uint32_t dequant_bias(uint32_t zp)
{
    const uint32_t b = F16 ? 0x8000u | (0x6400u + zp)   // -(1024 + zp): an f16 there counts in ones
                           : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(-(float)(128u + zp)));
    return b | (b << 16);
}
template <bool F16>
__device__ __forceinline__ uint32_t dequant(uint32_t w_shifted, uint32_t neg_bias)
{
    if constexpr (F16)
        return dequant_pair_f16(w_shifted, neg_bias);
    else
        return dequant_pair(w_shifted, neg_bias);
}
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
    else
        mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}

// Loads through the read-only path (ld_stream, ld_nc and __ldg): for the layer's own
// weights alone.  The path is for memory that nothing writes while the kernel
// runs, and a kernel launched with programmatic serialization runs beside the
// earlier ones that write its operands; the compiler may also move such a load
// above the wait for them.  Operands take plain loads, or ld_settled.

// Streaming 16-byte load that is read once (no L1 allocation).
__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 ld_nc(const void *p)
{
    return __ldg(reinterpret_cast<const uint4 *>(p));
}

// Programmatic dependent launch: let the next kernel in the stream start, and
// wait for the previous kernel's results (no-ops without the launch attribute).
__device__ __forceinline__ void pdl_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// An operand's address after pdl_wait(): loads through it come after the wait,
// and may otherwise be moved freely by the compiler (a plain load may not pass
// the stores before it).
template <class T>
__device__ __forceinline__ const T *settled(const T *p)
{
    asm volatile("" : "+l"(p)::"memory");
    return p;
}
__device__ __forceinline__ uint4 ld_settled(const void *p)
{
    uint4 v;
    asm("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_settled8(const void *p)
{
    uint2 v;
    asm("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// fp32 rounded to the tf32 grid (10 explicit mantissa bits, round to nearest, ties away).
__device__ __forceinline__ float to_tf32(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return __uint_as_float(r);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two fp32 values as e4m3 (round to nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two e4m3 values (low byte first) as f16x2: every e4m3 value, NaN included, is one of f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
    return d;
}

// The four e4m3 values of a word as bf16, in order.  Moved to the low bits of a
// bf16's exponent and the high ones of its mantissa they are 2^-120 times their
// value, subnormals included, and the product with 2^120 is exact.  (The
// conversion instructions run at a quarter of this rate or less.)  A NaN comes
// out as +-480: for sums beside a product of the same values that keeps NaNs.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t a = prmt(w, 0u, 0x1404), b = prmt(w, 0u, 0x3424);   // a value in the high byte of each half
    const uint32_t x = ((a >> 4) & 0x07F007F0u) | (a & 0x80008000u);
    const uint32_t y = ((b >> 4) & 0x07F007F0u) | (b & 0x80008000u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x7B807B80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x7B807B80u));
}

// f16x2 as bf16x2; exact for values that came from e4m3 (four significant bits).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t v)
{
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
    return pack_bf16x2(lo, hi);
}

}  // namespace spear
