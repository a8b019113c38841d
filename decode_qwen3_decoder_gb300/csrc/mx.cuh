// The microscaled (MX) matrix format and the conversions that its kernels share.
//
// A matrix [rows][cols] holds each run of 32 columns of a row as a power of two 2^e and 32 codes:
// e4m3 (8 bits, largest value 448) or e2m1 (4 bits, largest 6), e = min{e >= -127 : max|x| <= L 2^e}.
// Codes lie row by row, a row padded with zeros to a multiple of 128 columns. The exponents are bytes
// e + 127 (255: a run with a NaN or an infinity) in tiles of 128 rows by 4 runs, the order in which
// tcgen05.cp spreads a tile over tensor memory: byte 16 (r % 32) + 4 (r / 32 % 4) + run % 4.
#pragma once

#include "qw_internal.h"

// As in the 8-bit cache's kernels: every kernel is launched with programmatic stream serialization
// and each of its CTAs waits for the kernels before it (pdl_wait) before it reads anything or ends.

namespace {

constexpr int MX_RUN = 32;
constexpr int MX_ATOM = 128;        // columns of a scale tile, and the padding of a row
constexpr int MX_TILE_BYTES = 512;  // 128 rows x 4 runs

__host__ __device__ inline size_t mx_atoms(int cols) { return ((size_t)cols + MX_ATOM - 1) / MX_ATOM; }
__host__ __device__ inline size_t mx_row_bytes(int bits, int cols) { return mx_atoms(cols) * (MX_ATOM * bits / 8); }
// Offset of the four exponent bytes of a row's atom `ka` (columns 128 ka .. + 127).
__device__ __forceinline__ size_t mx_scale_word(int row, int ka, int atoms) {
    return ((size_t)(row >> 7) * atoms + ka) * MX_TILE_BYTES + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Bits of the largest magnitude (NaN and infinities above every number) to the run's exponent byte.
template <int BITS>
__device__ __forceinline__ int mx_exp_byte(uint32_t amax) {
    constexpr int S = BITS == 8 ? 8 : 2;                        // L = 1.75 * 2^8 or 1.5 * 2^2
    constexpr uint32_t M = BITS == 8 ? 0x600000u : 0x400000u;
    const int e = (int)(amax >> 23) - S + ((amax & 0x7FFFFFu) > M);
    return amax >= 0x7F800000u ? 255 : max(0, e);               // subnormals: byte 0, e = -127
}
// 2^-e of an exponent byte (0 for 255), and 2^e (NaN for 255).
__device__ __forceinline__ float mx_inv_scale(int byte) { return __int_as_float((254 - min(byte, 254)) << 23); }
__device__ __forceinline__ float mx_scale(int byte) {
    return __int_as_float(byte == 0 ? 0x400000 : byte == 255 ? 0x7FC00000 : byte << 23);
}

// 8 values already divided by their scale to codes, round to nearest even: 8 bytes (w[0], w[1]) or 4 (w[0]).
template <int BITS>
__device__ __forceinline__ void mx_enc8(const float* x, uint32_t* w) {
    if (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                "mov.b32 %0, {a, b};\n\t}"
                : "=r"(w[i])
                : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(w[0])
            : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
        w[1] = 0;
    }
}
// 8 codes to pairs of halves (exact).
template <int BITS>
__device__ __forceinline__ void mx_dec8(const uint32_t* w, uint32_t* h) {
    if (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 a, b;\n\t"
                "mov.b32 {a, b}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
                "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
                : "r"(w[i]));
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w[0]));
    }
}

// 32 bytes, 32-byte aligned: a whole sector.
__device__ __forceinline__ void mx_st32(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 8 elements of a row as they lie in memory: asked for first (vector loads of whole, 16-byte aligned groups), filled up
// where a row ends inside, unpacked last, so that many can be on their way at once.
struct MxRaw {
    uint4 a, b;  // b: of QW_F32 only
};
template <int DT>
__device__ __forceinline__ MxRaw mx_fetch8(const void* base, size_t off, int left) {
    MxRaw r = {};
    if (left >= 8) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + off * (DT == QW_F32 ? 4 : 2));
        r.a = p[0];
        if (DT == QW_F32) r.b = p[1];
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void mx_fill8(const void* base, size_t off, int left, MxRaw& r) {
    if (left <= 0 || left >= 8) return;
    uint32_t w[8] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) {
            if (DT == QW_F32) w[i] = reinterpret_cast<const uint32_t*>(base)[off + i];
            else w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(base)[off + i] << (i % 2 * 16);
        }
    r = {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
template <int DT>
__device__ __forceinline__ void mx_unpack8(const MxRaw& r, float* x) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = DT == QW_F32    ? __uint_as_float(w[i])
               : DT == QW_BF16 ? (i % 2 ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]))
                               : (i % 2 ? h_hi(w[i / 2]) : h_lo(w[i / 2]));
}
// Bits, as a float's, of the largest magnitude of 8 elements; NaN and infinities are above every number. 16-bit
// elements are compared in pairs, as integers.
template <int DT>
__device__ __forceinline__ uint32_t mx_absmax8(const MxRaw& r) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = DT == QW_F32 ? max(m, w[i] & 0x7FFFFFFFu) : i < 4 ? __vmaxu2(m, w[i] & 0x7FFF7FFFu) : m;
    if (DT == QW_F32) return m;
    m = max(m & 0xFFFFu, m >> 16);
    return DT == QW_BF16 ? m << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) & 0x7FFFFFFFu;
}
template <int DT>
__device__ __forceinline__ void mx_load8(const void* base, size_t off, int left, float* x) {
    MxRaw r = mx_fetch8<DT>(base, off, left);
    mx_fill8<DT>(base, off, left, r);
    mx_unpack8<DT>(r, x);
}

// fp16 results stop at 65504, as those of the 8-bit cache do; NaN stays.
__device__ __forceinline__ float mx_sat16(float v) { return fabsf(v) > 65504.f ? copysignf(65504.f, v) : v; }

// Two elements of type DT (16 bits) as a word.
template <int DT, bool SAT = true>
__device__ __forceinline__ uint32_t mx_pack2(float a, float b) {
    return DT == QW_F16 ? SAT ? pack_h2(mx_sat16(a), mx_sat16(b)) : pack_h2(a, b) : pack_bf2(a, b);
}

// 8 elements to `off`, the first `left` of them. SAT false: values of the type itself, infinities among them.
template <int DT, bool SAT = true>
__device__ __forceinline__ void mx_store8(void* base, size_t off, int left, const float* x) {
    if (left >= 8) {
        if (DT == QW_F32) {
            float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + off) =
                make_uint4(mx_pack2<DT, SAT>(x[0], x[1]), mx_pack2<DT, SAT>(x[2], x[3]), mx_pack2<DT, SAT>(x[4], x[5]), mx_pack2<DT, SAT>(x[6], x[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < left) {
                if (DT == QW_F32) reinterpret_cast<float*>(base)[off + i] = x[i];
                else reinterpret_cast<uint16_t*>(base)[off + i] = (uint16_t)mx_pack2<DT, SAT>(x[i], 0.f);
            }
        }
    }
}

}  // namespace

// Host-side check of a matrix; QW_OK or the recorded error. A matrix without rows may have no memory.
qw_status mx_check(const qw_mx* m, const char* what, const char* name);

// Memory of an operand: `rows` of `len` bytes, `step` bytes apart.
struct MxSpan {
    uintptr_t at;
    size_t rows, len, step;
};
inline MxSpan mx_rows_span(const void* p, int rows, int cols, size_t ld, int dtype) {
    const size_t es = dtype == QW_F32 ? 4 : 2;
    return {(uintptr_t)p, p ? (size_t)rows : 0, cols * es, ld * es};
}
// Whether two operands share a byte. Rows may lie between another's rows (column slices of one buffer, which have one
// step); of two operands with gaps and different steps it is not looked at.
bool mx_meet(const MxSpan& a, const MxSpan& b);
// The same of an operand and a matrix's codes and exponents, and of two matrices.
bool mx_meet(const qw_mx& m, const MxSpan& b);
bool mx_meet(const qw_mx& a, const qw_mx& b);
