// Microscaled matrices: quantisation of rows (qw_mx_quantize), their values (qw_mx_read) and RMSNorm with
// the branch's addition and a quantised output (qw_mx_rmsnorm). mx.cuh states the format.
//
// Quantise. A thread has 8 columns of a run of 32, or 16 in a large matrix, where the instructions around the values
// would otherwise bound the kernel (ALU: 69 of 132 instructions a thread's 8 values). The exponent follows from the
// largest magnitude alone and x 2^-e is exact, so the codes are those of the definition bit for bit. Read. A thread
// has 8 columns; a warp of a large matrix asks for four pieces of 256 before it uses one. Bytes bound both: 151936 x 1024
// from bf16 to 4 bits 64 us, 6.1 TB/s, and back 67 us.
//
// RMSNorm. s = x + add rounded to the stream's type, y = s / sqrt(mean(s^2) + eps) * w, codes of y. y has no
// type of its own: the codes are those of the real y, whatever the order of the sums. y is computed in fp32 with a
// relative error d below 18 2^-24; a run in which a value between y (1 - d) and y (1 + d) could get another code or
// exponent, one in 1300, is computed again: the row's sum of squares as an unevaluated pair of floats (the
// products' and sums' errors are added up, by Dekker's and Knuth's methods), 1 / sqrt and the products as pairs, 2^-43 in all.
// Where fp32 cannot hold the pairs (runs below 2^-30, weights above 2^50) the products are in 64 bits, and so is a whole row whose
// squares leave fp32. (1 / sqrt in fp64, whose rate is low here: 2048 x 8192 35.0 us, as pairs 31.2.)
// 8192 x 1024 fp32 with a bf16 branch 17.1 us, 92 MB (bytes alone 13.6); 2048 x 4096 18.2, 88 MB (13.0); bf16 with a bf16 branch
// 17.3. Neither bytes nor instructions fill it: 43 instructions an element take 67% (half at 4096 columns) of the issue slots, and a
// warp waits, in this order, for its row's loads, for shuffles and conversions, and at the row's two barriers, with 65% (45%) of
// the warps that fit. Pairs for every value would double the instructions; persistent CTAs that had the next row copied ahead took 22.3 us.
// One CTA a row (up to 256 columns one warp); up to 16384 columns a row's elements stay in registers between the passes. Longer rows
// are read twice and summed in pairs: 1024 x 20000 bf16 with a bf16 branch 52 us, 225 MB with the second reading (33).
#include <algorithm>

#include "mx.cuh"

namespace {

constexpr int MQ_WARPS = 8;

// The bytes of four runs as a word, in the first lane of each group that has 128 columns, V a lane.
template <int V>
__device__ __forceinline__ uint32_t mx_gather_word(int byte) {
    uint32_t w = (uint32_t)byte;
    w |= __shfl_down_sync(0xffffffffu, w, 32 / V) << 8;
    return w | (__shfl_down_sync(0xffffffffu, w, 64 / V) << 16);
}

// A warp's pieces of 32 V columns in row order: one division, then steps.
template <int V>
struct Piece {
    int row, c;  // this lane's first column
    __device__ __forceinline__ Piece(unsigned u, unsigned per_row, int lane) : row((int)(u / per_row)), c((int)(u % per_row) * 32 * V + lane * V) {}
    __device__ __forceinline__ void next(unsigned per_row, int lane) {
        c += 32 * V;
        if (c >= (int)per_row * 32 * V) c = lane * V, ++row;
    }
};

struct MxRowsP {
    uint8_t* codes;
    uint8_t* scales;
    int rows, cols, atoms;
    const void* src;
    void* dst;
    size_t ld;
    unsigned units, per_row;  // warps' pieces
};

template <int DT, int BITS, int V>
__global__ void __launch_bounds__(MQ_WARPS * 32) k_mx_quantize(const __grid_constant__ MxRowsP p) {
    constexpr int G = V / 8;  // groups of 8 columns a lane
    pdl_wait();
    pdl_launch();
    const unsigned u = blockIdx.x * MQ_WARPS + (threadIdx.x >> 5);
    if (u >= p.units) return;
    const int lane = threadIdx.x & 31;
    const Piece<V> t(u, p.per_row, lane);
    const size_t from = (size_t)t.row * p.ld + t.c;
    const int left = p.cols - t.c;
    MxRaw raw[G];
#pragma unroll
    for (int g = 0; g < G; ++g) raw[g] = mx_fetch8<DT>(p.src, from + 8 * g, left - 8 * g);
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        mx_fill8<DT>(p.src, from + 8 * g, left - 8 * g, raw[g]);
        m = max(m, mx_absmax8<DT>(raw[g]));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (V == 8) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int byte = mx_exp_byte<BITS>(m);
    const float inv = mx_inv_scale(byte);
    uint32_t w[2 * G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float x[8];
        mx_unpack8<DT>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
        mx_enc8<BITS>(x, w + g * (BITS / 4));
    }
    const uint32_t sw = mx_gather_word<V>(byte);
    if (t.c >= p.atoms * MX_ATOM) return;
    uint8_t* at = p.codes + (size_t)t.row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)t.c * BITS / 8;
    if (V * BITS == 128) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2 * G - 2], w[2 * G - 1]);
    else if (V * BITS == 64) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(at) = w[0];
    if (lane % (128 / V) == 0) *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(t.row, t.c / MX_ATOM, p.atoms)) = sw;
}

// U neighbouring pieces a warp.
template <int DT, int BITS, int U>
__global__ void __launch_bounds__(MQ_WARPS * 32) k_mx_read(const __grid_constant__ MxRowsP p) {
    pdl_wait();
    pdl_launch();
    const unsigned u0 = (blockIdx.x * MQ_WARPS + (threadIdx.x >> 5)) * U;
    const int lane = threadIdx.x & 31;
    const Piece<8> first(u0, p.per_row, lane);
    Piece<8> t = first;
    uint32_t w[U][2];
    uint8_t e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        w[k][0] = w[k][1] = 0;
        e[k] = 0;
        if (u0 + k < p.units && t.c < p.cols) {
            const uint8_t* at = p.codes + (size_t)t.row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)t.c * BITS / 8;
            if (BITS == 8) {
                const uint2 v = *reinterpret_cast<const uint2*>(at);
                w[k][0] = v.x, w[k][1] = v.y;
            } else {
                w[k][0] = *reinterpret_cast<const uint32_t*>(at);
            }
            e[k] = p.scales[mx_scale_word(t.row, t.c / MX_ATOM, p.atoms) + (t.c / MX_RUN & 3)];
        }
        t.next(p.per_row, lane);
    }
    t = first;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (u0 + k < p.units && t.c < p.cols) {
            uint32_t h[4];
            mx_dec8<BITS>(w[k], h);
            const float s = mx_scale(e[k]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = h_lo(h[i]) * s;
                x[2 * i + 1] = h_hi(h[i]) * s;
            }
            mx_store8<DT>(p.dst, (size_t)t.row * p.ld + t.c, p.cols - t.c, x);
        }
        t.next(p.per_row, lane);
    }
}

// ---- RMSNorm --------------------------------------------------------------------------------------------

// A sum as an unevaluated pair: hi + lo.
struct Pair {
    float hi, lo;
};

struct MxNormP {
    uint8_t* codes;
    uint8_t* scales;
    int rows, cols, atoms;
    const void* x;
    const void* add;
    void* sum;
    const bf16* w;
    size_t ld_x, ld_add, ld_sum;
    int dt_add;  // QW_F16, QW_BF16, QW_F32 or -1
    float eps;
    Pair inv_n;  // 1 / cols
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ void add_square(Pair& t, float v) {
    const float q = __fmul_rn(v, v);
    const Pair s = two_sum(t.hi, q);
    t.hi = s.hi;
    t.lo = __fadd_rn(t.lo, __fadd_rn(s.lo, __fmaf_rn(v, v, -q)));
}
__device__ __forceinline__ Pair add_pairs(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s.hi, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}

// A sum as DT holds it: fp16 stops at 65504, but an infinity that was there before stays one.
template <int DT>
__device__ __forceinline__ float round_to(float v) {
    if (DT == QW_F16) return __half2float(__float2half_rn(fabsf(v) <= 3.402823466e38f ? mx_sat16(v) : v));
    if (DT == QW_BF16) return bf2f(__float2bfloat16_rn(v));
    return v;
}

// hi + lo to the float that rounds like it to fewer bits: towards zero, the last bit set if inexact. |lo| is at most
// half a unit of hi's last place.
__device__ __forceinline__ float to_odd(Pair t) {
    if (t.lo == 0.f) return t.hi;
    const uint32_t u = __float_as_uint(t.hi);
    return __uint_as_float(((t.lo < 0.f) != (t.hi < 0.f) ? u - 1 : u) | 1u);
}
__device__ __forceinline__ float to_odd(double t) {
    const float f = __double2float_rz(t);
    return (double)f == t ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// s r w to 2^-45, r = 1 / sqrt as a pair, of what norm_codes lets through: the products' rests are fp32 numbers there.
__device__ __forceinline__ Pair scale_pair(float s, Pair r, float w) {
    const float a = __fmul_rn(s, r.hi), b = __fmaf_rn(s, r.lo, __fmaf_rn(s, r.hi, -a));
    const float q = __fmul_rn(a, w), f = __fmaf_rn(b, w, __fmaf_rn(a, w, -q));
    const float hi = __fadd_rn(q, f);
    return {hi, __fsub_rn(f, __fsub_rn(hi, q))};
}

// 1 / sqrt(t inv_n + eps): one step of third order from an fp32 value r0 (2^-22), whose residual 1 - a r0^2 is taken from
// exact products: 2^-44.
__device__ __forceinline__ Pair refine_rsqrt(Pair t, Pair inv_n, float eps, float r0) {
    const float m = __fmul_rn(t.hi, inv_n.hi);
    const float ml = __fmaf_rn(t.hi, inv_n.lo, __fmaf_rn(t.lo, inv_n.hi, __fmaf_rn(t.hi, inv_n.hi, -m)));
    const Pair a = add_pairs({m, ml}, {eps, 0.f});
    const float q = __fmul_rn(r0, r0), ql = __fmaf_rn(r0, r0, -q);
    const float b = __fmul_rn(a.hi, q), bl = __fmaf_rn(a.lo, q, __fmaf_rn(a.hi, ql, __fmaf_rn(a.hi, q, -b)));
    const float e = __fsub_rn(__fsub_rn(1.f, b), bl);
    const float d = __fmul_rn(__fmul_rn(r0, e), __fmaf_rn(0.375f, e, 0.5f));
    const float hi = __fadd_rn(r0, d);
    return {hi, __fsub_rn(d, __fsub_rn(hi, r0))};
}

// Roundings of y, in units of 2^-24: s rstd, times w, times the scale 1 each; rsqrtf 4 (2 units of the last place); its
// argument 1 (two, halved by the root); the sum of squares at most 16 on the way of a term (see k_mx_rmsnorm), halved.
constexpr float NORM_LO = 1.f - 0x1.2p-20f, NORM_HI = 1.f + 0x1.2p-20f;

// Codes and exponent byte of 8 columns from fp32 values; the whole warp calls, with rstd 0 for padding. again: this thread's
// part of the run has to be computed again, as another code or exponent is possible (NORM_DOUBT) or as fp32 does not hold what
// its products need (NORM_WIDE). Where the run's largest |y| is at least 2^-30 and no weight above 2^50, a |y| that does not
// round to 0 (2^-19 of the largest, or more) has an |s| rstd of 2^-99 or more, normal with 24 bits to spare, and none nears fp32's end.
enum : int { NORM_DOUBT = 1, NORM_WIDE = 2 };
template <int BITS>
__device__ __forceinline__ int norm_codes(const float* s, const float* w, float rstd, uint32_t* codes, int& again) {
    float y[8], top = 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = s[i] * rstd * w[i];
        m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
        top = fmaxf(top, fabsf(w[i]));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int byte = mx_exp_byte<BITS>(m);
    // the largest next to L 2^e (d of 1.75 is 16 units of the mantissa)
    constexpr uint32_t M = BITS == 8 ? 0x600000u : 0x400000u;
    again = ((m - M + 16u) & 0x7FFFFFu) <= 32u ? NORM_DOUBT : 0;
    const float inv = mx_inv_scale(byte);
    const float lo = inv * NORM_LO, hi = inv * NORM_HI;
    float a[8];
    uint32_t cb[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = y[i] * lo;
    mx_enc8<BITS>(a, codes);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = y[i] * hi;
    mx_enc8<BITS>(a, cb);
    if (codes[0] != cb[0] || codes[1] != cb[1]) again = NORM_DOUBT;
    if (top > 0x1p50f) again = NORM_WIDE;
    if (m < 0x30800000u) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s[i] != 0.f && w[i] != 0.f) again = NORM_WIDE;
    }
    return byte;
}

// The same from pairs: r = 1 / sqrt as a pair (0 for padding). The four lanes of a run (mask) call together.
template <int BITS>
__device__ __forceinline__ int norm_pairs(const float* s, const float* w, Pair r, uint32_t mask, uint32_t* codes) {
    // the largest |y|: the pair's first float decides but where it is L 2^e itself
    float top = 0.f;
    bool above = false, nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Pair t = scale_pair(s[i], r, w[i]);
        const float h = fabsf(t.hi);
        const bool more = t.lo != 0.f && (t.lo < 0.f) == (t.hi < 0.f);
        nan |= !(h <= 3.402823466e38f);
        if (h > top) top = h, above = more;
        else if (h == top) above |= more;
    }
    uint32_t k = nan ? 0x7FC00000u : __float_as_uint(top);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const uint32_t ko = __shfl_xor_sync(mask, k, o);
        const bool ao = __shfl_xor_sync(mask, (int)above, o);
        above = ko > k ? ao : ko == k ? above || ao : above;
        k = max(k, ko);
    }
    int byte = mx_exp_byte<BITS>(k);
    if (above && byte < 254) byte = max(byte, mx_exp_byte<BITS>(k + 1));
    const float inv = mx_inv_scale(byte);
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Pair t = scale_pair(s[i], r, w[i]);
        a[i] = to_odd(Pair{t.hi * inv, t.lo * inv});
    }
    mx_enc8<BITS>(a, codes);
    return byte;
}

// x and add of 8 columns, asked for; their rounded sum.
struct NormRaw {
    MxRaw x, add;
};
template <int DT>
__device__ __forceinline__ NormRaw norm_fetch(const MxNormP& p, size_t row, int c, int left) {
    NormRaw r = {mx_fetch8<DT>(p.x, row * p.ld_x + c, left), {}};
    if (p.dt_add == QW_F32) r.add = mx_fetch8<QW_F32>(p.add, row * p.ld_add + c, left);
    else if (p.dt_add >= 0) r.add = mx_fetch8<QW_F16>(p.add, row * p.ld_add + c, left);
    return r;
}
template <int DT>
__device__ __forceinline__ void norm_sum(const MxNormP& p, size_t row, int c, int left, NormRaw& r, float* d) {
    mx_fill8<DT>(p.x, row * p.ld_x + c, left, r.x);
    mx_unpack8<DT>(r.x, d);
    if (p.dt_add >= 0) {
        float a[8];
        const size_t at = row * p.ld_add + c;
        if (p.dt_add == QW_F32) {
            mx_fill8<QW_F32>(p.add, at, left, r.add);
            mx_unpack8<QW_F32>(r.add, a);
        } else {
            mx_fill8<QW_F16>(p.add, at, left, r.add);
            if (p.dt_add == QW_BF16) mx_unpack8<QW_BF16>(r.add, a);
            else mx_unpack8<QW_F16>(r.add, a);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = round_to<DT>(d[i] + a[i]);
    }
}
template <int DT>
__device__ __forceinline__ void norm_load(const MxNormP& p, size_t row, int c, int left, float* d) {
    NormRaw r = norm_fetch<DT>(p, row, c, left);
    norm_sum<DT>(p, row, c, left, r, d);
}

// 8 columns' codes; the scale word of 128 from each half warp's first lane (the whole warp calls).
template <int BITS>
__device__ __forceinline__ void norm_store(const MxNormP& p, size_t row, int v, const uint32_t* q) {
    uint8_t* at = p.codes + row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)v * BITS;
    if (BITS == 8) *reinterpret_cast<uint2*>(at) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(at) = q[0];
}
__device__ __forceinline__ void norm_store_scales(const MxNormP& p, size_t row, int v, bool ok, int byte) {
    const uint32_t sw = mx_gather_word<8>(byte);
    if (ok && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word((int)row, v / 16, p.atoms)) = sw;
}

// Codes and exponent byte of 8 columns from 64-bit values; the four lanes of a run (mask) call together.
template <int BITS>
__device__ __forceinline__ int norm_codes64(const double* y, uint32_t mask, uint32_t* codes) {
    double m = 0.0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bad |= !(fabs(y[i]) <= 3.4028234663852886e38);
        m = fmax(m, fabs(y[i]));
    }
    m = fmax(m, __shfl_xor_sync(mask, m, 1));
    m = fmax(m, __shfl_xor_sync(mask, m, 2));
    bad = (__ballot_sync(mask, bad) & mask) != 0;
    // e = min{e >= -127 : m <= L 2^e}; m = (1 + frac 2^-52) 2^x
    const long long b = __double_as_longlong(m);
    const int x = (int)(b >> 52) - 1023;
    const long long frac = b & 0xFFFFFFFFFFFFFll;
    const int e = BITS == 8 ? x - 8 + (frac > 0xC000000000000ll) : x - 2 + (frac > 0x8000000000000ll);
    const int byte = bad ? 255 : min(254, max(0, e + 127));
    const double inv = bad ? 0.0 : __longlong_as_double((long long)(1023 + 127 - byte) << 52);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_odd(y[i] * inv);
    mx_enc8<BITS>(f, codes);
    return byte;
}

// 8 columns of a NORM_WIDE run, r = 1 / sqrt as a pair: s, read back if it was written (x may be under it), and y in 64 bits.
// Such runs are rare: a call keeps what they need out of the others' registers.
struct RunCodes {
    uint32_t q[2];
    int byte;
};
template <int DT, int BITS>
__device__ __noinline__ RunCodes norm_wide_run(const MxNormP& p, int row, int v, int left, Pair r, uint32_t mask) {
    float s[8], w[8];
    if (p.sum) mx_load8<DT>(p.sum, (size_t)row * p.ld_sum + v * 8, left, s);
    else norm_load<DT>(p, row, v * 8, left, s);
    mx_load8<QW_BF16>(p.w, v * 8, left, w);
    const double rstd = (double)r.hi + (double)r.lo;
    double y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = left > 0 ? (double)s[i] * rstd * (double)w[i] : 0.0;
    RunCodes c;
    c.byte = norm_codes64<BITS>(y, mask, c.q);
    return c;
}

// A row whose squares (or what pairs hold of them) leave fp32, or that holds a NaN or an infinity: everything in fp64, read again from memory.
template <int DT, int BITS>
__device__ __noinline__ void norm_wide_row(const MxNormP& p, int row, double* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int vecs = p.atoms * (MX_ATOM / 8), steps = (vecs + blockDim.x - 1) / blockDim.x;
    double sum = 0.0;
    for (int j = 0; j < steps; ++j) {
        const int v = j * blockDim.x + threadIdx.x;
        float s[8];
        norm_load<DT>(p, row, v * 8, v < vecs ? p.cols - v * 8 : 0, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)s[i] * (double)s[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (warps > 1) {
        __syncthreads();
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < warps; ++i) sum += part[i];
    }
    const double rstd = 1.0 / sqrt(sum / p.cols + (double)p.eps);
    for (int j = 0; j < steps; ++j) {
        const int v = j * blockDim.x + threadIdx.x, left = v < vecs ? p.cols - v * 8 : 0;
        float s[8], w[8];
        norm_load<DT>(p, row, v * 8, left, s);
        mx_load8<QW_BF16>(p.w, v * 8, left, w);
        if (p.sum && left > 0) mx_store8<DT, false>(p.sum, row * p.ld_sum + v * 8, left, s);
        double y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = left > 0 ? (double)s[i] * rstd * (double)w[i] : 0.0;
        uint32_t q[2];
        const int byte = norm_codes64<BITS>(y, 0xFu << (lane & 28), q);
        if (v < vecs) norm_store<BITS>(p, row, v, q);
        norm_store_scales(p, row, v, v < vecs, byte);
    }
}

// A pair summed over the CTA.
__device__ __forceinline__ Pair block_sum(Pair t, Pair* part) {
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) t = add_pairs(t, {__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    if (warps == 1) return t;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
    __syncthreads();
    t = (int)(threadIdx.x & 15) < warps ? part[threadIdx.x & 15] : Pair{0.f, 0.f};
#pragma unroll
    for (int o = 8; o; o >>= 1) t = add_pairs(t, {__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    return t;
}

// VPT: vectors of 8 columns a thread keeps in registers; 0: any number, read twice.
// The bounds of VPT 1 hold a thread to 40 registers; 16 to 24 bytes a thread wait on the stack while a run is redone. 8192 x 1024
// 17.1 us, with 48 registers and none on the stack 17.8.
template <int DT, int BITS, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 128 : 512, VPT == 1 ? 12 : VPT == 2 ? 2 : 1) k_mx_rmsnorm(const __grid_constant__ MxNormP p) {
    constexpr int N = VPT ? VPT : 1;
    __shared__ double part[16];  // of the warps: a pair of floats or, in a wide row, a double
    pdl_wait();
    pdl_launch();
    const int row = blockIdx.x * blockDim.y + threadIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if ((unsigned)row >= (unsigned)p.rows) return;
    const int vecs = p.atoms * (MX_ATOM / 8), steps = VPT ? 1 : (vecs + blockDim.x - 1) / blockDim.x;
    float s[N][8];
    MxRaw wr[N];  // the weight, on its way during the first pass
    {
        NormRaw r[N];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * blockDim.x + threadIdx.x;
            r[k] = norm_fetch<DT>(p, row, v * 8, v < vecs ? p.cols - v * 8 : 0);
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * blockDim.x + threadIdx.x;
            wr[k] = mx_fetch8<QW_BF16>(p.w, v * 8, v < vecs ? p.cols - v * 8 : 0);
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * blockDim.x + threadIdx.x;
            norm_sum<DT>(p, row, v * 8, v < vecs ? p.cols - v * 8 : 0, r[k], s[k]);
        }
    }
    // the sum of squares: at most 16 roundings on the way of each term (4 sums of VPT to 4 + 3 in a thread, 5 + 4 across
    // the CTA); a row of any length in pairs
    Pair t = {0.f, 0.f};
    float sum;
    if (VPT) {
        constexpr int A = VPT < 4 ? 4 : 8;
        float acc[A] = {};
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i % A] = fmaf(s[k][i], s[k][i], acc[i % A]);
#pragma unroll
        for (int o = A / 2; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) acc[i] += acc[i + o];
        sum = warp_sum(acc[0]);
        if (warps > 1) {
            float* sums = reinterpret_cast<float*>(part);
            if (lane == 0) sums[warp] = sum;
            __syncthreads();
            sum = (lane & 15) < warps ? sums[lane & 15] : 0.f;
#pragma unroll
            for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
    } else {
        for (int j = 0; j < steps; ++j) {
            const int v = j * blockDim.x + threadIdx.x;
            norm_load<DT>(p, row, v * 8, v < vecs ? p.cols - v * 8 : 0, s[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) add_square(t, s[0][i]);
        }
        t = block_sum(t, reinterpret_cast<Pair*>(part));
        sum = t.hi;
    }
    const float mean = fmaf(sum, p.inv_n.hi, p.eps);
    if (!(sum > 0x1p-80f && mean < 0x1p90f)) {
        norm_wide_row<DT, BITS>(p, row, part);
        return;
    }
    const float rstd = rsqrtf(mean);
    Pair r = {0.f, 0.f};
    const uint32_t mask = 0xFu << (lane & 28);  // the four lanes of a run
    int again[N], byte[N];
    bool any = false;
    if constexpr (!VPT) r = refine_rsqrt(t, p.inv_n, p.eps, rstd);
    for (int j = 0; j < steps; ++j) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int v = (VPT ? k : j) * blockDim.x + threadIdx.x, left = v < vecs ? p.cols - v * 8 : 0;
            if (!VPT) {
                norm_load<DT>(p, row, v * 8, left, s[0]);
                wr[k] = mx_fetch8<QW_BF16>(p.w, v * 8, left);
            }
            float w[8];
            mx_fill8<QW_BF16>(p.w, v * 8, left, wr[k]);
            mx_unpack8<QW_BF16>(wr[k], w);
            if (p.sum && left > 0) mx_store8<DT, false>(p.sum, row * p.ld_sum + v * 8, left, s[k]);
            uint32_t q[2];
            byte[k] = norm_codes<BITS>(s[k], w, left > 0 ? rstd : 0.f, q, again[k]);
            if (!VPT) {
                const uint32_t doubt = __ballot_sync(0xffffffffu, again[k]), wide = __ballot_sync(0xffffffffu, again[k] == NORM_WIDE);
                if (wide & mask) {
                    const RunCodes c = norm_wide_run<DT, BITS>(p, row, v, left, r, mask);
                    byte[k] = c.byte, q[0] = c.q[0], q[1] = c.q[1];
                } else if (doubt & mask) {
                    byte[k] = norm_pairs<BITS>(s[k], w, left > 0 ? r : Pair{0.f, 0.f}, mask, q);
                }
                __syncwarp();
            }
            any |= again[k] != 0;
            if (v < vecs) norm_store<BITS>(p, row, v, q);
            norm_store_scales(p, row, v, v < vecs, byte[k]);
        }
    }
    if constexpr (VPT > 0) {
        if (!(warps > 1 ? __syncthreads_or(any) : __any_sync(0xffffffffu, any))) return;
        // the runs in doubt again
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) add_square(t, s[k][i]);
        t = block_sum(t, reinterpret_cast<Pair*>(part));
        r = refine_rsqrt(t, p.inv_n, p.eps, rstd);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int v = k * blockDim.x + threadIdx.x, left = v < vecs ? p.cols - v * 8 : 0;
            const uint32_t doubt = __ballot_sync(0xffffffffu, again[k]), wide = __ballot_sync(0xffffffffu, again[k] == NORM_WIDE);
            if (!doubt) continue;
            if (wide & mask) {
                const RunCodes c = norm_wide_run<DT, BITS>(p, row, v, left, r, mask);
                byte[k] = c.byte;
                if (v < vecs) norm_store<BITS>(p, row, v, c.q);
            } else if (doubt & mask) {
                float w[8];
                mx_unpack8<QW_BF16>(wr[k], w);
                uint32_t q[2];
                byte[k] = norm_pairs<BITS>(s[k], w, left > 0 ? r : Pair{0.f, 0.f}, mask, q);
                if (v < vecs) norm_store<BITS>(p, row, v, q);
            }
            __syncwarp();
            norm_store_scales(p, row, v, v < vecs, byte[k]);
        }
    }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

qw_status rows_check(const void* x, size_t ld, int dtype, int cols, const char* what, const char* name) {
    if (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) return qw_fail(QW_ERR_INVALID_ARG, "%s: dtype %d", what, dtype);
    if (!x) return qw_fail(QW_ERR_INVALID_ARG, "%s: NULL %s", what, name);
    if (ld < (size_t)cols) return qw_fail(QW_ERR_INVALID_ARG, "%s: row stride of %s below its columns", what, name);
    if (!aligned16(x) || ld % (dtype == QW_F32 ? 4 : 8)) return qw_fail(QW_ERR_INVALID_ARG, "%s: rows of %s not 16-byte aligned", what, name);
    return QW_OK;
}

MxRowsP rows_p(const qw_mx* m, const void* src, void* dst, size_t ld) {
    return {(uint8_t*)m->dev_codes, (uint8_t*)m->dev_scales, m->rows, m->cols, (int)mx_atoms(m->cols), src, dst, ld, 0, 0};
}

qw_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// `atoms` of 128 columns a piece, `pieces` a warp.
template <typename K>
cudaError_t launch_rows(K kern, MxRowsP p, unsigned atoms, unsigned pieces, cudaStream_t st) {
    p.per_row = ((unsigned)p.atoms + atoms - 1) / atoms;
    p.units = (unsigned)p.rows * p.per_row;
    return launch_k({st, true, nullptr}, kern, dim3((p.units - 1) / (MQ_WARPS * pieces) + 1), dim3(MQ_WARPS * 32), 0, p);
}
// From some waves of CTAs on. Measured (us): 64 x 2048 from fp16 to 8 bits 1.3 small; 1024 x 2048 2.4 small, 2.3 large; 8192 x 2048
// 12.1 and 8.9; 151936 x 1024 from bf16 to 4 bits 99 and 64.
bool large(const MxRowsP& p) { return (double)p.rows * p.atoms >= 16384.0; }

template <int DT, int BITS>
cudaError_t launch_quantize(const MxRowsP& p, cudaStream_t st) {
    return large(p) ? launch_rows(k_mx_quantize<DT, BITS, 16>, p, 4, 1, st) : launch_rows(k_mx_quantize<DT, BITS, 8>, p, 2, 1, st);
}
template <int DT, int BITS>
cudaError_t launch_read(const MxRowsP& p, cudaStream_t st) {
    return large(p) ? launch_rows(k_mx_read<DT, BITS, 4>, p, 2, 4, st) : launch_rows(k_mx_read<DT, BITS, 1>, p, 2, 1, st);
}

template <int DT, int BITS>
cudaError_t launch_norm(const MxNormP& p, cudaStream_t st) {
    const LaunchCtx c = {st, true, nullptr};
    const int vecs = p.atoms * (MX_ATOM / 8);
    // up to 1024 columns a thread has 8 of them, to 8192 16, to 16384 32. Measured (us; fp32 with a bf16 branch): 1 x 1024 1.75 with 8,
    // 2.2 with 16; 8192 x 1024 17.0 both; 4096 x 2048 18.6 with 8, 17.6 with 16, 21.3 with 32; 2048 x 4096 20.9, 19.0 and 22.0; 1024 x
    // 16384 (bf16) 40.3 with 32, read twice 43.1
    const int vpt = vecs <= 128 ? 1 : vecs <= 1024 ? 2 : vecs <= 2048 ? 4 : 0;
    const unsigned threads = vpt ? ((vecs + vpt - 1) / vpt + 31) / 32 * 32 : 512;
    // many rows of one warp: four a CTA (16384 x 256 bf16 7.9 us, one a CTA 17.2)
    const unsigned rows = threads == 32 && p.rows >= 4096 ? 4 : 1;
    const dim3 block(threads, rows), grid(((unsigned)p.rows + rows - 1) / rows);
    switch (vpt) {
        case 1: return launch_k(c, k_mx_rmsnorm<DT, BITS, 1>, grid, block, 0, p);
        case 2: return launch_k(c, k_mx_rmsnorm<DT, BITS, 2>, grid, block, 0, p);
        case 4: return launch_k(c, k_mx_rmsnorm<DT, BITS, 4>, grid, block, 0, p);
        default: return launch_k(c, k_mx_rmsnorm<DT, BITS, 0>, grid, block, 0, p);
    }
}

}  // namespace

#define MX_DISPATCH(fn, dt, bits)                                                                               \
    ((bits) == 8 ? ((dt) == QW_F16 ? fn(QW_F16, 8) : (dt) == QW_BF16 ? fn(QW_BF16, 8) : fn(QW_F32, 8))           \
                 : ((dt) == QW_F16 ? fn(QW_F16, 4) : (dt) == QW_BF16 ? fn(QW_BF16, 4) : fn(QW_F32, 4)))

extern "C" size_t qw_mx_code_bytes(int bits, int rows, int cols) {
    return (bits == 8 || bits == 4) && rows >= 0 && cols > 0 && cols <= QW_MX_MAX_COLS ? (size_t)rows * mx_row_bytes(bits, cols) : 0;
}
extern "C" size_t qw_mx_scale_bytes(int rows, int cols) {
    return rows >= 0 && cols > 0 && cols <= QW_MX_MAX_COLS ? ((size_t)rows + 127) / 128 * mx_atoms(cols) * MX_TILE_BYTES : 0;
}

qw_status mx_check(const qw_mx* m, const char* what, const char* name) {
    if (!m) return qw_fail(QW_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
    if (m->bits != 8 && m->bits != 4) return qw_fail(QW_ERR_UNSUPPORTED, "%s: %s has %d bits (8 and 4 are built)", what, name, m->bits);
    if (m->rows < 0 || m->cols < 1 || m->cols > QW_MX_MAX_COLS || (double)m->rows * mx_atoms(m->cols) > 2147483647.0)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: rows or cols of %s out of range", what, name);
    if (m->rows && (!m->dev_codes || !m->dev_scales)) return qw_fail(QW_ERR_INVALID_ARG, "%s: %s has no memory", what, name);
    if (((uintptr_t)m->dev_codes | (uintptr_t)m->dev_scales) & 31)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: %s not 32-byte aligned", what, name);
    return QW_OK;
}

bool mx_meet(const MxSpan& a, const MxSpan& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    if (a.rows == 1 || a.len == a.step) {  // one block against rows
        const uintptr_t lo = a.at, hi = a.at + (a.rows - 1) * a.step + a.len;
        const size_t i = b.rows == 1 || lo <= b.at ? 0 : std::min(b.rows - 1, (lo - b.at) / b.step);  // the last row that begins before the block
        const uintptr_t row = b.at + i * b.step;
        return (lo < row + b.len && row < hi) || (i + 1 < b.rows && row + b.step < hi);
    }
    if (b.rows == 1 || b.len == b.step) return mx_meet(b, a);
    if (a.step != b.step) return false;
    // b's row j begins d bytes after a's row k + j
    const long long step = (long long)a.step, off = (long long)(b.at - a.at), k = off >= 0 ? off / step : -((step - 1 - off) / step);
    const size_t d = (size_t)(off - k * step);
    const auto both = [&](long long first) { return first < (long long)a.rows && first + (long long)b.rows > 0; };
    return (d < a.len && both(k)) || (d + b.len > a.step && both(k + 1));
}
bool mx_meet(const qw_mx& m, const MxSpan& b) {
    const size_t codes = qw_mx_code_bytes(m.bits, m.rows, m.cols), scales = qw_mx_scale_bytes(m.rows, m.cols);
    return m.rows && (mx_meet(MxSpan{(uintptr_t)m.dev_codes, 1, codes, codes}, b) || mx_meet(MxSpan{(uintptr_t)m.dev_scales, 1, scales, scales}, b));
}
bool mx_meet(const qw_mx& a, const qw_mx& b) {
    const size_t codes = qw_mx_code_bytes(b.bits, b.rows, b.cols), scales = qw_mx_scale_bytes(b.rows, b.cols);
    return b.rows && (mx_meet(a, MxSpan{(uintptr_t)b.dev_codes, 1, codes, codes}) || mx_meet(a, MxSpan{(uintptr_t)b.dev_scales, 1, scales, scales}));
}

extern "C" qw_status qw_mx_quantize(const qw_mx* out, const void* dev_x, size_t ld_x, int dtype, void* stream) {
    if (qw_status s = mx_check(out, "mx_quantize", "out")) return s;
    if (out->rows == 0) return QW_OK;
    if (qw_status s = rows_check(dev_x, ld_x, dtype, out->cols, "mx_quantize", "x")) return s;
    if (mx_meet(*out, mx_rows_span(dev_x, out->rows, out->cols, ld_x, dtype))) return qw_fail(QW_ERR_INVALID_ARG, "mx_quantize: out overlaps x");
    const MxRowsP p = rows_p(out, dev_x, nullptr, ld_x);
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_Q(dt, bits) launch_quantize<dt, bits>(p, st)
    return done(MX_DISPATCH(MX_Q, dtype, out->bits), "mx_quantize");
}

extern "C" qw_status qw_mx_read(const qw_mx* m, void* dev_x, size_t ld_x, int dtype, void* stream) {
    if (qw_status s = mx_check(m, "mx_read", "m")) return s;
    if (m->rows == 0) return QW_OK;
    if (qw_status s = rows_check(dev_x, ld_x, dtype, m->cols, "mx_read", "x")) return s;
    if (mx_meet(*m, mx_rows_span(dev_x, m->rows, m->cols, ld_x, dtype))) return qw_fail(QW_ERR_INVALID_ARG, "mx_read: x overlaps m");
    const MxRowsP p = rows_p(m, nullptr, dev_x, ld_x);
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_R(dt, bits) launch_read<dt, bits>(p, st)
    return done(MX_DISPATCH(MX_R, dtype, m->bits), "mx_read");
}

extern "C" qw_status qw_mx_rmsnorm(const qw_mx* out, const void* dev_x, size_t ld_x, int x_dtype, const void* dev_add,
                                   size_t ld_add, int add_dtype, void* dev_sum, size_t ld_sum, const void* dev_weight,
                                   float eps, void* stream) {
    if (qw_status s = mx_check(out, "mx_rmsnorm", "out")) return s;
    if (!(eps > 0.f) || eps > 3e38f) return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: eps must be positive and finite");
    if (out->rows == 0) return QW_OK;
    if (qw_status s = rows_check(dev_x, ld_x, x_dtype, out->cols, "mx_rmsnorm", "x")) return s;
    if (dev_add)
        if (qw_status s = rows_check(dev_add, ld_add, add_dtype, out->cols, "mx_rmsnorm", "add")) return s;
    if (dev_sum) {
        if (qw_status s = rows_check(dev_sum, ld_sum, x_dtype, out->cols, "mx_rmsnorm", "sum")) return s;
        if (dev_sum == dev_x && ld_sum != ld_x) return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: sum over x with another row stride");
        if (dev_sum == dev_add) return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: sum over add");
    }
    if (!dev_weight || !aligned16(dev_weight)) return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: weight NULL or not 16-byte aligned");
    const MxSpan x = mx_rows_span(dev_x, out->rows, out->cols, ld_x, x_dtype), add = mx_rows_span(dev_add, out->rows, out->cols, ld_add, add_dtype),
                 sum = mx_rows_span(dev_sum, out->rows, out->cols, ld_sum, x_dtype), w = mx_rows_span(dev_weight, 1, out->cols, out->cols, QW_BF16);
    if ((dev_sum != dev_x && mx_meet(sum, x)) || mx_meet(sum, add) || mx_meet(sum, w))
        return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: sum overlaps an input that it is not");
    if (mx_meet(*out, x) || mx_meet(*out, add) || mx_meet(*out, sum) || mx_meet(*out, w))
        return qw_fail(QW_ERR_INVALID_ARG, "mx_rmsnorm: out overlaps another operand");
    const double inv_n = 1.0 / out->cols;
    const MxNormP p = {(uint8_t*)out->dev_codes, (uint8_t*)out->dev_scales, out->rows, out->cols, (int)mx_atoms(out->cols), dev_x,
                       dev_add, dev_sum, (const bf16*)dev_weight, ld_x, ld_add, ld_sum, dev_add ? add_dtype : -1, eps,
                       {(float)inv_n, (float)(inv_n - (float)inv_n)}};
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_N(dt, bits) launch_norm<dt, bits>(p, st)
    return done(MX_DISPATCH(MX_N, x_dtype, out->bits), "mx_rmsnorm");
}
