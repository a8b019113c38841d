// Microscaled matrices: quantisation of rows (qw_mx_quantize), their values (qw_mx_read) and RMSNorm with
// the branch's addition and a quantised output (qw_mx_rmsnorm). mx.cuh states the format.
//
// Quantise and read. A thread has 8 columns, four a run, sixteen a row's scale word. The exponent follows
// from the largest magnitude alone and x 2^-e is exact, so the codes are those of the definition bit for
// bit. Bytes bound both.
//
// RMSNorm. s = x + add rounded to the stream's type, y = s / sqrt(mean(s^2) + eps) * w, codes of y. y has no
// type of its own: the codes are those of the real y, whatever the order of the sums. To that end the row's
// sum of squares is carried as an unevaluated pair of floats (the products' and sums' errors are added up;
// about 2^-45 relative), y is computed in fp32 with a relative error below 2^-21, and a run in which a value
// between y (1 - 2^-20) and y (1 + 2^-20) could get another code or exponent, one in 1500, is computed again
// in fp64 from the pair. One CTA a row; a row's elements stay in registers between the two passes.
#include <algorithm>

#include "mx.cuh"

namespace {

constexpr int MQ_WARPS = 8;

// Four bytes of a run's first lane (lanes 0, 4, 8, 12 of each half warp) as a word, in the half warp's lane 0.
__device__ __forceinline__ uint32_t mx_gather_word(int byte) {
    uint32_t w = (uint32_t)byte;
    w |= __shfl_down_sync(0xffffffffu, w, 4) << 8;
    return w | (__shfl_down_sync(0xffffffffu, w, 8) << 16);
}

struct MxRowsP {
    uint8_t* codes;
    uint8_t* scales;
    int rows, cols, atoms;
    const void* src;
    void* dst;
    size_t ld;
    unsigned units, per_row;  // warps' pieces of 256 columns
};

template <int DT, int BITS>
__global__ void __launch_bounds__(MQ_WARPS * 32) k_mx_quantize(const __grid_constant__ MxRowsP p) {
    pdl_wait();
    pdl_launch();
    const unsigned u = blockIdx.x * MQ_WARPS + (threadIdx.x >> 5);
    if (u >= p.units) return;
    const int lane = threadIdx.x & 31, row = (int)(u / p.per_row), c = (int)(u % p.per_row) * 256 + lane * 8;
    float x[8];
    mx_load8<DT>(p.src, (size_t)row * p.ld + c, p.cols - c, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int byte = mx_exp_byte<BITS>(m);
    const float inv = mx_inv_scale(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    uint32_t w[2];
    mx_enc8<BITS>(x, w);
    const uint32_t sw = mx_gather_word(byte);
    if (c >= p.atoms * MX_ATOM) return;
    uint8_t* at = p.codes + (size_t)row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)c * BITS / 8;
    if (BITS == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(at) = w[0];
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, c / MX_ATOM, p.atoms)) = sw;
}

template <int DT, int BITS>
__global__ void __launch_bounds__(MQ_WARPS * 32) k_mx_read(const __grid_constant__ MxRowsP p) {
    pdl_wait();
    pdl_launch();
    const unsigned u = blockIdx.x * MQ_WARPS + (threadIdx.x >> 5);
    if (u >= p.units) return;
    const int lane = threadIdx.x & 31, row = (int)(u / p.per_row), c = (int)(u % p.per_row) * 256 + lane * 8;
    if (c >= p.cols) return;
    const uint8_t* at = p.codes + (size_t)row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)c * BITS / 8;
    uint32_t w[2], h[4];
    if (BITS == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
    const float s = mx_scale(p.scales[mx_scale_word(row, c / MX_ATOM, p.atoms) + (c / MX_RUN & 3)]);
    mx_dec8<BITS>(w, h);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = h_lo(h[i]) * s;
        x[2 * i + 1] = h_hi(h[i]) * s;
    }
    mx_store8<DT>(p.dst, (size_t)row * p.ld + c, p.cols - c, x);
}

// ---- RMSNorm --------------------------------------------------------------------------------------------

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
};

// A sum as an unevaluated pair: hi + lo.
struct Pair {
    float hi, lo;
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

template <int DT>
__device__ __forceinline__ float round_to(float v) {
    if (DT == QW_F16) return __half2float(__float2half_rn(v));
    if (DT == QW_BF16) return bf2f(__float2bfloat16_rn(v));
    return v;
}

// A double to the float that rounds like it to fewer bits: towards zero, the last bit set if inexact.
__device__ __forceinline__ float to_odd(double t) {
    const float f = __double2float_rz(t);
    return (double)f == t ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The run's exponent byte and this thread's codes in fp64 (the four lanes of a run together).
template <int BITS>
__device__ __noinline__ int norm_exact(const float* s, const float* w, double rstd, uint32_t mask, uint32_t* codes) {
    double y[8], m = 0.0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = (double)s[i] * rstd * (double)w[i];
        bad |= !(fabs(y[i]) <= 3.4028234663852886e38);
        m = fmax(m, fabs(y[i]));
    }
    m = fmax(m, __shfl_xor_sync(mask, m, 1));
    m = fmax(m, __shfl_xor_sync(mask, m, 2));
    bad = __any_sync(mask, bad);
    // e = min{e >= -127 : m <= L 2^e}; m = f 2^x, 1 <= f < 2
    const long long b = __double_as_longlong(m);
    const int x = (int)(b >> 52) - 1023;
    const long long frac = b & 0xFFFFFFFFFFFFFll;
    const int e = BITS == 8 ? x - 8 + (frac > 0xC000000000000ll) : x - 2 + (frac > 0x8000000000000ll);
    const int byte = bad ? 255 : min(254, max(0, e + 127));
    const double inv = byte == 255 ? 0.0 : __longlong_as_double((long long)(1023 + 127 - byte) << 52);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_odd(y[i] * inv);
    mx_enc8<BITS>(f, codes);
    return byte;
}

constexpr float NORM_LO = 1.f - 0x1p-20f, NORM_HI = 1.f + 0x1p-20f;

// Quantises 8 columns; the whole warp calls. inside: the columns are not padding, which is zeros whatever the row.
template <int BITS>
__device__ __forceinline__ int norm_codes(const float* s, const float* w, bool inside, float rstd, Pair sum, double sum64, bool wide,
                                          int n, float eps, uint32_t* codes) {
    if (!inside) rstd = 0.f;
    float y[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = s[i] * rstd * w[i];
        m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float am = __uint_as_float(m);
    int byte = mx_exp_byte<BITS>(m);
    // a run of tiny values: s rstd may have underflowed
    bool again = wide || (am < 0x1p-30f && am > 0.f) ||
                 mx_exp_byte<BITS>(__float_as_uint(am * NORM_LO)) != mx_exp_byte<BITS>(__float_as_uint(am * NORM_HI));
    const float inv = mx_inv_scale(byte);
    const float lo = inv * NORM_LO, hi = inv * NORM_HI;  // inv is a power of two: no rounding
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = y[i] * lo;
        b[i] = y[i] * hi;
    }
    uint32_t cb[2];
    mx_enc8<BITS>(a, codes);
    mx_enc8<BITS>(b, cb);
    again |= codes[0] != cb[0] || codes[1] != cb[1];
    const uint32_t lane = threadIdx.x & 31, mask = 0xFu << (lane & 28u);
    again = (__ballot_sync(0xffffffffu, again) & mask) != 0;
    if (again) {
        const double t = wide ? sum64 : (double)sum.hi + (double)sum.lo;
        byte = norm_exact<BITS>(s, w, inside ? 1.0 / sqrt(t / n + (double)eps) : 0.0, mask, codes);
    }
    __syncwarp();
    return byte;
}

// VPT: vectors of 8 columns a thread keeps in registers; 0: any number, read twice.
template <int DT, int BITS, int VPT>
__global__ void __launch_bounds__(512) k_mx_rmsnorm(const __grid_constant__ MxNormP p) {
    constexpr int N = VPT ? VPT : 1;
    __shared__ Pair part[16];
    __shared__ double part64[16];
    pdl_wait();
    pdl_launch();
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int vecs = p.atoms * (MX_ATOM / 8), steps = (vecs + blockDim.x - 1) / blockDim.x;  // steps: VPT 0
    const size_t rx = (size_t)row * p.ld_x, ra = (size_t)row * p.ld_add, rs = (size_t)row * p.ld_sum;
    float s[N][8];
    auto load = [&](int v, float* d) {
        const int c = v * 8, left = v < vecs ? p.cols - c : 0;
        mx_load8<DT>(p.x, rx + c, left, d);
        if (p.dt_add >= 0) {
            float a[8];
            if (p.dt_add == QW_F32) mx_load8<QW_F32>(p.add, ra + c, left, a);
            else if (p.dt_add == QW_BF16) mx_load8<QW_BF16>(p.add, ra + c, left, a);
            else mx_load8<QW_F16>(p.add, ra + c, left, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = round_to<DT>(d[i] + a[i]);
        }
    };
    Pair t = {0.f, 0.f};
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
        if (VPT) load(jj * blockDim.x + threadIdx.x, s[jj]);
    }
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
        for (int j = jj; j < (VPT ? jj + 1 : steps); ++j) {
            if (!VPT) load(j * blockDim.x + threadIdx.x, s[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) add_square(t, s[jj][i]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) t = add_pairs(t, {__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    if (warps > 1) {
        if (lane == 0) part[warp] = t;
        __syncthreads();
        t = part[0];
        for (int i = 1; i < warps; ++i) t = add_pairs(t, part[i]);
    }
    // squares that fp32 cannot hold (or not in a pair): the sum in fp64, and every run
    const bool wide = !(t.hi > 0x1p-80f && t.hi < 0x1p120f);
    double sum64 = 0.0;
    if (wide) {
#pragma unroll
        for (int jj = 0; jj < N; ++jj) {
            for (int j = jj; j < (VPT ? jj + 1 : steps); ++j) {
                if (!VPT) load(j * blockDim.x + threadIdx.x, s[0]);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum64 += (double)s[jj][i] * (double)s[jj][i];
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum64 += __shfl_xor_sync(0xffffffffu, sum64, o);
        if (warps > 1) {
            if (lane == 0) part64[warp] = sum64;
            __syncthreads();
            sum64 = part64[0];
            for (int i = 1; i < warps; ++i) sum64 += part64[i];
        }
    }
    const float rstd = wide ? 0.f : 1.f / sqrtf(t.hi / p.cols + p.eps);
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
        for (int j = jj; j < (VPT ? jj + 1 : steps); ++j) {
            const int v = j * blockDim.x + threadIdx.x, c = v * 8, left = v < vecs ? p.cols - c : 0;
            float* d = s[jj];
            if (!VPT) load(v, d);
            float w[8];
            mx_load8<QW_BF16>(p.w, c, left, w);
            if (p.sum && left > 0) mx_store8<DT>(p.sum, rs + c, left, d);
            uint32_t q[2];
            const int byte = norm_codes<BITS>(d, w, left > 0, rstd, t, sum64, wide, p.cols, p.eps, q);
            const uint32_t sw = mx_gather_word(byte);
            if (v < vecs) {
                uint8_t* at = p.codes + (size_t)row * p.atoms * (MX_ATOM * BITS / 8) + (size_t)c * BITS / 8;
                if (BITS == 8) *reinterpret_cast<uint2*>(at) = make_uint2(q[0], q[1]);
                else *reinterpret_cast<uint32_t*>(at) = q[0];
                if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, c / MX_ATOM, p.atoms)) = sw;
            }
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
    const int atoms = (int)mx_atoms(m->cols);
    const unsigned per = (unsigned)(atoms + 1) / 2;
    return {(uint8_t*)m->dev_codes, (uint8_t*)m->dev_scales, m->rows, m->cols, atoms, src, dst, ld, (unsigned)m->rows * per, per};
}

qw_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <typename K>
cudaError_t launch_rows(K kern, const MxRowsP& p, cudaStream_t st) {
    return launch_k({st, true, nullptr}, kern, dim3((p.units + MQ_WARPS - 1) / MQ_WARPS), dim3(MQ_WARPS * 32), 0, p);
}

template <int DT, int BITS>
cudaError_t launch_norm(const MxNormP& p, cudaStream_t st) {
    const LaunchCtx c = {st, true, nullptr};
    const int vecs = p.atoms * (MX_ATOM / 8);
    // a row of up to 2048 columns has a thread for every 8; a longer one two or four vectors a thread
    const int vpt = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : vecs <= 2048 ? 4 : 0;
    const dim3 block(vpt ? ((vecs + vpt - 1) / vpt + 31) / 32 * 32 : 512), grid(p.rows);
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

extern "C" qw_status qw_mx_quantize(const qw_mx* out, const void* dev_x, size_t ld_x, int dtype, void* stream) {
    if (qw_status s = mx_check(out, "mx_quantize", "out")) return s;
    if (out->rows == 0) return QW_OK;
    if (qw_status s = rows_check(dev_x, ld_x, dtype, out->cols, "mx_quantize", "x")) return s;
    const MxRowsP p = rows_p(out, dev_x, nullptr, ld_x);
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_Q(dt, bits) launch_rows(k_mx_quantize<dt, bits>, p, st)
    return done(MX_DISPATCH(MX_Q, dtype, out->bits), "mx_quantize");
}

extern "C" qw_status qw_mx_read(const qw_mx* m, void* dev_x, size_t ld_x, int dtype, void* stream) {
    if (qw_status s = mx_check(m, "mx_read", "m")) return s;
    if (m->rows == 0) return QW_OK;
    if (qw_status s = rows_check(dev_x, ld_x, dtype, m->cols, "mx_read", "x")) return s;
    const MxRowsP p = rows_p(m, nullptr, dev_x, ld_x);
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_R(dt, bits) launch_rows(k_mx_read<dt, bits>, p, st)
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
    const MxNormP p = {(uint8_t*)out->dev_codes, (uint8_t*)out->dev_scales, out->rows, out->cols, (int)mx_atoms(out->cols), dev_x,
                       dev_add, dev_sum, (const bf16*)dev_weight, ld_x, ld_add, ld_sum, dev_add ? add_dtype : -1, eps};
    const cudaStream_t st = (cudaStream_t)stream;
#define MX_N(dt, bits) launch_norm<dt, bits>(p, st)
    return done(MX_DISPATCH(MX_N, x_dtype, out->bits), "mx_rmsnorm");
}
