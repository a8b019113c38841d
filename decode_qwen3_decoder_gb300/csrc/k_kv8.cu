// Append to and read back from the 8-bit paged KV cache (qw_kv8_append, qw_kv8_read).
//
// Append. A page's exponent for one KV head and tensor is e = min{e : max|x| <= 448 * 2^e} over
// its tokens and its codes are e4m3(x * 2^-e). Both follow exactly from the fp16 values, so
// the result does not depend on any order. One warp owns the (page, head, tensor): it keeps the
// page's 16 x HD values in registers (64 per lane at HD = 128, in pairs), takes the maximum by shuffles
// and writes the codes once. Tokens the page already holds are decoded, exact in fp32, and
// re-coded with the larger exponent; a power of two leaves them as they are but for codes that
// become subnormal. Bytes bound it: each input element is read once and each code written once. 16
// prompts of 512 tokens (8 heads of 128, 50 MB): 15 us, 3.4 TB/s, in a wave and a half of CTAs whose row
// loads wait for the page id; values held as fp32 instead of fp16 pairs took 17 (80 registers instead
// of 56). A step of 64 sequences is a launch, 4 us.
//
// Read. The same cut into warps; 28 layers of 2048 tokens (353 MB) take 60 us, 5.9 TB/s.
#include "kv8.cuh"

#include <algorithm>

namespace {

constexpr int KA_WARPS = 4;

struct Kv8AppendP {
    Kv8View kv;
    const int* start;
    const int* cu;
    const void* src[2];
    size_t ld[2];
    int T, max_len, pages;  // pages: most pages an entry can touch
    bool staged;            // source rows in pages of 16 tokens
    int* status;
};

// Entry b's start and row range; false (and the status bit) if they break the bounds.
__device__ __forceinline__ bool kv8_entry(const Kv8View& kv, const int* start, const int* cu, int b, int T, int max_len,
                                          int& s, int& r0, int& n) {
    s = start[b];
    r0 = cu[b];
    n = cu[b + 1] - r0;
    return s >= 0 && r0 >= 0 && n >= 0 && n <= max_len && r0 <= T - n &&
           (long long)s + n <= (long long)kv.max_pages * KV8_PAGE;
}

// Two elements as halves; one outside the fp16 range is taken as 0 and noted.
__device__ __forceinline__ uint32_t pack_ok(float a, float b, bool& bad) {
    const bool ba = f16_out_of_range(a), bb = f16_out_of_range(b);
    bad |= ba || bb;
    return pack_h2(ba ? 0.f : a, bb ? 0.f : b);
}

// 16 consecutive elements as their fp16 roundings, in pairs; `bad` if one is outside the fp16 range
// (taken as 0).
template <int DT>
__device__ __forceinline__ void load16(const void* base, size_t off, uint32_t* x, bool& bad) {
    if (DT == QW_F32) {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = p[i];
            x[2 * i] = pack_ok(v.x, v.y, bad);
            x[2 * i + 1] = pack_ok(v.z, v.w, bad);
        }
    } else {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + off);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = p[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t y = w[k];
                if (DT == QW_BF16) {
                    y = pack_ok(bf_lo(y), bf_hi(y), bad);
                } else if ((y & 0x7C00u) == 0x7C00u || (y & 0x7C000000u) == 0x7C000000u) {  // infinity or NaN
                    y = pack_ok(h_lo(y), h_hi(y), bad);
                }
                x[4 * i + k] = y;
            }
        }
    }
}

template <int HD, int DT>
__global__ void __launch_bounds__(KA_WARPS * 32) k_kv8_append(const __grid_constant__ Kv8AppendP p) {
    constexpr int CH = Kv8<HD>::CH, TSTEP = 32 / CH, UPL = KV8_PAGE / TSTEP;
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int job = blockIdx.x * KA_WARPS + (threadIdx.x >> 5);
    const int which = job & 1, head = (job >> 1) % p.kv.n_kv, pi = (job >> 1) / p.kv.n_kv;
    pdl_wait();
    pdl_launch();
    if (pi >= p.pages) return;
    int s, r0, n;
    if (!kv8_entry(p.kv, p.start, p.cu, b, p.T, p.max_len, s, r0, n)) {
        if (job == 0 && lane == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        return;
    }
    const int page_i = s / KV8_PAGE + pi;
    if (n == 0 || page_i * KV8_PAGE >= s + n) return;
    const int page = kv8_row(p.kv, p.kv.table, b)[page_i];
    if (page < 0 || page >= p.kv.n_pages) {
        if (lane == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        return;
    }
    uint8_t* blk = kv8_block(p.kv, b, page, head, Kv8<HD>::BLK);
    uint8_t* codes = blk + (which ? Kv8<HD>::VOFF : 0);
    float* scale = reinterpret_cast<float*>(blk + Kv8<HD>::SOFF) + which;
    const int ch = lane % CH, t0 = lane / CH;
    const int had = max(0, s - page_i * KV8_PAGE);  // tokens the page already holds
    const void* src = p.src[which];
    uint32_t x[UPL][8];  // fp16 pairs
    uint32_t m2 = 0u;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < UPL; ++u) {
        const int pos = page_i * KV8_PAGE + t0 + u * TSTEP;
        if (pos >= s && pos < s + n) {
            const int row = r0 + pos - s;
            const size_t at = p.staged ? (((size_t)(row >> 4) * p.kv.n_kv + head) * 16 + (row & 15)) * HD
                                       : (size_t)row * p.ld[which] + head * HD;
            load16<DT>(src, at + ch * 16, x[u], bad);
#pragma unroll
            for (int i = 0; i < 8; ++i) m2 = kv8_absmax2(m2, x[u][i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0u;
        }
    }
    int e = kv8_exponent(warp_max(kv8_max2(m2)));
    float so = 1.f;
    if (had) {
        so = *scale;
        e = max(e, kv8_log2(so));
        __syncwarp();  // every lane has read the old scale
    }
    const float mul = kv8_pow2(-e);
#pragma unroll
    for (int u = 0; u < UPL; ++u) {
        const int t = t0 + u * TSTEP;
        uint4* at = reinterpret_cast<uint4*>(codes + t * HD + (which ? kv8_v_pos<HD>(t, ch) : kv8_k_pos<HD>(t, ch)) * 16);
        if (t < had) {
            if (so * mul != 1.f) *at = kv8_recode16(*at, so * mul);
        } else {
            float f[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[2 * i] = h_lo(x[u][i]);
                f[2 * i + 1] = h_hi(x[u][i]);
            }
            *at = kv8_enc16(f, mul);
        }
    }
    if (lane == 0) *scale = kv8_pow2(e);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, QW_KV8_RANGE);
}

struct Kv8ReadP {
    Kv8View kv;
    const int* start;
    const int* cu;
    void* dst[2];
    size_t ld[2];
    int T, max_len, pages;
    int* status;
};

// The code of a value next to 65504 can stand for 65536.
__device__ __forceinline__ float sat16(float v) { return fminf(fmaxf(v, -65504.f), 65504.f); }

template <int DT>
__device__ __forceinline__ void store16(void* base, size_t off, const float* x) {
    if (DT == QW_F32) {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + off);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = DT == QW_F16 ? pack_h2(sat16(x[8 * i + 2 * k]), sat16(x[8 * i + 2 * k + 1])) : pack_bf2(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]);
            p[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// One warp per (page, head, tensor), lanes as in the append; writes only the entry's rows.
template <int HD, int DT>
__global__ void __launch_bounds__(KA_WARPS * 32) k_kv8_read(const __grid_constant__ Kv8ReadP p) {
    constexpr int CH = Kv8<HD>::CH, TSTEP = 32 / CH, UPL = KV8_PAGE / TSTEP;
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int job = blockIdx.x * KA_WARPS + (threadIdx.x >> 5);
    const int which = job & 1, head = (job >> 1) % p.kv.n_kv, pi = (job >> 1) / p.kv.n_kv;
    pdl_wait();
    pdl_launch();
    if (pi >= p.pages) return;
    int s, r0, n;
    if (!kv8_entry(p.kv, p.start, p.cu, b, p.T, p.max_len, s, r0, n)) {
        if (job == 0 && lane == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        // rows that can be told are zeros
        if (r0 < 0 || n < 0 || n > p.max_len || r0 > p.T - n) return;
        s = 0;
        const int i0 = pi * KV8_PAGE;
        float z[16] = {};
        for (int i = i0 + lane / CH; i < min(n, i0 + KV8_PAGE); i += TSTEP)
            store16<DT>(p.dst[which], (size_t)(r0 + i) * p.ld[which] + head * HD + (lane % CH) * 16, z);
        return;
    }
    const int page_i = s / KV8_PAGE + pi;
    if (n == 0 || page_i * KV8_PAGE >= s + n) return;
    const int page = kv8_row(p.kv, p.kv.table, b)[page_i];
    const bool ok = page >= 0 && page < p.kv.n_pages;
    if (!ok && lane == 0) atomicOr(p.status, QW_KV8_BAD_POS);
    const uint8_t* blk = kv8_block(p.kv, b, ok ? page : 0, head, Kv8<HD>::BLK);
    const uint8_t* codes = blk + (which ? Kv8<HD>::VOFF : 0);
    const float scale = reinterpret_cast<const float*>(blk + Kv8<HD>::SOFF)[which];
    const int ch = lane % CH, t0 = lane / CH;
#pragma unroll
    for (int u = 0; u < UPL; ++u) {
        const int t = t0 + u * TSTEP, pos = page_i * KV8_PAGE + t;
        if (pos < s || pos >= s + n) continue;
        const int at = which ? kv8_v_pos<HD>(t, ch) : kv8_k_pos<HD>(t, ch);
        float x[16];
        kv8_dec16(*reinterpret_cast<const uint4*>(codes + t * HD + at * 16), x);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = ok ? x[i] * scale : 0.f;
        store16<DT>(p.dst[which], (size_t)(r0 + pos - s) * p.ld[which] + head * HD + ch * 16, x);
    }
}

template <typename P, typename K>
cudaError_t launch_pages(K kern, const P& p, int B, cudaStream_t st, int* launches) {
    const int n_kv = p.kv.n_kv;
    LaunchCtx c = {st, true, launches};
    const long long jobs = 2ll * p.pages * n_kv;
    return launch_k(c, kern, dim3((unsigned)((jobs + KA_WARPS - 1) / KA_WARPS), B), dim3(KA_WARPS * 32), 0, p);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

qw_status kv8_check(const qw_kv8* kv, int B, const char* what) {
    if (!kv) return qw_fail(QW_ERR_INVALID_ARG, "%s: kv is NULL", what);
    if (kv->head_dim != 64 && kv->head_dim != 128)
        return qw_fail(QW_ERR_UNSUPPORTED, "%s: head_dim %d (64 and 128 are built)", what, kv->head_dim);
    if (!kv->dev_blocks || !kv->dev_page_table) return qw_fail(QW_ERR_INVALID_ARG, "%s: NULL blocks or page table", what);
    if ((uintptr_t)kv->dev_blocks & 31) return qw_fail(QW_ERR_INVALID_ARG, "%s: blocks not 32-byte aligned", what);
    if (kv->n_pages < 1 || kv->max_pages < 1 || kv->max_pages > (1 << 26) || kv->n_kv_heads < 1 || kv->n_kv_heads > 1024)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: n_pages, max_pages or n_kv_heads out of range", what);
    if (B < 1 || B > QW_KV8_MAX_BATCH) return qw_fail(QW_ERR_INVALID_ARG, "%s: B=%d outside [1, %d]", what, B, QW_KV8_MAX_BATCH);
    return QW_OK;
}

static qw_status kv8_rows_check(const qw_kv8* kv, int B, int T, int max_len, const int32_t* start, const int32_t* cu,
                                const void* k, size_t ld_k, const void* v, size_t ld_v, int dtype, const int32_t* status,
                                const char* what) {
    if (qw_status s = kv8_check(kv, B, what)) return s;
    if (T < 0 || max_len < 1 || max_len > (1 << 26)) return qw_fail(QW_ERR_INVALID_ARG, "%s: T or max_len out of range", what);
    if (!start || !cu || !status) return qw_fail(QW_ERR_INVALID_ARG, "%s: NULL argument", what);
    if (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) return qw_fail(QW_ERR_INVALID_ARG, "%s: dtype %d", what, dtype);
    if (T == 0) return QW_OK;  // no rows to look at
    if (!k || !v) return qw_fail(QW_ERR_INVALID_ARG, "%s: NULL argument", what);
    const size_t row = (size_t)kv->n_kv_heads * kv->head_dim, al = dtype == QW_F32 ? 4 : 8;
    if (ld_k < row || ld_v < row) return qw_fail(QW_ERR_INVALID_ARG, "%s: row stride below n_kv_heads * head_dim", what);
    if (!aligned16(k) || !aligned16(v) || ld_k % al || ld_v % al)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: rows not 16-byte aligned", what);
    return QW_OK;
}

#define KV8_DISPATCH(kern, hd, dt, p)                                                                         \
    ((hd) == 128 ? ((dt) == QW_F16    ? launch_pages(kern<128, QW_F16>, p, B, st, launches)             \
                    : (dt) == QW_BF16 ? launch_pages(kern<128, QW_BF16>, p, B, st, launches)            \
                                      : launch_pages(kern<128, QW_F32>, p, B, st, launches))            \
                 : ((dt) == QW_F16    ? launch_pages(kern<64, QW_F16>, p, B, st, launches)              \
                    : (dt) == QW_BF16 ? launch_pages(kern<64, QW_BF16>, p, B, st, launches)             \
                                      : launch_pages(kern<64, QW_F32>, p, B, st, launches)))

extern "C" size_t qw_kv8_block_bytes(int head_dim) {
    return head_dim == 64 || head_dim == 128 ? 32 * (size_t)head_dim + 32 : 0;
}

qw_status kv8_append(const Kv8View& v, int head_dim, int B, int T, int max_len, const int* start, const int* cu, const void* k,
                     size_t ld_k, const void* val, size_t ld_v, int dtype, bool staged, int* status, cudaStream_t st, int* launches) {
    const int len = std::min(max_len, T);
    Kv8AppendP p = {v, start, cu, {k, val}, {ld_k, ld_v}, T, max_len, (len + 14) / 16 + 1, staged, status};
    cudaError_t e = KV8_DISPATCH(k_kv8_append, head_dim, dtype, p);
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "append: %s", cudaGetErrorString(e));
}

extern "C" qw_status qw_kv8_append(const qw_kv8* kv, int B, int T, int max_len, const int32_t* dev_start,
                                   const int32_t* dev_cu, const void* dev_k, size_t ld_k, const void* dev_v, size_t ld_v,
                                   int dtype, int32_t* dev_status, void* stream) {
    if (qw_status s = kv8_rows_check(kv, B, T, max_len, dev_start, dev_cu, dev_k, ld_k, dev_v, ld_v, dtype, dev_status,
                                     "append"))
        return s;
    if (T == 0) return QW_OK;
    return kv8_append(kv8_view(kv), kv->head_dim, B, T, max_len, dev_start, dev_cu, dev_k, ld_k, dev_v, ld_v, dtype, false,
                      dev_status, (cudaStream_t)stream);
}

extern "C" qw_status qw_kv8_read(const qw_kv8* kv, int B, int T, int max_len, const int32_t* dev_start,
                                 const int32_t* dev_cu, void* dev_k, size_t ld_k, void* dev_v, size_t ld_v, int dtype,
                                 int32_t* dev_status, void* stream) {
    if (qw_status s = kv8_rows_check(kv, B, T, max_len, dev_start, dev_cu, dev_k, ld_k, dev_v, ld_v, dtype, dev_status,
                                     "read"))
        return s;
    if (T == 0) return QW_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const int len = std::min(max_len, T);
    int* launches = nullptr;
    Kv8ReadP p = {kv8_view(kv), dev_start, dev_cu, {dev_k, dev_v}, {ld_k, ld_v}, T, max_len, (len + 14) / 16 + 1, dev_status};
    cudaError_t e = KV8_DISPATCH(k_kv8_read, kv->head_dim, dtype, p);
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "read: %s", cudaGetErrorString(e));
}
