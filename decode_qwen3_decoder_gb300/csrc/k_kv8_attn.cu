// Attention over the 8-bit paged KV cache (qw_kv8_attn).
//
// A query row (token i of an entry, one query head) at position p sees cached positions 0 .. p:
//   t_j = scale log2(e) 2^ek q.k_j,  out = sum_j 2^(t_j - m) 2^ev v_j / sum_j 2^(t_j - m)
// with the page's scales 2^ek, 2^ev and the codes k_j, v_j as the MMA operands: an e4m3 value
// is exact in fp16, so the products see exactly what the cache holds. The weight that goes into
// the PV product is w_j = 2^(t_j + ev_j - R + 8): the V scale joins the exponent, so pages of
// very different scales meet in one fp16 range, and the sum of the softmax takes w_j 2^-ev_j,
// in fp32. The reference R of a row moves only when a weight would pass 2^15; the weights' fp16
// rounding (2^-11 each, 2^-25 absolute where they are subnormal, against a largest weight of at
// least 2^8) is the only rounding below 32 bits before the output's.
#include "kv8.cuh"

#include <algorithm>

namespace {

constexpr float KV8_LOG2E = 1.4426950408889634f, KV8_LN2 = 0.6931471805599453f;
constexpr float KV8_LIFT = 8.f, KV8_SLACK = 7.f;  // weights aim at 2^8 and may grow to 2^15
constexpr int KR_WARPS = 8, KR_ROWS = 16;

struct Kv8AttnP {
    Kv8View kv;
    const int* start;
    const int* cu;
    const void* q;
    size_t ld_q;
    int T, max_len, max_keys, n_heads, G;
    float scale_log2;
    void* out;
    size_t ld_out;
    float* lse;   // optional
    float* lse2;  // optional: in log2 units, for the scores
    const float* score_in;
    float* score_out;
    size_t ld_score;
    int* status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Entry b: start, first row, rows; false when the lengths break their bounds (dead entry).
__device__ __forceinline__ bool attn_entry(const Kv8AttnP& p, int b, int& s, int& r0, int& n) {
    s = p.start[b];
    r0 = p.cu[b];
    n = p.cu[b + 1] - r0;
    return s >= 0 && r0 >= 0 && n >= 0 && n <= p.max_len && r0 <= p.T - n && (long long)s + n <= p.max_keys &&
           (long long)s + n <= (long long)p.kv.max_pages * KV8_PAGE;
}

// Lane (g, c)'s share of the 8-row query tile as the B operand of S^T = K Q^T: for each 64 dims h
// the 16 dims 64 h + 16 c .. of row g. fp16 rows go in as they are; a bf16 row is first divided by
// the power of two of its largest value (`mul` gives it back), so every element within 2^-17 of that
// is exact in fp16 and smaller ones are off by 2^-25 of it.
template <int HD, int DT>
__device__ __forceinline__ void load_q(const Kv8AttnP& p, bool valid, size_t off, int c, uint32_t (*qf)[2], float& mul) {
    uint32_t w[HD / 64][8];
#pragma unroll
    for (int h = 0; h < HD / 64; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (valid) v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + off + 64 * h + 16 * c + 8 * u);
            w[h][4 * u] = v.x;
            w[h][4 * u + 1] = v.y;
            w[h][4 * u + 2] = v.z;
            w[h][4 * u + 3] = v.w;
        }
    mul = 1.f;
    if (DT == QW_BF16) {
        float a = 0.f;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, fmaxf(fabsf(bf_lo(w[h][i])), fabsf(bf_hi(w[h][i]))));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int x = min(max(kv8_log2(a), -100), 100);
        mul = kv8_pow2(x);
        const float inv = kv8_pow2(-x);
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[h][i] = pack_h2(bf_lo(w[h][i]) * inv, bf_hi(w[h][i]) * inv);
    }
#pragma unroll
    for (int h = 0; h < HD / 64; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            qf[4 * h + k][0] = w[h][2 * k];
            qf[4 * h + k][1] = w[h][2 * k + 1];
        }
}

// The token of row r (0, 1: rows g and g + 8 of the MMA) of a lane: the order of the S^T rows is
// chosen so that transposing the weights leaves lane c with tokens 4 c .. 4 c + 3.
__device__ __forceinline__ int kv8_tok(int g, int r) { return 4 * (g >> 1) + (g & 1) + 2 * r; }

// The page's K codes as the A operand: a[step] of the HD / 16 steps.
template <int HD>
__device__ __forceinline__ void load_k(const uint8_t* codes, int g, int c, uint32_t (*a)[4]) {
#pragma unroll
    for (int h = 0; h < HD / 64; ++h) {
        uint4 u[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = kv8_tok(g, r);
            u[r] = *reinterpret_cast<const uint4*>(codes + t * HD + kv8_k_pos<HD>(t, 4 * h + c) * 16);
        }
        const uint32_t w0[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, w1[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[4 * h + k][0] = kv8_dec2(w0[k] & 0xFFFFu);
            a[4 * h + k][1] = kv8_dec2(w1[k] & 0xFFFFu);
            a[4 * h + k][2] = kv8_dec2(w0[k] >> 16);
            a[4 * h + k][3] = kv8_dec2(w1[k] >> 16);
        }
    }
}

// Pages of 16 rows (8 warps split the pages of one row tile).
template <int HD, int DT>
__global__ void __launch_bounds__(KR_WARPS * 32) k_kv8_attn_rows(const __grid_constant__ Kv8AttnP p) {
    constexpr int NT = KR_ROWS / 8, KS = HD / 16, DW = HD / 32;  // DW: words of 4 dims of a lane's V row share
    extern __shared__ float sm_o[];                              // [warps][16][HD]
    __shared__ float sm_m[KR_WARPS][KR_ROWS], sm_l[KR_WARPS][KR_ROWS];
    __shared__ int sm_bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int b = blockIdx.z, head = blockIdx.y, row0 = blockIdx.x * KR_ROWS;
    int s, r0, n;
    const bool alive = attn_entry(p, b, s, r0, n);
    if (!alive) {
        if (threadIdx.x == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        if (r0 < 0 || n < 0 || n > p.max_len || r0 > p.T - n) return;
    }
    const int rows = n * p.G;
    if (row0 >= rows) return;
    if (threadIdx.x == 0) sm_bad = !alive;
    __syncthreads();
    const int last_row = min(row0 + KR_ROWS, rows) - 1;
    const int n_pages = alive ? (s + last_row / p.G) / KV8_PAGE + 1 : 0;
    const int* table = p.kv.table + (size_t)b * p.kv.max_pages;

    uint32_t qf[NT][KS][2];
    float qmul[NT][2];   // of the lane's columns: rows 8 nt + 2 c, + 1
    int limit[NT][2];    // last visible position of the columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + 8 * nt + g;
        const bool v = r < rows;
        const int i = v ? r / p.G : 0, h = head * p.G + (v ? r % p.G : 0);
        float mul;
        load_q<HD, DT>(p, v, (size_t)(r0 + i) * p.ld_q + (size_t)h * HD, c, qf[nt], mul);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            qmul[nt][e] = __shfl_sync(0xffffffffu, mul, (2 * c + e) * 4) * p.scale_log2;
            const int rr = row0 + 8 * nt + 2 * c + e;
            limit[nt][e] = rr < rows ? s + rr / p.G : -1;
        }
    }
    float R[NT][2], l[NT][2], o[NT][2 * DW][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        R[nt][0] = R[nt][1] = -1e30f;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * DW; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    for (int pi = warp; pi < n_pages; pi += KR_WARPS) {
        const int page = table[pi];
        if (page < 0 || page >= p.kv.n_pages) {
            sm_bad = 1;
            continue;
        }
        const uint8_t* blk = p.kv.blocks + ((size_t)page * p.kv.n_kv + head) * Kv8<HD>::BLK;
        const float sk = reinterpret_cast<const float*>(blk + Kv8<HD>::SOFF)[0];
        const float sv = reinterpret_cast<const float*>(blk + Kv8<HD>::SOFF)[1];
        const int ev = kv8_log2(sv);
        const float inv_sv = kv8_pow2(-ev);
        uint32_t a[KS][4];
        load_k<HD>(blk, g, c, a);
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) mma16816(d, a[k], qf[nt][k][0], qf[nt][k][1]);
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = qmul[nt][e] * sk;
                const int p0 = pi * KV8_PAGE + kv8_tok(g, 0);
                float t0 = p0 <= limit[nt][e] ? fmaf(d[e], f, (float)ev) : -INFINITY;
                float t1 = p0 + 2 <= limit[nt][e] ? fmaf(d[2 + e], f, (float)ev) : -INFINITY;
                float m = fmaxf(t0, t1);
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                if (m > R[nt][e] + KV8_SLACK) {
                    const float al = ex2(R[nt][e] - m);
                    R[nt][e] = m;
                    l[nt][e] *= al;
#pragma unroll
                    for (int i = 0; i < 2 * DW; ++i) {
                        o[nt][i][e] *= al;
                        o[nt][i][2 + e] *= al;
                    }
                }
                w[e] = ex2(t0 - R[nt][e] + KV8_LIFT);
                w[2 + e] = ex2(t1 - R[nt][e] + KV8_LIFT);
                l[nt][e] += (w[e] + w[2 + e]) * inv_sv;
            }
            pb[nt][0] = movmatrix(pack_h2(w[0], w[1]));
            pb[nt][1] = movmatrix(pack_h2(w[2], w[3]));
        }
        // V: lane (g, c) takes dims HD/8 g .. of tokens 4 c + k; byte permutes pair two tokens of a dim
        uint32_t v[4][DW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 4 * c + k;
            const uint8_t* row = blk + Kv8<HD>::VOFF + t * HD;
            if (HD == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(row + kv8_v_pos<HD>(t, g) * 16);
                v[k][0] = u.x;
                v[k][1] = u.y;
                v[k][DW - 2] = u.z;
                v[k][DW - 1] = u.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(row + kv8_v_pos<HD>(t, g >> 1) * 16 + (g & 1) * 8);
                v[k][0] = u.x;
                v[k][1] = u.y;
            }
        }
#pragma unroll
        for (int w = 0; w < DW; ++w) {
            const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140), b01 = __byte_perm(v[0][w], v[1][w], 0x7362);
            const uint32_t a23 = __byte_perm(v[2][w], v[3][w], 0x5140), b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
            const uint32_t f0[4] = {kv8_dec2(a01 & 0xFFFFu), kv8_dec2(a01 >> 16), kv8_dec2(a23 & 0xFFFFu), kv8_dec2(a23 >> 16)};
            const uint32_t f1[4] = {kv8_dec2(b01 & 0xFFFFu), kv8_dec2(b01 >> 16), kv8_dec2(b23 & 0xFFFFu), kv8_dec2(b23 >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[nt][2 * w], f0, pb[nt][0], pb[nt][1]);
                mma16816(o[nt][2 * w + 1], f1, pb[nt][0], pb[nt][1]);
            }
        }
    }
    // ---- merge the warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = l[nt][e];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            const int r = 8 * nt + 2 * c + e;
            if (g == 0) {
                sm_m[warp][r] = R[nt][e];
                sm_l[warp][r] = x;
            }
            float* dst = sm_o + ((size_t)warp * KR_ROWS + r) * HD + g * (HD / 8);
#pragma unroll
            for (int i = 0; i < 2 * DW; ++i) {  // tile i: dims 2 i, 2 i + 1 of the lane's HD / 8
                dst[2 * i] = o[nt][i][e];
                dst[2 * i + 1] = o[nt][i][2 + e];
            }
        }
    __syncthreads();
    const bool bad = sm_bad;
    if (bad && threadIdx.x == 0) atomicOr(p.status, QW_KV8_BAD_POS);
    for (int x = threadIdx.x; x < KR_ROWS * HD / 2; x += KR_WARPS * 32) {
        const int r = x / (HD / 2), d = (x % (HD / 2)) * 2;
        if (row0 + r >= rows) break;
        float M = -1e30f;
        for (int w = 0; w < KR_WARPS; ++w) M = fmaxf(M, sm_m[w][r]);
        float L = 0.f, o0 = 0.f, o1 = 0.f;
        for (int w = 0; w < KR_WARPS; ++w) {
            const float f = ex2(sm_m[w][r] - M);
            L += sm_l[w][r] * f;
            o0 += sm_o[((size_t)w * KR_ROWS + r) * HD + d] * f;
            o1 += sm_o[((size_t)w * KR_ROWS + r) * HD + d + 1] * f;
        }
        const float inv = bad ? 0.f : 1.f / L;
        if (bad) o0 = o1 = 0.f;
        const int i = (row0 + r) / p.G, h = head * p.G + (row0 + r) % p.G;
        const uint32_t v = DT == QW_F16 ? pack_h2(o0 * inv, o1 * inv) : pack_bf2(o0 * inv, o1 * inv);
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)(r0 + i) * p.ld_out + (size_t)h * HD + d) = v;
        if (d == 0) {
            const float z = log2f(L) + M - KV8_LIFT;
            const size_t at = (size_t)(r0 + i) * p.n_heads + h;
            if (p.lse2) p.lse2[at] = bad ? __int_as_float(0x7fffffff) : z;
            if (p.lse) p.lse[at] = bad ? 0.f : z * KV8_LN2;
        }
    }
}

// Scores: score_out[j] = score_in[j] + sum over the rows of 2^(t_j - lse2). One warp per page: it
// keeps the page's K as the A operand and walks the query rows in tiles of 8.
template <int HD, int DT>
__global__ void __launch_bounds__(128) k_kv8_score(const __grid_constant__ Kv8AttnP p) {
    constexpr int KS = HD / 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int b = blockIdx.z, head = blockIdx.y, pi = blockIdx.x * 4 + warp;
    int s, r0, n;
    if (!attn_entry(p, b, s, r0, n) || n == 0 || pi * KV8_PAGE >= s + n) return;
    const int rows = n * p.G;
    const float z0 = p.lse2[(size_t)r0 * p.n_heads + head * p.G];
    if (__float_as_uint(z0) == 0x7fffffffu) return;  // an entry left out
    const int page = p.kv.table[(size_t)b * p.kv.max_pages + pi];
    if (page < 0 || page >= p.kv.n_pages) return;
    const uint8_t* blk = p.kv.blocks + ((size_t)page * p.kv.n_kv + head) * Kv8<HD>::BLK;
    const float sk = reinterpret_cast<const float*>(blk + Kv8<HD>::SOFF)[0];
    uint32_t a[KS][4];
    load_k<HD>(blk, g, c, a);
    const int p0 = pi * KV8_PAGE + kv8_tok(g, 0);
    float acc0 = 0.f, acc1 = 0.f;
    // rows of tokens before the page's first position see nothing of it
    const int first = max(0, pi * KV8_PAGE - s) * p.G;
    for (int row0 = first & ~7; row0 < rows; row0 += 8) {
        const int r = row0 + g;
        const bool v = r < rows;
        const int i = v ? r / p.G : 0, h = head * p.G + (v ? r % p.G : 0);
        uint32_t qf[KS][2];
        float mul;
        load_q<HD, DT>(p, v, (size_t)(r0 + i) * p.ld_q + (size_t)h * HD, c, qf, mul);
        const float z = v ? p.lse2[(size_t)(r0 + i) * p.n_heads + h] : 0.f;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) mma16816(d, a[k], qf[k][0], qf[k][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f = __shfl_sync(0xffffffffu, mul, (2 * c + e) * 4) * p.scale_log2 * sk;
            const float zc = __shfl_sync(0xffffffffu, z, (2 * c + e) * 4);
            const int rr = row0 + 2 * c + e, lim = rr < rows ? s + rr / p.G : -1;
            if (p0 <= lim) acc0 += ex2(fmaf(d[e], f, -zc));
            if (p0 + 2 <= lim) acc1 += ex2(fmaf(d[2 + e], f, -zc));
        }
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        acc0 += __shfl_xor_sync(0xffffffffu, acc0, m);
        acc1 += __shfl_xor_sync(0xffffffffu, acc1, m);
    }
    if (c < 2) {
        const int pos = p0 + 2 * c;
        if (pos < s + n) {
            const size_t at = ((size_t)b * p.kv.n_kv + head) * p.ld_score + pos;
            p.score_out[at] = (p.score_in ? p.score_in[at] : 0.f) + (c ? acc1 : acc0);
        }
    }
}

template <int HD, int DT>
cudaError_t run_attn(const Kv8AttnP& p, int B, cudaStream_t st) {
    const int smem = KR_WARPS * KR_ROWS * HD * 4;
    cudaError_t e = cudaFuncSetAttribute(k_kv8_attn_rows<HD, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCtx c = {st, false, nullptr};
    const int len = std::min(p.max_len, p.T);
    const unsigned tiles = (unsigned)(((long long)len * p.G + KR_ROWS - 1) / KR_ROWS);
    e = launch_k(c, k_kv8_attn_rows<HD, DT>, dim3(tiles, p.kv.n_kv, B), dim3(KR_WARPS * 32), (size_t)smem, p);
    if (e != cudaSuccess || !p.score_out) return e;
    const unsigned pages = (unsigned)((p.max_keys + KV8_PAGE - 1) / KV8_PAGE);
    return launch_k(c, k_kv8_score<HD, DT>, dim3((pages + 3) / 4, p.kv.n_kv, B), dim3(128), 0, p);
}

}  // namespace

static qw_status attn_sizes(const qw_kv8* kv, int B, int T, int max_len, int max_keys, int n_heads) {
    if (qw_status s = kv8_check(kv, B, "attn")) return s;
    if (T < 0 || max_len < 1 || max_len > (1 << 26)) return qw_fail(QW_ERR_INVALID_ARG, "attn: T or max_len out of range");
    if (max_keys < 1 || (long long)max_keys > (long long)kv->max_pages * 16)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: max_keys outside [1, 16 max_pages]");
    if (n_heads < kv->n_kv_heads || n_heads % kv->n_kv_heads)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: n_heads is not a multiple of n_kv_heads");
    if (n_heads / kv->n_kv_heads > 16) return qw_fail(QW_ERR_UNSUPPORTED, "attn: more than 16 query heads per KV head");
    return QW_OK;
}

extern "C" size_t qw_kv8_attn_ws_bytes(const qw_kv8* kv, int B, int T, int max_len, int max_keys, int n_heads,
                                       int with_score) {
    if (attn_sizes(kv, B, T, max_len, max_keys, n_heads)) return 0;
    return with_score ? (((size_t)T * n_heads * 4 + 255) & ~(size_t)255) : 256;
}

extern "C" qw_status qw_kv8_attn(const qw_kv8* kv, const qw_kv8_attn_args* a, void* stream) {
    if (!a) return qw_fail(QW_ERR_INVALID_ARG, "attn: args is NULL");
    if (qw_status s = attn_sizes(kv, a->B, a->T, a->max_len, a->max_keys, a->n_heads)) return s;
    if (!a->dev_start || !a->dev_cu || !a->dev_q || !a->dev_out || !a->dev_ws || !a->dev_status)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: NULL argument");
    if (a->dtype != QW_F16 && a->dtype != QW_BF16)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: dtype %d (QW_F16 and QW_BF16 are taken)", a->dtype);
    const size_t row = (size_t)a->n_heads * kv->head_dim;
    if (a->ld_q < row || a->ld_out < row) return qw_fail(QW_ERR_INVALID_ARG, "attn: row stride below n_heads * head_dim");
    if (((uintptr_t)a->dev_q | (uintptr_t)a->dev_out) & 15 || a->ld_q % 8 || a->ld_out % 8)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: rows not 16-byte aligned");
    if (!(a->scale > 0.f) || !(a->scale < 1e30f)) return qw_fail(QW_ERR_INVALID_ARG, "attn: scale not positive and finite");
    if (a->dev_score_in && !a->dev_score_out) return qw_fail(QW_ERR_INVALID_ARG, "attn: score_in without score_out");
    if (a->dev_score_out && a->ld_score < (size_t)a->max_keys) return qw_fail(QW_ERR_INVALID_ARG, "attn: ld_score < max_keys");
    if ((uintptr_t)a->dev_ws & 255 ||
        a->ws_bytes < qw_kv8_attn_ws_bytes(kv, a->B, a->T, a->max_len, a->max_keys, a->n_heads, a->dev_score_out != nullptr))
        return qw_fail(QW_ERR_INVALID_ARG, "attn: workspace too small or not 256-byte aligned");
    if (a->T == 0) return QW_OK;
    Kv8AttnP p = {};
    p.kv = kv8_view(kv);
    p.start = a->dev_start;
    p.cu = a->dev_cu;
    p.q = a->dev_q;
    p.ld_q = a->ld_q;
    p.T = a->T;
    p.max_len = a->max_len;
    p.max_keys = a->max_keys;
    p.n_heads = a->n_heads;
    p.G = a->n_heads / kv->n_kv_heads;
    p.scale_log2 = a->scale * KV8_LOG2E;
    p.out = a->dev_out;
    p.ld_out = a->ld_out;
    p.lse = a->dev_lse;
    p.lse2 = a->dev_score_out ? (float*)a->dev_ws : nullptr;
    p.score_in = a->dev_score_in;
    p.score_out = a->dev_score_out;
    p.ld_score = a->ld_score;
    p.status = a->dev_status;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = kv->head_dim == 128 ? (a->dtype == QW_F16 ? run_attn<128, QW_F16>(p, a->B, st) : run_attn<128, QW_BF16>(p, a->B, st))
                                              : (a->dtype == QW_F16 ? run_attn<64, QW_F16>(p, a->B, st) : run_attn<64, QW_BF16>(p, a->B, st));
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "attn: %s", cudaGetErrorString(e));
}
