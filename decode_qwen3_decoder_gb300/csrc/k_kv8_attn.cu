// Attention over the 8-bit paged KV cache (qw_kv8_attn).
//
// A query row (token i of an entry, one query head) at position p sees cached positions 0 .. p:
//   t_j = scale log2(e) 2^ek q.k_j,  out = sum_j 2^(t_j - m) 2^ev v_j / sum_j 2^(t_j - m)
// with the page's scales 2^ek, 2^ev and the codes k_j, v_j as the MMA operands: an e4m3 value
// is exact in fp16, so the products see exactly what the cache holds. The weight that goes into
// the PV product is w_j = 2^(t_j + ev_j - R + 8): the V scale joins the exponent, so pages of
// very different scales meet in one fp16 range, and the sum of the softmax takes w_j 2^-ev_j,
// in fp32. The reference R of a row moves only when a weight would pass 2^15. Two roundings below 32
// bits come before the output's. The weights' to fp16, the MMA's operand type (2^-11 each, 2^-25
// absolute where they are subnormal, against a largest weight of at least 2^8): against 64 bits fp16
// outputs are off by 2.1e-4 to 2.7e-4 in the mean, by 2.1e-4 with fp32 weights. And a bf16 query row's, whose
// elements below 2^-17 of its largest lose bits as fp16 (see row_operand). Exponentials are the
// hardware's (2^-22 relative).
#include "kv8.cuh"

#include <algorithm>
#include <type_traits>

#include "tc_sm103.cuh"

namespace {

constexpr float KV8_LOG2E = 1.4426950408889634f, KV8_LN2 = 0.6931471805599453f;
constexpr float KV8_LIFT = 8.f, KV8_SLACK = 7.f;  // weights aim at 2^8 and may grow to 2^15

struct Kv8AttnP {
    Kv8View kv;
    const int* start;
    const int* cu;
    const void* q;
    size_t ld_q;
    int T, max_len, max_keys, n_heads, G;
    uint32_t gmul;  // ceil(2^32 / G) (0: G = 1): row / G by a multiplication, exact for rows < 2^28
    float scale_log2;
    void* out;
    size_t ld_out;
    float* lse;   // optional
    float* lse2;  // optional: in log2 units, for the scores
    const float* score_in;
    float* score_out;
    size_t ld_score;
    int score_mul, score_add;  // see kv8_attn
    int* status;
};

__device__ __forceinline__ size_t score_row(const Kv8AttnP& p, int b, int head) {
    const size_t e = (size_t)p.score_mul * (p.kv.row ? p.kv.row[b] : b) + p.score_add;
    return (e * p.kv.n_kv + head) * p.ld_score;
}
// token of row r of an entry (rows are token major, G heads a token)
__device__ __forceinline__ int row_token(const Kv8AttnP& p, int r) { return p.gmul ? (int)__umulhi((uint32_t)r, p.gmul) : r; }

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

// Exponent of the power of two that a bf16 row with largest magnitude `a` is divided by; the range in which
// 2^e and 2^-e are both normal.
__device__ __forceinline__ int q_exponent(float a) { return min(max(kv8_log2(a), -126), 126); }

// Lane (g, c)'s share of the 8-row query tile as the B operand of S^T = K Q^T: for each 64 dims h
// the 16 dims 64 h + 16 c .. of row g. fp16 rows go in as they are; a bf16 row is first divided by
// the power of two of its largest value (`mul` gives it back), so every element within 2^-17 of that
// is exact in fp16 and smaller ones are off by 2^-25 of it.
template <int HD>
__device__ __forceinline__ void fetch_row(const Kv8AttnP& p, bool valid, size_t off, int c, uint4 (*w)[2]) {
#pragma unroll
    for (int h = 0; h < HD / 64; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[h][u] = make_uint4(0u, 0u, 0u, 0u);
            if (valid) w[h][u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + off + 64 * h + 16 * c + 8 * u);
        }
}
template <int HD, int DT>
__device__ __forceinline__ void row_operand(const uint4 (*x)[2], uint32_t (*qf)[2], float& mul) {
    uint32_t w[HD / 64][8];
#pragma unroll
    for (int h = 0; h < HD / 64; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[h][4 * u] = x[h][u].x;
            w[h][4 * u + 1] = x[h][u].y;
            w[h][4 * u + 2] = x[h][u].z;
            w[h][4 * u + 3] = x[h][u].w;
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
        const int e = q_exponent(a);
        mul = kv8_pow2(e);
        const float inv = kv8_pow2(-e);
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

// O^T += V^T P^T of one page. Lane (g, c) takes dims HD/8 g .. of tokens 4 c + k; byte permutes pair
// two tokens of a dim. Tile 2 w + u of the accumulators: dims 4 w + 2 u, + 1 of the lane's HD / 8.
template <int HD, int NT>
__device__ __forceinline__ void mma_pv(const uint8_t* codes, int g, int c, const uint32_t (*pb)[2], float (*o)[HD / 16][4]) {
    constexpr int DW = HD / 32;
    uint32_t v[4][DW];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = 4 * c + k;
        const uint8_t* row = codes + t * HD;
        if constexpr (HD == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + kv8_v_pos<HD>(t, g) * 16);
            v[k][0] = u.x;
            v[k][1] = u.y;
            v[k][2] = u.z;
            v[k][3] = u.w;
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

// One page's share of the online softmax for the lane's two columns of a tile: scores d (raw
// q.k) become weights for the PV product. f: logit factor; v0, v1: the two keys are visible.
template <int HD>
__device__ __forceinline__ void softmax_page(const float* d, const float* f, const bool* v0, const bool* v1, int ev, float inv_sv,
                                             float* R, float* l, float (*o)[4], uint32_t* pb) {
    float w[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float t0 = v0[e] ? fmaf(d[e], f[e], (float)ev) : -INFINITY;
        const float t1 = v1[e] ? fmaf(d[2 + e], f[e], (float)ev) : -INFINITY;
        float m = fmaxf(t0, t1);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (m > R[e] + KV8_SLACK) {
            const float al = ex2(R[e] - m);
            R[e] = m;
            l[e] *= al;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
                o[i][e] *= al;
                o[i][2 + e] *= al;
            }
        }
        w[e] = ex2(t0 - R[e] + KV8_LIFT);
        w[2 + e] = ex2(t1 - R[e] + KV8_LIFT);
        l[e] += (w[e] + w[2 + e]) * inv_sv;
    }
    pb[0] = movmatrix(pack_h2(w[0], w[1]));
    pb[1] = movmatrix(pack_h2(w[2], w[3]));
}

// =======================================================================================
// k_kv8_decode: few query rows per KV head (a decode step, up to 16 rows of tokens x heads).
//
// Reading the cache bounds it: 32 HD + 32 bytes per page and head, once. 8 sequences of 1k-32k tokens
// (289 MB): 53 us, 5.5 TB/s, of which ~6 are the start (lengths, page table, first pages) and ~4 the
// merges; 64 of 1100 tokens (143 MB): 32 us. The items (entry, KV head, page), entry-major, are cut into equal runs, one per CTA and
// again one per warp, so ragged lengths cost no imbalance and a warp needs no other warp: it
// streams its pages through its own ring with one bulk copy per block (codes and scales are
// contiguous), multiplies with the keys as the M of the MMA (16 keys of a page, 8 query rows as N)
// and keeps the online softmax in registers. A run that covers a whole (entry, head) pair writes
// the output; the pieces of a pair inside a CTA are merged in shared memory, and pairs that cross
// CTAs go through two partial slots per CTA, merged by k_kv8_combine (launched early, in the
// order of the slots, so sums have one order). With `pair_mode` (short caches) a CTA takes one
// pair and nothing is left to combine: 5 us for one sequence of 69 tokens, 10 without.
// With scores, the logits also go to `tbuf`, from which the combine kernel forms the weights
// once the normalisers are known: 8 bytes a row and key instead of K again.
// =======================================================================================
constexpr int KD_WARPS = 8;

struct Kv8DecP {
    Kv8AttnP a;
    int B, nrow;      // rows (max_len * G) a pair has at most
    int stages;
    int pair_mode;
    float* part_o;    // [CTAs][2][nrow][HD]
    float* part_ml;   // [CTAs][2][nrow][2]
    float* tbuf;      // optional [B * n_kv][nrow][ld_t] logits in log2 units
    size_t ld_t;
    int n_cta;        // CTAs of the decode kernel
};

// cum[b] = pages of the entries before b (b <= B), by all 256 threads of the CTA; with `ent` also
// (start, first row) of each entry.
__device__ __forceinline__ void kd_prefix(const Kv8AttnP& p, int B, int* cum, int* ws, int2* ent) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += KD_WARPS * 32) {
        int v = 0;
        if (b0 + tid < B) {
            int s, r0, n;
            const bool ok = attn_entry(p, b0 + tid, s, r0, n);
            v = ok && n > 0 ? (s + n + KV8_PAGE - 1) / KV8_PAGE : 0;
            if (ent) ent[b0 + tid] = make_int2(s, r0);
        }
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += t;
        }
        if (lane == 31) ws[w] = x;
        __syncthreads();
        int before = base, all = base;
#pragma unroll
        for (int i = 0; i < KD_WARPS; ++i) {
            if (i < w) before += ws[i];
            all += ws[i];
        }
        if (b0 + tid < B) cum[b0 + tid] = before + x - v;
        base = all;
        __syncthreads();
    }
    if (tid == 0) cum[B] = base;
    __syncthreads();
}

// The entry whose pages hold page number `pg` of all entries' pages laid end to end.
__device__ __forceinline__ int kd_find(const int* cum, int B, int pg) {
    int lo = 0, hi = B;  // cum[lo] <= pg < cum[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cum[m] <= pg) lo = m;
        else hi = m;
    }
    return lo;
}

// The items are cut into `runs` equal runs, CTA w taking items [kd_start(w), kd_start(w + 1)): one run a CTA, but no
// more runs than items, so every run has an item and its CTA writes each partial slot that the combine
// kernel reads. CTAs past the last run get none.
__device__ __forceinline__ int kd_runs(int items, int n_cta) { return max(1, min(items, n_cta)); }
__device__ __forceinline__ int kd_start(int items, int runs, int w) { return (int)((long long)items * min(w, runs) / runs); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Two output elements. A value next to 65504 is held as 65536 (see kv8.cuh), so fp16 outputs stop at 65504 as
// values read back do; NaN stays NaN.
template <int DT>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
    if (DT == QW_BF16) return pack_bf2(lo, hi);
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2 N consecutive output elements of one row from fp32 (N words, 16-byte aligned).
template <int DT, int N>
__device__ __forceinline__ void store_row(void* base, size_t off, const float* x) {
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = pack_out<DT>(x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + off + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

template <int HD, int DT, int NT>
__global__ void __launch_bounds__(KD_WARPS * 32, NT == 1 ? 2 : 1) k_kv8_decode(const __grid_constant__ Kv8DecP P) {
    constexpr int KS = HD / 16, BLK = Kv8<HD>::BLK, LD = HD / 8;  // LD: output dims of a lane
    const Kv8AttnP& p = P.a;
    extern __shared__ __align__(128) uint8_t kd_smem[];  // [warps][stages][BLK], the slots, then [B] (start, first row)
    __shared__ uint64_t bars[KD_WARPS][8];
    __shared__ int cum[QW_KV8_MAX_BATCH + 1];
    __shared__ int ws[KD_WARPS], slot_pair[2 * KD_WARPS], s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_launch();
    const int H = p.kv.n_kv, S = P.stages;
    float* slot_o = reinterpret_cast<float*>(kd_smem + (size_t)KD_WARPS * S * BLK);  // [warps][2][nrow][HD]
    float* slot_ml = slot_o + (size_t)2 * KD_WARPS * P.nrow * HD;                    // [warps][2][nrow][2]
    int2* ent = reinterpret_cast<int2*>(slot_ml + (size_t)2 * KD_WARPS * P.nrow * 2);
    if (lane == 0)
        for (int i = 0; i < S; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    if (tid == 0) {
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < 2 * KD_WARPS) slot_pair[tid] = -1;
    // ---- this CTA's and this warp's run of items ----
    int c0, c1;
    // entry of the pair that the warp works on: b, its start, first row and rows of a KV head
    int b = 0, head = 0, page = 0, pages = 0, s = 0, r0 = 0, rows = 0;
    if (P.pair_mode) {
        int n;
        b = blockIdx.x / H;
        head = blockIdx.x % H;
        const bool ok = attn_entry(p, b, s, r0, n);
        rows = n * p.G;
        c0 = 0;
        c1 = ok && n > 0 ? (s + n + KV8_PAGE - 1) / KV8_PAGE : 0;
    } else {
        kd_prefix(p, P.B, cum, ws, ent);
        const int items = cum[P.B] * H, runs = kd_runs(items, gridDim.x);
        c0 = kd_start(items, runs, blockIdx.x);
        c1 = kd_start(items, runs, blockIdx.x + 1);
    }
    if (blockIdx.x == 0 && !P.pair_mode)  // entries left out: reported, their rows zeroed
        for (int b = warp; b < P.B; b += KD_WARPS) {
            int s, r0, n;
            if (attn_entry(p, b, s, r0, n)) continue;
            if (lane == 0) atomicOr(p.status, QW_KV8_BAD_POS);
            if (r0 < 0 || n < 0 || n > p.max_len || r0 > p.T - n) continue;
            for (int i = 0; i < n; ++i)
                for (int d = lane * 8; d < p.n_heads * HD; d += 256)
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)(r0 + i) * p.ld_out + d) = make_uint4(0u, 0u, 0u, 0u);
        }
    if (P.pair_mode && c1 == 0) {
        int n;
        if (!attn_entry(p, b, s, r0, n)) {
            if (tid == 0) atomicOr(p.status, QW_KV8_BAD_POS);
            if (r0 < 0 || n < 0 || n > p.max_len || r0 > p.T - n) return;
            for (int x = tid; x < n * p.G * HD; x += KD_WARPS * 32) {
                const int r = x / HD;
                reinterpret_cast<uint16_t*>(p.out)[(size_t)(r0 + r / p.G) * p.ld_out + (size_t)(head * p.G + r % p.G) * HD + x % HD] = 0;
            }
        }
        return;
    }
    __syncthreads();
    const int i0 = c0 + (int)((long long)(c1 - c0) * warp / KD_WARPS), i1 = c0 + (int)((long long)(c1 - c0) * (warp + 1) / KD_WARPS);
    auto locate = [&](int j, int& b, int& head, int& page, int& pages) {
        if (P.pair_mode) {
            page = j;
            pages = c1;
        } else {
            b = kd_find(cum, P.B, j / H);
            pages = cum[b + 1] - cum[b];
            const int off = j - cum[b] * H;
            head = off / pages;
            page = off - head * pages;
        }
    };
    uint4 qx[NT][HD / 64][2];
    // the pair of item j: where it begins, and its query rows on the way
    auto enter = [&](int j) {
        locate(j, b, head, page, pages);
        if (!P.pair_mode) {
            s = ent[b].x;
            r0 = ent[b].y;
            rows = (p.cu[b + 1] - r0) * p.G;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const bool v = r < rows;
            const int i = v ? row_token(p, r) : 0, h = head * p.G + (v ? r - i * p.G : 0);
            fetch_row<HD>(p, v, (size_t)(r0 + i) * p.ld_q + (size_t)h * HD, c, qx[nt]);
        }
    };
    if (i0 < i1) enter(i0);  // before the page table and the first pages, which take as long
    const uint32_t ring = smem_u32(kd_smem) + warp * S * BLK;
    // lane l holds the block address of the l-th item of the batch of 32 being issued, and of the next
    auto address = [&](int j) -> const uint8_t* {
        if (j >= i1) return nullptr;
        int b2 = b, head2 = head, page2, pages2;
        locate(j, b2, head2, page2, pages2);
        int id = kv8_row(p.kv, p.kv.table, b2)[page2];
        if (id < 0 || id >= p.kv.n_pages) {
            atomicOr(p.status, QW_KV8_BAD_POS);
            id = 0;
        }
        return kv8_block(p.kv, b2, id, head2, BLK);
    };
    const uint8_t* cur = address(i0 + lane);
    const uint8_t* nxt = address(i0 + 32 + lane);
    int issued = 0;
    auto issue = [&](int st) {
        if (i0 + issued >= i1) return;
        if (issued && (issued & 31) == 0) {
            cur = nxt;
            nxt = address(i0 + issued + 32 + lane);
        }
        if (lane == (issued & 31)) {
            const uint32_t bar = smem_u32(&bars[warp][st]);
            mbar_expect_tx(bar, BLK);
            bulk_copy(ring + st * BLK, cur, BLK, bar);
        }
        ++issued;
    };
    for (int i = 0; i < S; ++i) issue(i);

    uint32_t qf[NT][KS][2];
    float qmul[NT][2], R[NT][2], l[NT][2], o[NT][KS][4];
    int limit[NT][2];
    int page_lo = 0, n_slots = 0;
    auto flush = [&]() {  // the segment [page_lo, page) of the pair (b, head)
        const bool whole = page_lo == 0 && page == pages;
        const int slot = warp * 2 + n_slots;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int r = 8 * nt + 2 * c + e;
                if (r >= rows) continue;
                float v[LD];
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    v[2 * i] = o[nt][i][e];
                    v[2 * i + 1] = o[nt][i][2 + e];
                }
                if (whole) {
                    const float inv = 1.f / x;
#pragma unroll
                    for (int i = 0; i < LD; ++i) v[i] *= inv;
                    const int i = row_token(p, r), tok = r0 + i, h = head * p.G + r - i * p.G;
                    store_row<DT, LD / 2>(p.out, (size_t)tok * p.ld_out + (size_t)h * HD + g * LD, v);
                    if (g == 0) {
                        const float z = log2f(x) + R[nt][e] - KV8_LIFT;
                        if (p.lse2) p.lse2[(size_t)tok * p.n_heads + h] = z;
                        if (p.lse) p.lse[(size_t)tok * p.n_heads + h] = z * KV8_LN2;
                    }
                } else {
                    float* dst = slot_o + ((size_t)slot * P.nrow + r) * HD + g * LD;
#pragma unroll
                    for (int i = 0; i < LD; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    if (g == 0) {
                        slot_ml[((size_t)slot * P.nrow + r) * 2] = R[nt][e];
                        slot_ml[((size_t)slot * P.nrow + r) * 2 + 1] = x;
                    }
                }
            }
        if (!whole) {
            if (lane == 0) slot_pair[slot] = b * H + head;
            ++n_slots;
        }
    };
    auto begin = [&]() {
        page_lo = page;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mul;
            row_operand<HD, DT>(qx[nt], qf[nt], mul);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qmul[nt][e] = __shfl_sync(0xffffffffu, mul, (2 * c + e) * 4) * p.scale_log2;
                const int rr = 8 * nt + 2 * c + e;
                limit[nt][e] = rr < rows ? s + row_token(p, rr) : -1;
                R[nt][e] = -1e30f;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int i2 = 0; i2 < KS; ++i2) o[nt][i2][0] = o[nt][i2][1] = o[nt][i2][2] = o[nt][i2][3] = 0.f;
        }
    };
    if (i0 < i1) begin();
    int st = 0, ph = 0;
    for (int j = i0; j < i1; ++j) {
        if (page == pages) {
            flush();
            enter(j);
            begin();
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), ph, &s_abort))) {
            // give up: the outputs are not valid. The copies in flight land before the CTA ends.
            if (lane == 0) {
                atomicOr(p.status, QW_KV8_TIMEOUT);
                s_abort = 1;
            }
            const uint64_t t0 = globaltimer_ns();
            for (int k = j; k < i0 + issued; ++k) {
                while (!mbar_try_wait(smem_u32(&bars[warp][st]), ph) && globaltimer_ns() - t0 < kTcWaitNs) {
                }
                if (++st == S) {
                    st = 0;
                    ph ^= 1;
                }
            }
            break;
        }
        const uint8_t* blk = kd_smem + ((size_t)warp * S + st) * BLK;
        const float2 sc = *reinterpret_cast<const float2*>(blk + Kv8<HD>::SOFF);
        const int ev = kv8_log2(sc.y);
        const float inv_sv = kv8_pow2(-ev);
        uint32_t a[KS][4], pb[NT][2];
        load_k<HD>(blk, g, c, a);
        const int p0 = page * KV8_PAGE + kv8_tok(g, 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) mma16816(d, a[k], qf[nt][k][0], qf[nt][k][1]);
            const float f[2] = {qmul[nt][0] * sc.x, qmul[nt][1] * sc.x};
            const bool v0[2] = {p0 <= limit[nt][0], p0 <= limit[nt][1]}, v1[2] = {p0 + 2 <= limit[nt][0], p0 + 2 <= limit[nt][1]};
            if (P.tbuf) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* tr = P.tbuf + ((size_t)(b * H + head) * P.nrow + 8 * nt + 2 * c + e) * P.ld_t + p0;
                    if (v0[e]) tr[0] = d[e] * f[e];
                    if (v1[e]) tr[2] = d[2 + e] * f[e];
                }
            }
            softmax_page<HD>(d, f, v0, v1, ev, inv_sv, R[nt], l[nt], o[nt], pb[nt]);
        }
        mma_pv<HD, NT>(blk + Kv8<HD>::VOFF, g, c, pb, o);
        __syncwarp();
        issue(st);
        ++page;
        if (++st == S) {
            st = 0;
            ph ^= 1;
        }
    }
    if (i1 > i0 && !s_abort) flush();
    __syncthreads();
    if (s_abort) return;
    // ---- merge the pieces of a pair that several warps hold ----
    // Lane k < 16 holds slot k's pair; `heads` marks the first slot of each pair (slots are in item order).
    const int mine = lane < 2 * KD_WARPS ? slot_pair[lane] : -1;
    const uint32_t used = __ballot_sync(0xffffffffu, mine >= 0);
    const uint32_t below = used & ((1u << lane) - 1u);
    const int before = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : 0);
    const uint32_t heads = __ballot_sync(0xffffffffu, mine >= 0 && (!below || before != mine));
    const int per = P.nrow * (HD / 4), total = __popc(heads) * per;  // groups x (row, 4 dims)
    for (int x0 = 0; x0 < total; x0 += KD_WARPS * 32) {
        const int x = x0 + tid, gi = min(x, total - 1) / per, y = min(x, total - 1) - gi * per;
        uint32_t m = heads;
        for (int i = 0; i < gi; ++i) m &= m - 1;
        const int a0 = __ffs(m) - 1;
        m &= m - 1;
        const int a1 = m ? __ffs(m) - 1 : 2 * KD_WARPS;
        const int pair = slot_pair[a0], eb = P.pair_mode ? b : pair / H, eh = P.pair_mode ? head : pair - eb * H;
        const int er0 = P.pair_mode ? r0 : ent[eb].y, erows = P.pair_mode ? rows : (p.cu[eb + 1] - er0) * p.G;
        const int r = y / (HD / 4), d = (y - r * (HD / 4)) * 4;
        if (x >= total || r >= erows) continue;
        int first = 0, last = c1;  // the pair's items
        if (!P.pair_mode) {
            const int np = cum[eb + 1] - cum[eb];
            first = cum[eb] * H + eh * np;
            last = first + np;
        }
        float M = -1e30f, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = a0; k < a1; ++k) {
            if (!(used >> k & 1)) continue;
            const float2 ml = *reinterpret_cast<const float2*>(slot_ml + ((size_t)k * P.nrow + r) * 2);
            const float4 v = *reinterpret_cast<const float4*>(slot_o + ((size_t)k * P.nrow + r) * HD + d);
            const float mm = fmaxf(M, ml.x), fo = ex2(M - mm), fn = ex2(ml.x - mm);
            M = mm;
            L = L * fo + ml.y * fn;
            acc.x = acc.x * fo + v.x * fn;
            acc.y = acc.y * fo + v.y * fn;
            acc.z = acc.z * fo + v.z * fn;
            acc.w = acc.w * fo + v.w * fn;
        }
        if (first >= c0 && last <= c1) {
            const float inv = 1.f / L;
            const int i = row_token(p, r), tok = er0 + i, h = eh * p.G + r - i * p.G;
            uint2 w;
            w.x = pack_out<DT>(acc.x * inv, acc.y * inv);
            w.y = pack_out<DT>(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)tok * p.ld_out + (size_t)h * HD + d) = w;
            if (d == 0) {
                const float z = log2f(L) + M - KV8_LIFT;
                if (p.lse2) p.lse2[(size_t)tok * p.n_heads + h] = z;
                if (p.lse) p.lse[(size_t)tok * p.n_heads + h] = z * KV8_LN2;
            }
        } else {
            const size_t at = ((size_t)blockIdx.x * 2 + (first > c0 ? 1 : 0)) * P.nrow + r;
            *reinterpret_cast<float4*>(P.part_o + at * HD + d) = acc;
            if (d == 0) {
                P.part_ml[at * 2] = M;
                P.part_ml[at * 2 + 1] = L;
            }
        }
    }
}

// Pairs that cross CTAs of k_kv8_decode: out = sum of the slots' partials. First a warp a row and a lane
// a slot find each row's maximum and sum, then the warps add the slots' values and one exchange through
// shared memory joins them. Few pairs deal their rows to several CTAs (blockIdx.y): one CTA with all 16
// rows of 38 slots took 30 us. Many have one CTA each: 512 pairs of 16 rows with a CTA a row took 25 us
// longer. With scores a pair has a CTA for each KC_KEYS keys, which also forms their weights from the
// stored logits, four keys a thread.
constexpr int KC_KEYS = 1024;
inline int kc_smem(int nrow, int hd) { return KD_WARPS * nrow * hd * 4; }

template <int HD, int DT>
__global__ void __launch_bounds__(KD_WARPS * 32) k_kv8_combine(const __grid_constant__ Kv8DecP P) {
    const Kv8AttnP& p = P.a;
    extern __shared__ __align__(16) float kc_o[];  // [own rows][warps a row][HD]
    __shared__ int cum[QW_KV8_MAX_BATCH + 1];
    __shared__ int ws[KD_WARPS];
    __shared__ float s_m[16], s_l[16], s_z[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.kv.n_kv;
    const int b = blockIdx.x / H, head = blockIdx.x % H, key0 = blockIdx.y * KC_KEYS;
    pdl_launch();
    int s, r0, n;
    const bool on = attn_entry(p, b, s, r0, n) && n > 0 && (!p.score_out || key0 < s + n);
    const int rows = n * p.G;
    bool split = false;
    int w0 = 0, w1 = 0, first = 0, items = 0, runs = 0;
    if (on && !P.pair_mode) {
        kd_prefix(p, P.B, cum, ws, nullptr);
        items = cum[P.B] * H;
        runs = kd_runs(items, P.n_cta);
        const int np = cum[b + 1] - cum[b];
        first = cum[b] * H + head * np;
        w0 = (int)((((long long)first + 1) * runs - 1) / items);
        w1 = (int)((((long long)first + np) * runs - 1) / items);
        split = w1 > w0;
    }
    pdl_wait();  // in every CTA: what follows this kernel must not pass the one before it
    if (!on || (!split && !p.score_out)) return;
    if (split) {
        // this CTA's rows: y, y + ny, ...
        const int y = blockIdx.y, ny = p.score_out ? (s + n + KC_KEYS - 1) / KC_KEYS : (int)gridDim.y;
        auto slot = [&](int w) {  // of the pair in CTA w
            return ((size_t)w * 2 + (kd_start(items, runs, w) >= first ? 0 : 1)) * P.nrow;
        };
        for (int r = warp; r < rows; r += KD_WARPS) {
            float M = -1e30f, L = 0.f;
            for (int w = w0 + lane; w <= w1; w += 32) {
                const float2 x = *reinterpret_cast<const float2*>(P.part_ml + (slot(w) + r) * 2);
                const float m = fmaxf(M, x.x);
                L = L * ex2(M - m) + x.y * ex2(x.x - m);
                M = m;
            }
            float m = M;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            L *= ex2(M - m);
#pragma unroll
            for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            if (lane == 0) {
                s_m[r] = m;
                s_l[r] = L;
                s_z[r] = log2f(L) + m - KV8_LIFT;
            }
        }
        __syncthreads();
        int per = 1;  // warps a row: as many as it has slots, the others take other rows
        while (per < KD_WARPS && per <= w1 - w0) per <<= 1;
        const int own = rows > y ? (rows - y + ny - 1) / ny : 0;
        if (lane < HD / 4)
            for (int k = warp / per; k < own; k += KD_WARPS / per) {
                const int r = y + k * ny;
                const float m = s_m[r];
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int w = w0 + warp % per; w <= w1; w += per) {
                    const size_t at = slot(w) + r;
                    const float f = ex2(P.part_ml[at * 2] - m);
                    const float4 v = *reinterpret_cast<const float4*>(P.part_o + at * HD + lane * 4);
                    acc.x += v.x * f;
                    acc.y += v.y * f;
                    acc.z += v.z * f;
                    acc.w += v.w * f;
                }
                *reinterpret_cast<float4*>(kc_o + ((size_t)k * per + warp % per) * HD + lane * 4) = acc;
            }
        __syncthreads();
        for (int x = tid; x < own * (HD / 4); x += KD_WARPS * 32) {
            const int k = x / (HD / 4), r = y + k * ny, d = (x - k * (HD / 4)) * 4;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < per; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(kc_o + ((size_t)k * per + w) * HD + d);
                t.x += v.x;
                t.y += v.y;
                t.z += v.z;
                t.w += v.w;
            }
            const float inv = 1.f / s_l[r];
            const int tok = r0 + r / p.G, h = head * p.G + r % p.G;
            uint2 w;
            w.x = pack_out<DT>(t.x * inv, t.y * inv);
            w.y = pack_out<DT>(t.z * inv, t.w * inv);
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)tok * p.ld_out + (size_t)h * HD + d) = w;
            if (d == 0 && p.lse) p.lse[(size_t)tok * p.n_heads + h] = s_z[r] * KV8_LN2;
            if (d == 0 && p.lse2 && !p.score_out) p.lse2[(size_t)tok * p.n_heads + h] = s_z[r];
        }
    } else if (tid < rows) {
        s_z[tid] = p.lse2[(size_t)(r0 + tid / p.G) * p.n_heads + head * p.G + tid % p.G];
    }
    if (!p.score_out || kv8_stopped(p.kv, b)) return;
    const size_t base = score_row(p, b, head);
    const int j = key0 + tid * 4, end = s + n;
    float in[4] = {0.f, 0.f, 0.f, 0.f};
    float4 t[8];  // the logits are stored for at most 8 rows
    if (j < end) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < rows) t[r] = *reinterpret_cast<const float4*>(P.tbuf + ((size_t)(b * H + head) * P.nrow + r) * P.ld_t + j);
        if (p.score_in)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < end) in[k] = p.score_in[base + j + k];
    }
    __syncthreads();
    if (j >= end) return;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (r >= rows) break;
        const float z = s_z[r];
        const int lim = s + r / p.G;  // keys past it have no logit of this row
        const float v[4] = {t[r].x, t[r].y, t[r].z, t[r].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += j + k <= lim ? ex2(v[k] - z) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (j + k < end) p.score_out[base + j + k] = in[k] + acc[k];
}

// =======================================================================================
// k_kv8_chunk: many query rows (prompts and chunks of them) on tcgen05.
//
// A CTA takes two tiles of 128 rows of one (entry, KV head): rows are (token, head of the group)
// pairs, token major, so any group size fills the MMA. Per step of 128 keys (8 pages):
//   copies         a lane a page brings the codes with bulk copies through a ring (a block's K and
//                  its V are contiguous, so no tensor map is needed) and the page's scales;
//   converters     four warps: codes -> fp16 operands for both row tiles, K and V alike as
//                  [key][dim] rows in the 128-byte swizzle;
//   S = Q K^T      S in TMEM, 128 columns a row tile;
//   softmax        four warps a row tile, thread = row = TMEM lane, its 128 scores in registers;
//                  the page scales enter the exponent's FMA, P (fp16) overwrites half of S;
//   O += P V       A = P from TMEM, B = V, O in TMEM.
// Each row tile has its own issuing warp, and a step's keys go in two halves of 64: while the softmax
// works on one, P V and the next step's S of the other run (whole steps in turn took 1.13 to 1.2 times as long).
// Registers go by role (setmaxnreg). When the rows give too few CTAs, the keys are split (`splits`)
// and k_kv8_chunk_combine adds the partials in order. Every wait is bounded.
//
// What bounds it: a CTA's start and end. Of 512-token prompts (16 of them, 8 KV heads of 2, head_dim
// 128: 48 us, 17 GFLOP and 84 MB) a CTA's 12 us are 4 until its first S (all CTAs fetch their queries
// at the same time), 5 for its 2.5 steps, 2 for the output and 1 to the next CTA; a second query
// buffer, which would overlap them, does not fit beside the operands. Long caches: a step of 128 keys
// x 256 rows takes 1.7 us (head_dim 64; 2 chunks of 500 tokens x 28 heads over 6k-9k keys, 54 GFLOP:
// 102 us, 530 TFLOP/s, and 12 to add the partials of 4 splits), of which the softmax, the conversion
// and the MMAs each hide behind the others' hand-overs (taking one out gains at most a tenth).
// =======================================================================================
constexpr int CT_THREADS = 512;        // warps 0-3, 4-7 softmax; 8-11 converters; 12, 13 MMA; 14 copies; 15 idle
constexpr int CT_REGS = 128;           // a thread's at launch: 512 x 128 = 128 x (176 + 176 + 104 + 56)
constexpr int CT_BK = 128, CT_ROWS = 128;
constexpr int CT_SUB = 128 * 128;      // [128 rows][64 dims] fp16, swizzled
constexpr int CT_TMEM = 512, CT_O = 256;

template <int HD>
struct Ct {
    static constexpr int MAT = CT_SUB * (HD / 64), RAW = CT_BK * HD;
    static constexpr int RING = HD == 128 ? 5 : 8;  // code tiles (K or V) in flight
    static constexpr int NB = HD == 128 ? 1 : 2;    // operand buffers of K and of V
    static constexpr int OFF_K = 2 * MAT, OFF_V = OFF_K + NB * MAT, OFF_R = OFF_V + NB * MAT;
    static constexpr int OFF_MUL = OFF_R + RING * RAW, OFF_SC = OFF_MUL + 2 * CT_ROWS * 4, OFF_BAR = OFF_SC + 8 * 8 * 16;
    static constexpr int SMEM = 1024 + OFF_BAR + 512;
};

// mbar_wait that looks at the clock only after 64 failed tries.
__device__ __forceinline__ bool ct_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
    for (int n = 0; n < 64; ++n)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, abort_flag);
}

struct Kv8ChunkP {
    Kv8AttnP a;
    int splits;
    float* part_o;   // [B * n_kv][tiles][splits][HD / 4][128][4]: a warp, with a row a lane, writes whole lines
    float* part_ml;  // [B * n_kv][tiles][splits][128][2]
    int tiles;
};

__device__ __forceinline__ float fl(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// pairs of fp32 in one 64-bit register: one instruction for two operations
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Rows [row0, row0 + 128) of an entry's (token, head) rows as a swizzled fp16 operand, by four warps
// (w = 0 .. 3), fetched into registers and given to sink(byte offset, 16 bytes): HD / 8 lanes take a
// row's 16-byte chunks, so a request covers whole rows. A bf16 row is divided by the power of two of its largest
// value (see row_operand), which goes to put(row, mul); rows past the entry are zeros.
template <int HD>
struct QTile {
    static constexpr int LPR = HD / 8, RPI = 32 / LPR, NI = 32 / RPI;  // lanes a row, rows a request, requests a warp
    uint4 x[NI];
};
template <int HD>
__device__ __forceinline__ void fetch_q(QTile<HD>& q, const Kv8AttnP& p, int r0, int head, int row0, int rows, int w, int lane) {
    const int ch = lane % QTile<HD>::LPR, rw = w * 32 + lane / QTile<HD>::LPR;
#pragma unroll
    for (int i = 0; i < QTile<HD>::NI; ++i) {
        const int row = row0 + rw + i * QTile<HD>::RPI, tok = row_token(p, row);
        q.x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
            q.x[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + (size_t)(r0 + tok) * p.ld_q +
                                                     (size_t)(head * p.G + row - tok * p.G) * HD + ch * 8);
    }
}
template <int HD, int DT, typename Sink, typename Put>
__device__ __forceinline__ void store_q(QTile<HD>& q, int w, int lane, Sink sink, Put put) {
    constexpr int LPR = QTile<HD>::LPR;
    const int ch = lane % LPR, rw = w * 32 + lane / LPR;
#pragma unroll
    for (int i = 0; i < QTile<HD>::NI; ++i) {
        const int r = rw + i * QTile<HD>::RPI;
        float mul = 1.f;
        uint4& x = q.x[i];
        if (DT == QW_BF16) {
            uint32_t v[4] = {x.x, x.y, x.z, x.w};
            float am = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) am = fmaxf(am, fmaxf(fabsf(bf_lo(v[k])), fabsf(bf_hi(v[k]))));
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int e = q_exponent(am);
            mul = kv8_pow2(e);
            const float inv = kv8_pow2(-e);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = pack_h2(bf_lo(v[k]) * inv, bf_hi(v[k]) * inv);
            x = make_uint4(v[0], v[1], v[2], v[3]);
        }
        sink((ch >> 3) * CT_SUB + r * 128 + (((ch & 7) ^ (r & 7)) << 4), x);
        if (ch == 0) put(r, mul);
    }
}

template <int HD, int DT>
__global__ void __launch_bounds__(CT_THREADS, 1) k_kv8_chunk(const __grid_constant__ Kv8ChunkP P) {
    const Kv8AttnP& p = P.a;
    constexpr int NSUB = HD / 64, CH = HD / 16, RP = 128 / CH, NU = CT_BK / RP, MAT = Ct<HD>::MAT, NB = Ct<HD>::NB, RAW = Ct<HD>::RAW, RING = Ct<HD>::RING;
    extern __shared__ uint8_t ct_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ct_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ct<HD>::OFF_BAR);
    uint64_t *r_full = bars, *r_empty = bars + 8, *k_full = bars + 16, *k_empty = bars + 18, *v_full = bars + 20, *v_empty = bars + 22;
    uint64_t *s_full = bars + 24, *p_full = bars + 28, *pv_done = bars + 32, *q_ready = bars + 34, *mma_fin = bars + 36;  // s, p: [t][half]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 38);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float4* scales = reinterpret_cast<float4*>(sm + Ct<HD>::OFF_SC);  // [8][8]: 2^ek, ev, 2^-ev of the pages of step i % 8
    pdl_wait();
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, head = blockIdx.x;
    const int tile = (P.tiles + 1) / 2 - 1 - (int)(blockIdx.z / P.splits), split = blockIdx.z % P.splits;  // the longest rows start first
    const int row0 = tile * 2 * CT_ROWS;
    int s, r0, n;
    if (!attn_entry(p, b, s, r0, n)) {
        if (threadIdx.x == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        if (split || r0 < 0 || n < 0 || n > p.max_len || r0 > p.T - n) return;
        const int rows = n * p.G;
        for (int x = threadIdx.x; x < 2 * CT_ROWS * (HD / 8); x += CT_THREADS) {
            const int r = row0 + x / (HD / 8);
            if (r >= rows) break;
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)(r0 + r / p.G) * p.ld_out +
                                      (size_t)(head * p.G + r % p.G) * HD + (x % (HD / 8)) * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int rows = n * p.G;
    if (row0 >= rows) return;
    const int n_rt = row0 + CT_ROWS < rows ? 2 : 1;                      // row tiles with rows
    const int kend = s + (min(row0 + 2 * CT_ROWS, rows) - 1) / p.G + 1;  // keys the last row sees
    const int n_kt = (kend + CT_BK - 1) / CT_BK;
    const int j0 = (int)((long long)n_kt * split / P.splits), j1 = (int)((long long)n_kt * (split + 1) / P.splits), nt = j1 - j0;
    // partials of row tile t: part(t) [128 rows]
    auto part = [&](int t) { return (((size_t)b * p.kv.n_kv + head) * P.tiles + 2 * tile + t) * P.splits + split; };
    if (nt == 0) {  // nothing to add
        const int t = threadIdx.x / CT_ROWS;
        if (t < n_rt) {
            P.part_ml[(part(t) * CT_ROWS + threadIdx.x % CT_ROWS) * 2] = -1e30f;
            P.part_ml[(part(t) * CT_ROWS + threadIdx.x % CT_ROWS) * 2 + 1] = 0.f;
        }
        return;
    }
    // the first pages' table entries come while barriers and TMEM are set up
    const int* table = kv8_row(p.kv, p.kv.table, b);
    const int page_end = min((kend + KV8_PAGE - 1) / KV8_PAGE, j1 * 8);
    int first_id = 0;
    if (warp == 14 && j0 * 8 + lane < page_end) first_id = table[j0 * 8 + lane];
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(smem_u32(r_full + i), 1);
            mbar_init(smem_u32(r_empty + i), 4);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(smem_u32(k_full + i), 4);
            mbar_init(smem_u32(k_empty + i), n_rt);
            mbar_init(smem_u32(v_full + i), 4);
            mbar_init(smem_u32(v_empty + i), n_rt);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(s_full + i), 1);
            mbar_init(smem_u32(p_full + i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(pv_done + i), 1);
            mbar_init(smem_u32(q_ready + i), 4);
            mbar_init(smem_u32(mma_fin + i), 1);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(CT_TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // warp-uniform outcome of a bounded wait
    auto wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xffffffffu, ct_wait(smem_u32(bar), (uint32_t)parity & 1u, abort_flag));
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 14) {
            // ---------------- copies: lane l brings page l % 8 of steps 4 q + l / 8 ----------------
            // Table entries and scales come for four steps at once, ahead of their use, and the copies go out
            // before the scales are needed.
            bool ok = true;
            int st = 0, use = 0, issued = 0;  // ring stage and its use count
            auto block_of = [&](int q) -> const uint8_t* {
                const int pi = j0 * 8 + q * 32 + lane;
                if (pi >= page_end) return nullptr;
                int id = q ? table[pi] : first_id;
                if (id < 0 || id >= p.kv.n_pages) {
                    atomicOr(p.status, QW_KV8_BAD_POS);
                    id = 0;
                }
                return kv8_block(p.kv, b, id, head, Kv8<HD>::BLK);
            };
            // of no page 1 and 1: masked scores stay -inf
            auto scale_of = [&](const uint8_t* blk) {
                return blk ? *reinterpret_cast<const float2*>(blk + Kv8<HD>::SOFF) : make_float2(1.f, 1.f);
            };
            const uint8_t *blk = block_of(0), *next = nullptr;
            float2 sc = scale_of(blk), next_sc = make_float2(1.f, 1.f);
            for (int i = 0; i < nt && ok; ++i) {
                if (i && (i & 3) == 0) {
                    blk = next;
                    sc = next_sc;
                }
                if ((i & 3) == 0) next = block_of(i / 4 + 1);
                if ((i & 3) == 2) next_sc = scale_of(next);
                const bool mine = lane >> 3 == (i & 3);
                const int n = min(8, page_end - (j0 + i) * 8);  // pages of the step that hold keys
                for (int is_v = 0; is_v < 2; ++is_v) {
                    if (use && !wait(r_empty + st, use - 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(r_full + st);
                    if (mine && blk)
                        bulk_copy(smem_u32(sm + Ct<HD>::OFF_R + st * RAW + (lane & 7) * KV8_PAGE * HD), blk + (is_v ? Kv8<HD>::VOFF : 0), KV8_PAGE * HD, bar);
                    // [i % 8]: at most 4 steps are in the ring and 2 in the operand buffers, and S of a step follows
                    // the softmax of the step before, so the softmax of step i - 8 has passed
                    if (!is_v && mine) {
                        const int ev = kv8_log2(sc.y);
                        scales[(i & 7) * 8 + (lane & 7)] = make_float4(sc.x, (float)ev, kv8_pow2(-ev), 0.f);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(bar, n * KV8_PAGE * HD);  // the stage's one arrival
                    __syncwarp();
                    ++issued;
                    if (++st == RING) {
                        st = 0;
                        ++use;
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            // the copies issued land before the CTA ends
            const uint64_t w0 = globaltimer_ns();
            for (int i = max(0, issued - RING); i < issued; ++i)
                while (!mbar_try_wait(smem_u32(r_full + i % RING), (i / RING) & 1) && globaltimer_ns() - w0 < kTcWaitNs) {
                }
        } else if (warp - 12 < n_rt) {
            // ---------------- MMA issuer of row tile t ----------------
            // The whole warp walks the loop and one elected lane issues, so addresses and descriptors are
            // the warp's. A step's keys go in two halves: while the softmax works on one, P V and the next
            // step's S of the other run. S overwrites the columns of its half's P and waits for that P V.
            const int t = warp - 12;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + t * 128;
            const uint64_t qd = sw128_desc(smem_u32(sm + t * MAT)), kd = sw128_desc(smem_u32(sm + Ct<HD>::OFF_K));
            const uint64_t vd = sw128_desc_mn(smem_u32(sm + Ct<HD>::OFF_V), CT_SUB);
            auto issue_s = [&](int i, int h) {
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t k0 = kd + (uint32_t)((i % NB) * (MAT >> 4) + h * (64 * 128 >> 4));
#pragma unroll
                    for (int sub = 0; sub < NSUB; ++sub)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16(tm + h * 64, qd + sub * (CT_SUB >> 4) + 2 * kk, k0 + sub * (CT_SUB >> 4) + 2 * kk, idesc_f16(128, 64),
                                     (sub | kk) ? 1u : 0u);
                    umma_commit(smem_u32(s_full + 2 * t + h));
                    if (h) umma_commit(smem_u32(k_empty + i % NB));
                }
                __syncwarp();
            };
            bool ok = wait(q_ready + t, 0) && wait(k_full, 0);
            if (ok) {
                issue_s(0, 0);
                issue_s(0, 1);
            }
            for (int i = 0; i < nt && ok; ++i) {
                for (int h = 0; h < 2 && ok; ++h) {
                    if ((!h && !wait(v_full + i % NB, i / NB)) || !wait(p_full + 2 * t + h, i)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t v0 = vd + (uint32_t)((i % NB) * (MAT >> 4) + h * (64 * 128 >> 4));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ts(tm + CT_O, tm + h * 64 + kk * 8, v0 + kk * (16 * 128 >> 4), idesc_f16(128, HD) | kIdescBMajorMN,
                                        (i | h | kk) ? 1u : 0u);
                        umma_commit(smem_u32(pv_done + t));
                        if (h) umma_commit(smem_u32(v_empty + i % NB));
                    }
                    __syncwarp();
                    if (i + 1 < nt) {
                        ok = wait(pv_done + t, 2 * i + h) && (h || wait(k_full + (i + 1) % NB, (i + 1) / NB));
                        if (ok) issue_s(i + 1, h);
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            // the commits' asynchronous arrivals land before the CTA ends
            if (elect_one()) umma_commit(smem_u32(mma_fin + t));
            __syncwarp();
            const uint64_t w0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(mma_fin + t), 0) && globaltimer_ns() - w0 < kTcWaitNs) {
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------- converters ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // Thread t takes the 16 codes at 16-byte position t % CH of key rows t / CH + i RP: RP is 16 or 32,
        // so its token within a page, and with it every swizzle, is the same for all i.
        const int t = threadIdx.x - 8 * 32, prow = t / CH, pos = t % CH, tk = prow & 15;
        // the two 16-byte chunks of 8 halves that a unit becomes; the second 64 dims start with their
        // odd chunk, so 8 lanes of a row meet 8 positions
        auto dest = [&](int ch, bool second) {
            const int c = 2 * (ch & 3) + (second != (HD == 128 && (ch & 4) != 0));
            return (uint32_t)((ch >> 2) * CT_SUB + prow * 128 + ((c ^ (prow & 7)) << 4));
        };
        const int kch = kv8_k_pos<HD>(tk, pos), vch = kv8_v_pos<HD>(tk, pos);  // the permutations are their own inverses
        const uint32_t kd0 = smem_u32(sm + Ct<HD>::OFF_K) + dest(kch, false), kd1 = smem_u32(sm + Ct<HD>::OFF_K) + dest(kch, true);
        const uint32_t vd0 = smem_u32(sm + Ct<HD>::OFF_V) + dest(vch, false), vd1 = smem_u32(sm + Ct<HD>::OFF_V) + dest(vch, true);
        const bool kodd = HD == 128 && (kch & 4), vodd = HD == 128 && (vch & 4);
        int st = 0, use = 0;
        // one tile: waits for its codes and for the operand buffer, converts, hands both on
        auto take = [&](int i, uint64_t* full, uint64_t* empty, uint32_t d0, uint32_t d1, bool odd) {
            const int buf = i % NB;
            d0 += buf * MAT;
            d1 += buf * MAT;
            if (!wait(r_full + st, use)) return false;
            const uint8_t* raw = sm + Ct<HD>::OFF_R + st * RAW + t * 16;
            const int left = kend - (j0 + i) * CT_BK - prow;  // > u RP: the row holds a key
            uint4 r[NU];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                r[u] = *reinterpret_cast<const uint4*>(raw + u * RP * HD);
                // rows past the keys are zeros: weight 0 must add exactly 0
                if (left <= u * RP) r[u] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (i >= NB && !wait(empty + buf, i / NB - 1)) return false;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const uint32_t a = odd ? r[u].z : r[u].x, a2 = odd ? r[u].w : r[u].y, c = odd ? r[u].x : r[u].z, c2 = odd ? r[u].y : r[u].w;
                sts128(d0 + u * RP * 128, kv8_dec2(a & 0xFFFFu), kv8_dec2(a >> 16), kv8_dec2(a2 & 0xFFFFu), kv8_dec2(a2 >> 16));
                sts128(d1 + u * RP * 128, kv8_dec2(c & 0xFFFFu), kv8_dec2(c >> 16), kv8_dec2(c2 & 0xFFFFu), kv8_dec2(c2 >> 16));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(full + buf));
                mbar_arrive(smem_u32(r_empty + st));
            }
            if (++st == RING) {
                st = 0;
                ++use;
            }
            return true;
        };
        bool ok = true;
        for (int i = 0; i < nt && ok; ++i) ok = take(i, k_full, k_empty, kd0, kd1, kodd) && take(i, v_full, v_empty, vd0, vd1, vodd);
        if (!ok) *abort_flag = 1;
    } else {
        // ---------------- softmax / output: thread = row = TMEM lane of row tile t ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int t = warp >> 2, wq = warp & 3, r = threadIdx.x & 127, rt0 = row0 + t * CT_ROWS, row = rt0 + r;
        if (t < n_rt) {
            const bool valid = row < rows;
            const int qt_ = valid ? row_token(p, row) : 0;
            const int tok = r0 + qt_, hq = head * p.G + (valid ? row - qt_ * p.G : 0);
            const int qpos = valid ? s + qt_ : -1;
            const uint32_t lane_base = tmem + t * 128 + ((uint32_t)(wq * 32) << 16), qa = smem_u32(sm + t * MAT);
            float* muls = reinterpret_cast<float*>(sm + Ct<HD>::OFF_MUL) + t * CT_ROWS;  // written and read by the same warp
            {
                QTile<HD> qt;
                fetch_q<HD>(qt, p, r0, head, rt0, rows, wq, lane);
                store_q<HD, DT>(qt, wq, lane, [&](int off, const uint4& v) { sts128(qa + off, v.x, v.y, v.z, v.w); },
                                [&](int rr, float mul) { muls[rr] = mul; });
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(q_ready + t));
            // With a page's scale (2^-32 at least) the factor stays above 0, or hidden scores of -infinity would give NaN.
            // Products of 2^33 at most over a row's scale make logits of this factor less than 2^-50.
            const float qmul = fmaxf(p.scale_log2 * muls[r], 0x1p-94f);
            float R = -1e30f, l = 0.f;
            bool good = true;
            const int first_masked = s + rt0 / p.G;  // steps that end at or before it need no mask
            for (int g = 0; g < 2 * nt; ++g) {  // half-steps of 64 keys
                const int i = g >> 1, h = g & 1, k0 = (j0 + i) * CT_BK + h * 64;
                if (!wait(s_full + 2 * t + h, i)) {
                    good = false;
                    break;
                }
                tc_fence_after();
                const float4* scl = scales + (i & 7) * 8 + h * 4;
                uint32_t x[64];  // the row's scores stay in registers
                TMEM_LD32(lane_base + h * 64, x);
                TMEM_LD32(lane_base + h * 64 + 32, (x + 32));
                tmem_wait_ld();
                if (k0 + 63 > first_masked) {
#pragma unroll
                    for (int u = 0; u < 64; ++u)
                        if (k0 + u > qpos) x[u] = 0xFF800000u;
                }
                float mt = -INFINITY;
#pragma unroll
                for (int pg = 0; pg < 4; ++pg) {
                    const uint32_t* y = x + 16 * pg;  // three-way maxima
                    const float m0 = max3(max3(fl(y[0]), fl(y[1]), fl(y[2])), fl(y[3]), fl(y[4]));
                    const float m1 = max3(max3(fl(y[5]), fl(y[6]), fl(y[7])), fl(y[8]), fl(y[9]));
                    const float m2 = max3(max3(fl(y[10]), fl(y[11]), fl(y[12])), fl(y[13]), fl(y[14]));
                    const float4 sc = scl[pg];
                    mt = fmaxf(mt, fmaf(max3(max3(m0, m1, m2), fl(y[15]), m0), qmul * sc.x, sc.y));
                }
                const bool move = mt > R + KV8_SLACK;
                if (__any_sync(0xffffffffu, move)) {
                    const float al = move ? ex2(R - mt) : 1.f;
                    if (move) R = mt;
                    l *= al;
                    if (g > 0) {
                        if (!wait(pv_done + t, g - 1)) {  // the half-step before may still be adding to O
                            good = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < HD / 16; ++cc) {
                            uint32_t y[16];
                            TMEM_LD16(lane_base + CT_O + cc * 16, y);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; ++u) y[u] = __float_as_uint(__uint_as_float(y[u]) * al);
                            TMEM_ST16(lane_base + CT_O + cc * 16, y);
                        }
                    }
                }
                uint32_t w[32];
#pragma unroll
                for (int pg = 0; pg < 4; ++pg) {
                    const float4 sc = scl[pg];
                    const uint64_t f = pack2(qmul * sc.x, qmul * sc.x);
                    const float a0 = sc.y - R + KV8_LIFT;
                    const uint64_t a = pack2(a0, a0);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int at = 16 * pg + 2 * u;
                        float t0, t1;
                        unpack2(fma2(pack2u(x[at], x[at + 1]), f, a), t0, t1);
                        const float e0 = ex2(t0), e1 = ex2(t1);
                        sum[u & 1] = add2(sum[u & 1], pack2(e0, e1));
                        w[pg * 8 + u] = pack_h2(e0, e1);
                    }
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    l = fmaf(s0 + s1, sc.z, l);
                }
                TMEM_ST32(lane_base + h * 64, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + 2 * t + h));
            }
            // both halves of the last step: a wait tells a phase only from the one before it
            if (good && wait(pv_done + t, 2 * nt - 2) && wait(pv_done + t, 2 * nt - 1)) {
                tc_fence_after();
                const float inv = P.splits == 1 ? 1.f / l : 1.f;
                // With the whole row at hand the output goes through the warp's rows of the Q operand (no MMA
                // reads it any more), so that stores cover whole rows; partials are the thread's own.
#pragma unroll 1
                for (int cc = 0; cc < HD / 32; ++cc) {
                    uint32_t x[32];
                    TMEM_LD32(lane_base + CT_O + cc * 32, x);
                    tmem_wait_ld();
                    if (P.splits == 1) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float e0 = fl(x[8 * u + 2 * k]) * inv, e1 = fl(x[8 * u + 2 * k + 1]) * inv;
                                w[k] = pack_out<DT>(e0, e1);
                            }
                            const int ch = cc * 4 + u;
                            sts128(qa + (ch >> 3) * CT_SUB + r * 128 + (((ch & 7) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                    } else if (valid) {
                        float* dst = P.part_o + part(t) * CT_ROWS * HD + (cc * 8 * CT_ROWS + r) * 4;
#pragma unroll
                        for (int u = 0; u < 32; u += 4)
                            *reinterpret_cast<uint4*>(dst + u * CT_ROWS) = make_uint4(x[u], x[u + 1], x[u + 2], x[u + 3]);
                    }
                    __syncwarp();
                }
                if (P.splits == 1) {
                    constexpr int LPR = HD / 8;
                    const int ch = lane % LPR;
#pragma unroll
                    for (int k0 = 0; k0 < LPR; k0 += 8) {  // eight rows' chunks at a time
                        uint4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int rr = wq * 32 + (k0 + k) * (32 / LPR) + lane / LPR;
                            v[k] = *reinterpret_cast<const uint4*>(sm + t * MAT + (ch >> 3) * CT_SUB + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int rr = wq * 32 + (k0 + k) * (32 / LPR) + lane / LPR, tk = row_token(p, rt0 + rr);
                            if (rt0 + rr < rows)
                                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)(r0 + tk) * p.ld_out +
                                                          (size_t)(head * p.G + rt0 + rr - tk * p.G) * HD + ch * 8) = v[k];
                        }
                    }
                }
                if (valid && P.splits == 1) {
                    const float z = log2f(l) + R - KV8_LIFT;
                    if (p.lse2) p.lse2[(size_t)tok * p.n_heads + hq] = z;
                    if (p.lse) p.lse[(size_t)tok * p.n_heads + hq] = z * KV8_LN2;
                } else if (valid) {
                    P.part_ml[(part(t) * CT_ROWS + r) * 2] = R;
                    P.part_ml[(part(t) * CT_ROWS + r) * 2 + 1] = l;
                }
            } else {
                *abort_flag = 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) atomicOr(p.status, QW_KV8_TIMEOUT);
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(CT_TMEM) : "memory");
    }
}

// Adds a row tile's partials over the splits, in order. A thread takes 4 dims of a row; neighbours are
// rows, as the partials lie.
template <int HD>
constexpr int kCombineRows = 256 / (HD / 4);

template <int HD, int DT>
__global__ void __launch_bounds__(256) k_kv8_chunk_combine(const __grid_constant__ Kv8ChunkP P) {
    const Kv8AttnP& p = P.a;
    constexpr int NR = kCombineRows<HD>;
    const int b = blockIdx.z, head = blockIdx.y, row = blockIdx.x * NR + threadIdx.x % NR, d4 = threadIdx.x / NR;
    pdl_wait();
    pdl_launch();
    int s, r0, n;
    if (!attn_entry(p, b, s, r0, n) || row >= n * p.G) return;
    const size_t part = (((size_t)b * p.kv.n_kv + head) * P.tiles + row / CT_ROWS) * P.splits;
    float M = -1e30f, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < P.splits; ++k) {
        const float2 ml = *reinterpret_cast<const float2*>(P.part_ml + ((part + k) * CT_ROWS + row % CT_ROWS) * 2);
        float4 v = *reinterpret_cast<const float4*>(P.part_o + (part + k) * CT_ROWS * HD + ((size_t)d4 * CT_ROWS + row % CT_ROWS) * 4);
        if (ml.y == 0.f) continue;  // that split has no partial
        const float m = fmaxf(M, ml.x), fo = ex2(M - m), fn = ex2(ml.x - m);
        M = m;
        L = L * fo + ml.y * fn;
        acc.x = acc.x * fo + v.x * fn;
        acc.y = acc.y * fo + v.y * fn;
        acc.z = acc.z * fo + v.z * fn;
        acc.w = acc.w * fo + v.w * fn;
    }
    const float inv = 1.f / L;
    const int tok = r0 + row_token(p, row), h = head * p.G + row - row_token(p, row) * p.G;
    uint2 w;
    w.x = pack_out<DT>(acc.x * inv, acc.y * inv);
    w.y = pack_out<DT>(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)tok * p.ld_out + (size_t)h * HD + d4 * 4) = w;
    if (d4 == 0) {
        const float z = log2f(L) + M - KV8_LIFT;
        if (p.lse2) p.lse2[(size_t)tok * p.n_heads + h] = z;
        if (p.lse) p.lse[(size_t)tok * p.n_heads + h] = z * KV8_LN2;
    }
}

// =======================================================================================
// k_kv8_score: score_out[j] = score_in[j] + sum over the query rows of 2^(t_j - lse2), on tcgen05.
//
// The normalisers are known, so the weights need only S again, and the sum over rows is a thread's
// own if the keys are the rows of the MMA: a CTA keeps 128 keys of one (entry, head) as the A operand
// and walks the query rows in tiles of 128 (B). S^T = K Q^T lands in TMEM (two buffers); eight
// warps, thread = key and half of the rows, add the exponentials in order, so equal inputs give
// equal bits. 2 HD MACs and one exponential a (row, key) pair, and the exponentials bound it: every
// key tile needs every query tile, so k_kv8_score_prep lays these out once as swizzled operands with
// their rows' constants, and a tile costs two bulk copies (converting them here, in every CTA, took
// 29 us of 127 and the warps that the sums wanted). Two CTAs share an SM. 2 chunks of 500 tokens x 28
// heads over 6k-9k keys (head_dim 64, 212 M pairs): 88 us and 6 to lay out, 310 TFLOP/s and 2.4 T
// exponentials/s; at 32 a clock and SM these alone would take 23 us, the sums' other instructions and
// TMEM reads share the warps with them.
// =======================================================================================
constexpr int CS_THREADS = 288;  // warps 0-7 sums, 8 copies and MMAs
constexpr int CS_TMEM = 256;
template <int HD>
struct Cs {
    static constexpr int KEYS = 128;
    static constexpr int MAT = CT_SUB * (HD / 64), ROWC = 3 * CT_ROWS * 4;  // operand; -lse2, logit factor, last visible position
    static constexpr int PREP = MAT + ROWC;                                  // a prepared tile
    static constexpr int RING = HD == 128 ? 2 : 4;
    static constexpr int OFF_Q = MAT, OFF_ROW = OFF_Q + RING * MAT, OFF_ACC = OFF_ROW + 2 * RING * ROWC;
    static constexpr int OFF_BAR = OFF_ACC + KEYS * 4, SMEM = 1024 + OFF_BAR + 256;
};

// Prepared tiles lie [n_kv][T G / 128 + B]: entry b's begin at its first row / 128 + b, which leaves
// room for every tile of the entries before it, whatever the bounds on one entry are.
__host__ __device__ inline size_t prep_tiles(int B, int T, int G) { return (size_t)((long long)T * G / CT_ROWS) + B; }
__device__ __forceinline__ size_t prep_at(const Kv8AttnP& p, int B, int b, int head, int r0) {
    return head * prep_tiles(B, p.T, p.G) + (size_t)((long long)r0 * p.G / CT_ROWS) + b;
}

// One query tile of one (entry, head).
template <int HD, int DT>
__global__ void __launch_bounds__(128) k_kv8_score_prep(const __grid_constant__ Kv8AttnP p, uint8_t* prep) {
    pdl_wait();
    pdl_launch();
    const int t = threadIdx.x, b = blockIdx.z, head = blockIdx.y, tile = blockIdx.x;
    int s, r0, n;
    if (!attn_entry(p, b, s, r0, n) || tile * CT_ROWS >= n * p.G) return;
    const int rows = n * p.G, row = tile * CT_ROWS + t, tok = min(row_token(p, row), n - 1);
    uint8_t* at = prep + (prep_at(p, gridDim.z, b, head, r0) + tile) * Cs<HD>::PREP;
    float* rc = reinterpret_cast<float*>(at + Cs<HD>::MAT);
    QTile<HD> qt;
    fetch_q<HD>(qt, p, r0, head, tile * CT_ROWS, rows, t >> 5, t & 31);
    const float z = row < rows ? p.lse2[(size_t)(r0 + tok) * p.n_heads + head * p.G + row - tok * p.G] : 0.f;
    store_q<HD, DT>(qt, t >> 5, t & 31, [&](int off, const uint4& v) { *reinterpret_cast<uint4*>(at + off) = v; },
                    [&](int r, float mul) { rc[CT_ROWS + r] = mul * p.scale_log2; });
    rc[t] = -z;
    rc[2 * CT_ROWS + t] = __int_as_float(row < rows ? s + tok : -1);
}

template <int HD, int DT>
__global__ void __launch_bounds__(CS_THREADS, 2) k_kv8_score(const __grid_constant__ Kv8AttnP p, const uint8_t* prep) {
    constexpr int MAT = Cs<HD>::MAT, NSUB = HD / 64, CH = HD / 16, RING = Cs<HD>::RING, ROWC = Cs<HD>::ROWC;
    extern __shared__ uint8_t cs_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(cs_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cs<HD>::OFF_BAR);
    uint64_t *q_full = bars, *q_empty = bars + 4, *s_full = bars + 8, *s_empty = bars + 10, *mma_fin = bars + 12;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 13);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, head = blockIdx.y, key0 = blockIdx.x * Cs<HD>::KEYS;
    pdl_wait();
    pdl_launch();
    int s, r0, n;
    if (!attn_entry(p, b, s, r0, n) || n == 0 || key0 >= s + n || kv8_stopped(p.kv, b)) return;
    const int rows = n * p.G, kend = s + n;
    const int t0 = max(0, key0 - s) * p.G / CT_ROWS, t1 = (rows + CT_ROWS - 1) / CT_ROWS, nt = t1 - t0;  // row tiles that see a key of these
    auto wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xffffffffu, ct_wait(smem_u32(bar), (uint32_t)parity & 1u, abort_flag));
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(smem_u32(q_full + i), 1);
            mbar_init(smem_u32(q_empty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(s_full + i), 1);
            mbar_init(smem_u32(s_empty + i), 8);
        }
        mbar_init(smem_u32(mma_fin), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(CS_TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const int* table = kv8_row(p.kv, p.kv.table, b);
    auto block_of = [&](int pi) -> const uint8_t* {
        int id = table[pi];
        if (id < 0 || id >= p.kv.n_pages) {
            atomicOr(p.status, QW_KV8_BAD_POS);
            id = 0;
        }
        return kv8_block(p.kv, b, id, head, Kv8<HD>::BLK);
    };
    if (warp < 8) {  // the keys: thread = half a row
        const int row = threadIdx.x >> 1, tk = row & 15;
        const bool on = key0 + row < kend;
        const uint8_t* src = on ? block_of(key0 / KV8_PAGE + (row >> 4)) + tk * HD : nullptr;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
            const int pos = (threadIdx.x & 1) * (CH / 2) + i, ch = kv8_k_pos<HD>(tk, pos);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (on) v = *reinterpret_cast<const uint4*>(src + pos * 16);
            const uint32_t at = smem_u32(sm) + (ch >> 2) * CT_SUB + row * 128;
            const int c0 = 2 * (ch & 3);
            sts128(at + ((c0 ^ (row & 7)) << 4), kv8_dec2(v.x & 0xFFFFu), kv8_dec2(v.x >> 16), kv8_dec2(v.y & 0xFFFFu), kv8_dec2(v.y >> 16));
            sts128(at + (((c0 + 1) ^ (row & 7)) << 4), kv8_dec2(v.z & 0xFFFFu), kv8_dec2(v.z >> 16), kv8_dec2(v.w & 0xFFFFu), kv8_dec2(v.w >> 16));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    float acc = 0.f;
    bool good = true;
    const int key = key0 + (warp & 3) * 32 + lane;
    const bool on = warp < 8 && key < kend;
    if (warp == 8) {
        // ---------------- copies and MMAs ----------------
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t kd = sw128_desc(smem_u32(sm)), qd = sw128_desc(smem_u32(sm + Cs<HD>::OFF_Q));
        const uint8_t* src = prep + (prep_at(p, gridDim.z, b, head, r0) + t0) * Cs<HD>::PREP;
        int issued = 0;
        auto copy = [&](int i) {
            const int st = i % RING;
            if (elect_one()) {
                const uint32_t bar = smem_u32(q_full + st);
                mbar_expect_tx(bar, Cs<HD>::PREP);
                bulk_copy(smem_u32(sm + Cs<HD>::OFF_Q + st * MAT), src + (size_t)i * Cs<HD>::PREP, MAT, bar);
                // two rings deep: copy i follows the MMA of tile i - RING + 1, which waited for the sums of i - RING - 1
                bulk_copy(smem_u32(sm + Cs<HD>::OFF_ROW + (i % (2 * RING)) * ROWC), src + (size_t)i * Cs<HD>::PREP + MAT, ROWC, bar);
            }
            __syncwarp();
            issued = i + 1;
        };
        for (int i = 0; i < min(RING - 1, nt); ++i) copy(i);
        for (int i = 0; i < nt; ++i) {
            const int st = i % RING, buf = i & 1;
            if (!wait(q_full + st, i / RING) || (i >= 2 && !wait(s_empty + buf, (i >> 1) - 1))) {
                good = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t q0 = qd + (uint32_t)(st * (MAT >> 4));
#pragma unroll
                for (int sub = 0; sub < NSUB; ++sub)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16(tm + buf * 128, kd + sub * (CT_SUB >> 4) + 2 * kk, q0 + sub * (CT_SUB >> 4) + 2 * kk,
                                 idesc_f16(128, CT_ROWS), (sub | kk) ? 1u : 0u);
                umma_commit(smem_u32(s_full + buf));
                umma_commit(smem_u32(q_empty + st));
            }
            __syncwarp();
            const int c = i + RING - 1;  // into the stage of tile i - 1
            if (c < nt) {
                if (i >= 1 && !wait(q_empty + c % RING, (i - 1) / RING)) {
                    good = false;
                    break;
                }
                copy(c);
            }
        }
        if (!good) *abort_flag = 1;
        // the copies and the commits' asynchronous arrivals land before the CTA ends
        if (elect_one()) umma_commit(smem_u32(mma_fin));
        __syncwarp();
        const uint64_t w0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(mma_fin), 0) && globaltimer_ns() - w0 < kTcWaitNs) {
        }
        for (int i = max(0, issued - RING); i < issued; ++i)
            while (!mbar_try_wait(smem_u32(q_full + i % RING), (i / RING) & 1) && globaltimer_ns() - w0 < kTcWaitNs) {
            }
        __syncwarp();
    } else {
        // ---------------- sums: thread = key = TMEM lane, warps 4-7 the second 64 rows of a tile ----------------
        const int half = warp >> 2;
        const float sk = on ? *reinterpret_cast<const float*>(block_of(key / KV8_PAGE) + Kv8<HD>::SOFF) : 1.f;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 64;
        const float f16 = p.scale_log2 * sk;
        const uint64_t f2 = pack2(f16, f16), k2 = pack2(sk, sk);
        for (int i = 0; i < nt; ++i) {
            const int buf = i & 1, rt = t0 + i;
            if (!wait(s_full + buf, i >> 1)) {
                good = false;
                break;
            }
            tc_fence_after();
            const float* rc = reinterpret_cast<const float*>(sm + Cs<HD>::OFF_ROW + (i % (2 * RING)) * ROWC) + half * 64;
            // rows of the tile before the last key's token see not all of these keys
            const bool masked = s + rt * CT_ROWS / p.G < key0 + Cs<HD>::KEYS - 1 || (rt + 1) * CT_ROWS > rows;
            uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
            auto tile = [&](auto with_mask) {  // with the test in the loop 5 us more
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    uint32_t y[32];
                    TMEM_LD32(lane_base + buf * 128 + cc * 32, y);
                    tmem_wait_ld();
                    // four rows a turn: their constants are one or two 16-byte broadcasts
#pragma unroll
                    for (int u = 0; u < 32; u += 4) {
                        const float4 z = *reinterpret_cast<const float4*>(rc + cc * 32 + u);
                        uint64_t fa = f2, fb = f2;
                        if (DT == QW_BF16) {
                            const float4 f = *reinterpret_cast<const float4*>(rc + CT_ROWS + cc * 32 + u);
                            fa = mul2(pack2(f.x, f.y), k2);
                            fb = mul2(pack2(f.z, f.w), k2);
                        }
                        float e0, e1, e2, e3;
                        unpack2(fma2(pack2u(y[u], y[u + 1]), fa, pack2(z.x, z.y)), e0, e1);
                        unpack2(fma2(pack2u(y[u + 2], y[u + 3]), fb, pack2(z.z, z.w)), e2, e3);
                        if (decltype(with_mask)::value) {
                            const int4 lim = *reinterpret_cast<const int4*>(rc + 2 * CT_ROWS + cc * 32 + u);
                            e0 = key <= lim.x ? e0 : -INFINITY;
                            e1 = key <= lim.y ? e1 : -INFINITY;
                            e2 = key <= lim.z ? e2 : -INFINITY;
                            e3 = key <= lim.w ? e3 : -INFINITY;
                        }
                        sum[(u >> 1) & 3] = add2(sum[(u >> 1) & 3], pack2(ex2(e0), ex2(e1)));
                        sum[((u >> 1) + 1) & 3] = add2(sum[((u >> 1) + 1) & 3], pack2(ex2(e2), ex2(e3)));
                    }
                }
            };
            if (masked) tile(std::true_type());
            else tile(std::false_type());
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(s_empty + buf));
            float e0, e1;
            unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), e0, e1);
            acc += e0 + e1;
        }
        if (!good) *abort_flag = 1;
        if (half) reinterpret_cast<float*>(sm + Cs<HD>::OFF_ACC)[key - key0] = acc;
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) atomicOr(p.status, QW_KV8_TIMEOUT);
    if (warp < 4 && on && !*abort_flag) {
        const size_t at = score_row(p, b, head) + key;
        p.score_out[at] = (p.score_in ? p.score_in[at] : 0.f) + (acc + reinterpret_cast<const float*>(sm + Cs<HD>::OFF_ACC)[key - key0]);
    }
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(CS_TMEM) : "memory");
    }
}

// ---- which kernels a call runs, and its workspace ---------------------------------------

constexpr int KD_SMEM = 200 * 1024, KD_SMEM2 = 106 * 1024;  // k_kv8_decode's, with one and two CTAs an SM

struct Plan {
    bool decode;       // k_kv8_decode (max_len * G <= 16 rows)
    bool pair_mode;
    bool tbuf;         // scores from stored logits
    int nrow, stages, n_cta, smem;  // decode
    int tiles, splits;              // k_kv8_chunk
    size_t off_o, off_ml, off_t, off_prep, bytes;
};

// `avail`: most bytes that a decode's stored logits may take.
Plan make_plan(int n_kv, int HD, int B, int T, int max_len, int max_keys, int n_heads, bool score, size_t avail) {
    Plan q = {};
    const int G = n_heads / n_kv, BLK = 32 * HD + 32;
    auto put = [&](size_t n) {
        const size_t at = q.bytes;
        q.bytes = (at + n + 255) & ~(size_t)255;
        return at;
    };
    put(score ? (size_t)T * n_heads * 4 : 0);  // lse2
    const long long rows = (long long)std::min(max_len, std::max(T, 1)) * G;
    // to 16 rows k_kv8_decode: 16 rows over 30k tokens of one sequence 23 us (k_kv8_chunk 31), over 64 x 1000
    // tokens of 8 heads 55 (83), of 2 heads 26 (22); at 8 rows over 64 x 1000 tokens of 8 heads 40 (82)
    q.decode = rows <= 16;
    if (q.decode) {
        q.nrow = (int)rows;
        const int slots = 2 * KD_WARPS * q.nrow * (HD + 2) * 4, ent = B * 8;
        // two CTAs an SM where their rings and slots fit (rows <= 4 at head_dim 128), else one: 64 x 1100 tokens
        // of 2 rows take 33 us with two and 38 with one
        const int per_sm = KD_WARPS * 2 * BLK + slots + ent <= KD_SMEM2 && rows <= 8 ? 2 : 1;
        q.stages = std::min(8, ((per_sm == 2 ? KD_SMEM2 : KD_SMEM) - slots - ent) / (KD_WARPS * BLK));
        q.smem = KD_WARPS * q.stages * BLK + slots + ent;
        // 8 x 400 tokens 7.9 us, in runs 10.2; 64 x 400 20.0 and 19.8; 64 x 1100 33.7 and 33.3
        q.pair_mode = max_keys <= 512;
        q.n_cta = q.pair_mode ? B * n_kv : per_sm * kv8_sm_count();
        // a row's logits are written and read once (8 bytes a key) instead of its K (HD bytes): 8 x 4k tokens of
        // 4 rows 27 us, with k_kv8_score 67
        const size_t logits = (size_t)B * n_kv * q.nrow * (((size_t)max_keys + 3) & ~(size_t)3) * 4;
        // k_kv8_combine's launch has at most 65535 blocks of KC_KEYS keys
        q.tbuf = score && rows <= 8 && logits <= avail && max_keys <= 65535 * KC_KEYS;
        q.off_o = put(q.pair_mode ? 0 : (size_t)q.n_cta * 2 * q.nrow * HD * 4);
        q.off_ml = put(q.pair_mode ? 0 : (size_t)q.n_cta * 2 * q.nrow * 2 * 4);
        q.off_t = put(q.tbuf ? logits : 0);
    }
    if (!q.decode) {
        q.tiles = (int)((rows + CT_ROWS - 1) / CT_ROWS);
        // A CTA an SM. Row tiles that leave the last wave of CTAs part empty split their keys, if that
        // fills waves by a quarter better and each split keeps 512 keys: 2 chunks of 400 tokens (4 KV heads
        // of 4, 5k-9k keys, 56 CTAs) 79 us, unsplit 150.
        const long long ctas = (long long)(q.tiles + 1) / 2 * n_kv * B, slots = kv8_sm_count();
        auto fill = [&](long long n) { return (double)n / (double)((n + slots - 1) / slots * slots); };
        q.splits = 1;
        const int most = std::min(64, max_keys / 512);
        for (int n = 2; n <= most && ctas * n < 4 * slots; ++n)
            if (fill(ctas * n) >= 1.25 * fill(ctas * q.splits)) q.splits = n;
        const size_t part = q.splits == 1 ? 0 : (size_t)B * n_kv * q.tiles * q.splits * CT_ROWS;
        q.off_o = put(part * HD * 4);
        q.off_ml = put(part * 2 * 4);
    }
    if (score && !q.tbuf)
        q.off_prep = put(kv8_prep_bytes(n_kv, HD, B, T, G));
    q.bytes = std::max(q.bytes, (size_t)256);
    return q;
}

// The most that any call gives the kernel, so that calls in several host threads agree.
template <typename K>
cudaError_t allow_smem(K kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int HD, int DT>
cudaError_t run_score(const Kv8AttnP& p, int B, uint8_t* prep, cudaStream_t st, int* launches) {
    LaunchCtx c = {st, true, launches};
    if (cudaError_t e = allow_smem(k_kv8_score<HD, DT>, Cs<HD>::SMEM)) return e;
    const unsigned rows = (unsigned)(((long long)std::min(p.max_len, p.T) * p.G + CT_ROWS - 1) / CT_ROWS);
    cudaError_t e = launch_k(c, k_kv8_score_prep<HD, DT>, dim3(rows, p.kv.n_kv, B), dim3(128), 0, p, prep);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)((p.max_keys + Cs<HD>::KEYS - 1) / Cs<HD>::KEYS);
    return launch_k(c, k_kv8_score<HD, DT>, dim3(tiles, p.kv.n_kv, B), dim3(CS_THREADS), (size_t)Cs<HD>::SMEM, p, (const uint8_t*)prep);
}

template <int HD, int DT>
cudaError_t run_attn(const Kv8AttnP& p, const Plan& q, int B, char* ws, cudaStream_t st, int* launches) {
    LaunchCtx c = {st, true, launches};
    cudaError_t e;
    if (q.decode) {
        Kv8DecP P = {};
        P.a = p;
        P.B = B;
        P.nrow = q.nrow;
        P.stages = q.stages;
        P.pair_mode = q.pair_mode;
        P.part_o = (float*)(ws + q.off_o);
        P.part_ml = (float*)(ws + q.off_ml);
        P.tbuf = q.tbuf ? (float*)(ws + q.off_t) : nullptr;
        P.ld_t = ((size_t)p.max_keys + 3) & ~(size_t)3;
        P.n_cta = q.n_cta;
        auto kern = q.nrow <= 8 ? k_kv8_decode<HD, DT, 1> : k_kv8_decode<HD, DT, 2>;
        if ((e = allow_smem(kern, KD_SMEM)) != cudaSuccess) return e;
        if ((e = launch_k(c, kern, dim3(q.n_cta), dim3(KD_WARPS * 32), (size_t)q.smem, P)) != cudaSuccess) return e;
        if (!q.tbuf) P.a.score_out = nullptr;
        if (!q.pair_mode || q.tbuf) {
            const unsigned chunks = q.tbuf ? (unsigned)((p.max_keys + KC_KEYS - 1) / KC_KEYS)
                                           : (unsigned)std::max(1, std::min(q.nrow, 2 * kv8_sm_count() / (B * p.kv.n_kv)));
            const int smem = q.pair_mode ? 0 : kc_smem(q.nrow, HD);
            if ((e = allow_smem(k_kv8_combine<HD, DT>, kc_smem(16, HD))) != cudaSuccess) return e;
            e = launch_k(c, k_kv8_combine<HD, DT>, dim3(B * p.kv.n_kv, chunks), dim3(KD_WARPS * 32), (size_t)smem, P);
            if (e != cudaSuccess) return e;
        }
        return p.score_out && !q.tbuf ? run_score<HD, DT>(p, B, (uint8_t*)ws + q.off_prep, st, launches) : cudaSuccess;
    }
    Kv8ChunkP P = {};
    P.a = p;
    P.splits = q.splits;
    P.part_o = (float*)(ws + q.off_o);
    P.part_ml = (float*)(ws + q.off_ml);
    P.tiles = q.tiles;
    // the roles' register counts add up only if the kernel was given exactly CT_REGS a thread
    static const int regs = [] {
        cudaFuncAttributes fa = {};
        return cudaFuncGetAttributes(&fa, k_kv8_chunk<HD, DT>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs != CT_REGS) return cudaErrorInvalidKernelImage;
    if ((e = allow_smem(k_kv8_chunk<HD, DT>, Ct<HD>::SMEM)) != cudaSuccess) return e;
    e = launch_k(c, k_kv8_chunk<HD, DT>, dim3(p.kv.n_kv, B, (q.tiles + 1) / 2 * q.splits), dim3(CT_THREADS), (size_t)Ct<HD>::SMEM, P);
    if (e == cudaSuccess && q.splits > 1)
        e = launch_k(c, k_kv8_chunk_combine<HD, DT>, dim3(q.tiles * CT_ROWS / kCombineRows<HD>, p.kv.n_kv, B), dim3(256), 0, P);
    return e == cudaSuccess && p.score_out ? run_score<HD, DT>(p, B, (uint8_t*)ws + q.off_prep, st, launches) : e;
}

}  // namespace

int kv8_sm_count() {
    static const int n = [] {
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) v = 0;
        return v > 0 ? v : 152;
    }();
    return n;
}

size_t kv8_prep_bytes(int n_kv, int head_dim, int B, int T, int G) {
    return n_kv * prep_tiles(B, T, G) * (size_t)(head_dim == 128 ? Cs<128>::PREP : Cs<64>::PREP);
}

static qw_status attn_sizes(const qw_kv8* kv, int B, int T, int max_len, int max_keys, int n_heads) {
    if (qw_status s = kv8_check(kv, B, "attn")) return s;
    if (T < 0 || max_len < 1 || max_len > (1 << 26)) return qw_fail(QW_ERR_INVALID_ARG, "attn: T or max_len out of range");
    if (max_keys < 1 || (long long)max_keys > (long long)kv->max_pages * 16)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: max_keys outside [1, 16 max_pages]");
    if (n_heads < kv->n_kv_heads || n_heads % kv->n_kv_heads)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: n_heads is not a multiple of n_kv_heads");
    if ((long long)B * ((max_keys + 15) / 16) * kv->n_kv_heads > 0x7fffffffll)
        return qw_fail(QW_ERR_UNSUPPORTED, "attn: B * max_keys * n_kv_heads too large");
    // a launch has at most 65535 pairs of row tiles
    if ((long long)std::min(max_len, T) * (n_heads / kv->n_kv_heads) > 65535ll * 2 * CT_ROWS)
        return qw_fail(QW_ERR_UNSUPPORTED, "attn: more than 65535 * 256 query rows of one KV head and entry");
    if (n_heads / kv->n_kv_heads > 16) return qw_fail(QW_ERR_UNSUPPORTED, "attn: more than 16 query heads per KV head");
    return QW_OK;
}

qw_status kv8_attn(const Kv8View& v, int head_dim, const qw_kv8_attn_args& a, int score_mul, int score_add, cudaStream_t st,
                   int* launches) {
    // a caller's workspace always has room for the logits; a model's may not
    Plan q = make_plan(v.n_kv, head_dim, a.B, a.T, a.max_len, a.max_keys, a.n_heads, a.dev_score_out != nullptr, SIZE_MAX);
    if (q.bytes > a.ws_bytes)
        q = make_plan(v.n_kv, head_dim, a.B, a.T, a.max_len, a.max_keys, a.n_heads, a.dev_score_out != nullptr, 0);
    if (q.bytes > a.ws_bytes) return qw_fail(QW_ERR_INVALID_ARG, "attn: workspace too small");
    Kv8AttnP p = {};
    p.kv = v;
    p.start = a.dev_start;
    p.cu = a.dev_cu;
    p.q = a.dev_q;
    p.ld_q = a.ld_q;
    p.T = a.T;
    p.max_len = a.max_len;
    p.max_keys = a.max_keys;
    p.n_heads = a.n_heads;
    p.G = a.n_heads / v.n_kv;
    p.gmul = p.G == 1 ? 0u : (uint32_t)(((1ull << 32) + p.G - 1) / p.G);
    p.scale_log2 = a.scale * KV8_LOG2E;
    p.out = a.dev_out;
    p.ld_out = a.ld_out;
    p.lse = a.dev_lse;
    p.lse2 = a.dev_score_out ? (float*)a.dev_ws : nullptr;
    p.score_in = a.dev_score_in;
    p.score_out = a.dev_score_out;
    p.ld_score = a.ld_score;
    p.score_mul = score_mul;
    p.score_add = score_add;
    p.status = a.dev_status;
    char* ws = (char*)a.dev_ws;
    const bool h = a.dtype == QW_F16;
    const cudaError_t e = head_dim == 128
                              ? (h ? run_attn<128, QW_F16>(p, q, a.B, ws, st, launches) : run_attn<128, QW_BF16>(p, q, a.B, ws, st, launches))
                              : (h ? run_attn<64, QW_F16>(p, q, a.B, ws, st, launches) : run_attn<64, QW_BF16>(p, q, a.B, ws, st, launches));
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "attn: %s", cudaGetErrorString(e));
}

extern "C" size_t qw_kv8_attn_ws_bytes(const qw_kv8* kv, int B, int T, int max_len, int max_keys, int n_heads,
                                       int with_score) {
    if (attn_sizes(kv, B, T, max_len, max_keys, n_heads)) return 0;
    return make_plan(kv->n_kv_heads, kv->head_dim, B, T, max_len, max_keys, n_heads, with_score != 0, SIZE_MAX).bytes;
}

extern "C" qw_status qw_kv8_attn(const qw_kv8* kv, const qw_kv8_attn_args* a, void* stream) {
    if (!a) return qw_fail(QW_ERR_INVALID_ARG, "attn: args is NULL");
    if (qw_status s = attn_sizes(kv, a->B, a->T, a->max_len, a->max_keys, a->n_heads)) return s;
    if (!a->dev_start || !a->dev_cu || !a->dev_ws || !a->dev_status || (a->T > 0 && (!a->dev_q || !a->dev_out)))
        return qw_fail(QW_ERR_INVALID_ARG, "attn: NULL argument");
    if (a->dtype != QW_F16 && a->dtype != QW_BF16)
        return qw_fail(QW_ERR_INVALID_ARG, "attn: dtype %d (QW_F16 and QW_BF16 are taken)", a->dtype);
    const size_t row = (size_t)a->n_heads * kv->head_dim;
    if (a->T > 0 && (a->ld_q < row || a->ld_out < row)) return qw_fail(QW_ERR_INVALID_ARG, "attn: row stride below n_heads * head_dim");
    if (a->T > 0 && (((uintptr_t)a->dev_q | (uintptr_t)a->dev_out) & 15 || a->ld_q % 8 || a->ld_out % 8))
        return qw_fail(QW_ERR_INVALID_ARG, "attn: rows not 16-byte aligned");
    if (!(a->scale > 0.f) || !(a->scale < 1e30f)) return qw_fail(QW_ERR_INVALID_ARG, "attn: scale not positive and finite");
    if (a->dev_score_in && !a->dev_score_out) return qw_fail(QW_ERR_INVALID_ARG, "attn: score_in without score_out");
    if (a->dev_score_out && a->ld_score < (size_t)a->max_keys) return qw_fail(QW_ERR_INVALID_ARG, "attn: ld_score < max_keys");
    if ((uintptr_t)a->dev_ws & 255 ||
        a->ws_bytes < qw_kv8_attn_ws_bytes(kv, a->B, a->T, a->max_len, a->max_keys, a->n_heads, a->dev_score_out != nullptr))
        return qw_fail(QW_ERR_INVALID_ARG, "attn: workspace too small or not 256-byte aligned");
    if (a->T == 0) return QW_OK;
    return kv8_attn(kv8_view(kv), kv->head_dim, *a, 1, 0, (cudaStream_t)stream);
}
