// The 8-bit paged KV cache's block format and the conversions its kernels share.
//
// A block holds one page (16 tokens) of one KV head: 16 rows of HD K codes, 16 rows of V codes
// (e4m3, a row's 16-byte chunks permuted by token, see kv8_k_pos / kv8_v_pos), the scales 2^ek
// and 2^ev as fp32, 24 spare bytes. 32 HD + 32 bytes, so blocks stay 32-byte aligned and one
// bulk copy brings codes and scales together.
#pragma once

#include "qw_internal.h"

// Every kernel here is launched with programmatic stream serialization, and each of its CTAs waits for
// the kernels before it (pdl_wait) before it reads anything or ends: a CTA that ended without
// waiting could let the kernel after this one start before the one in front has finished.

namespace {

constexpr int KV8_PAGE = 16;
constexpr int KV8_EMIN = -32;  // exponent of a page of zeros; fp16 values never need less

template <int HD>
struct Kv8 {
    static constexpr int CH = HD / 16;        // 16-byte chunks of a row
    static constexpr int VOFF = 16 * HD;      // V codes
    static constexpr int SOFF = 32 * HD;      // scales: K, V
    static constexpr int BLK = 32 * HD + 32;
};

// 16-byte position of chunk `i` of token `t` in its K row. A fragment load of 8 lanes takes 4
// chunks of two neighbouring tokens: the odd token's other half keeps them on different banks.
template <int HD>
__device__ __forceinline__ int kv8_k_pos(int t, int i) {
    return HD == 128 ? i ^ ((t & 1) << 2) : i;
}
// ... in its V row: there 8 lanes take 2 chunks of tokens t, t + 4, t + 8, t + 12.
template <int HD>
__device__ __forceinline__ int kv8_v_pos(int t, int i) {
    return HD == 128 ? i ^ ((t >> 2) << 1) : i ^ (t >> 2);
}

__device__ __forceinline__ float kv8_pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ int kv8_log2(float p) { return (int)((__float_as_uint(p) >> 23) & 255) - 127; }  // of a power of two

// Smallest e >= KV8_EMIN with amax <= 448 * 2^e = 1.75 * 2^(e + 8), amax an fp16 value >= 0.
__device__ __forceinline__ int kv8_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;
    return amax > 0.f ? max(KV8_EMIN, x - 8 + ((u & 0x7FFFFFu) > 0x600000u)) : KV8_EMIN;
}

// Two e4m3 codes (low byte first) to two halves and back (round to nearest even, |x| <= 448).
__device__ __forceinline__ uint32_t kv8_dec2(uint32_t codes16) {
    uint32_t r;
    const unsigned short c = (unsigned short)codes16;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
__device__ __forceinline__ uint32_t kv8_enc2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void kv8_dec16(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = kv8_dec2(w[i] & 0xFFFFu), b = kv8_dec2(w[i] >> 16);
        x[4 * i] = h_lo(a);
        x[4 * i + 1] = h_hi(a);
        x[4 * i + 2] = h_lo(b);
        x[4 * i + 3] = h_hi(b);
    }
}
__device__ __forceinline__ uint4 kv8_enc16(const float* x, float mul) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = kv8_enc2(x[4 * i] * mul, x[4 * i + 1] * mul) | (kv8_enc2(x[4 * i + 2] * mul, x[4 * i + 3] * mul) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude of 16 codes (exact in fp16), and of pairs of halves.
__device__ __forceinline__ uint32_t kv8_absmax2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7FFF7FFFu));
    return r;
}
__device__ __forceinline__ float kv8_max2(uint32_t m) { return fmaxf(h_lo(m), h_hi(m)); }
__device__ __forceinline__ float kv8_absmax16(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = kv8_absmax2(kv8_absmax2(m, kv8_dec2(w[i] & 0xFFFFu)), kv8_dec2(w[i] >> 16));
    return kv8_max2(m);
}
// 16 codes under a scale that is 1 / f times theirs, f a power of two.
__device__ __forceinline__ uint4 kv8_recode16(const uint4& u, float f) {
    if (f == 1.f) return u;
    float x[16];
    kv8_dec16(u, x);
    return kv8_enc16(x, f);
}

}  // namespace

// Host-side check of a view; QW_OK or the recorded error.
qw_status kv8_check(const qw_kv8* kv, int B, const char* what);

// Device view passed to the kernels. A model's cache differs from a caller's in how entries find
// their pages: through the sequence ids of the batch (row), or every entry (a layer) through the same
// row of the table with its own range of blocks (row_stride 0, page_step).
struct Kv8View {
    uint8_t* blocks;
    const int* table;
    int n_pages, max_pages, n_kv;
    const int* row;   // optional [B]: the table row of entry b
    int row_stride;   // ints between rows
    int page_step;    // added to the page ids of entry b, b times
    const int* stopped = nullptr;  // optional, by table row: non-zero leaves the row's scores as they are
};
inline Kv8View kv8_view(const qw_kv8* kv) {
    return {(uint8_t*)kv->dev_blocks, kv->dev_page_table, kv->n_pages, kv->max_pages, kv->n_kv_heads, nullptr, kv->max_pages, 0, nullptr};
}
#ifdef __CUDACC__
__device__ __forceinline__ const int* kv8_row(const Kv8View& v, const int* table, int b) {
    return table + (size_t)(v.row ? v.row[b] : b) * v.row_stride;
}
__device__ __forceinline__ bool kv8_stopped(const Kv8View& v, int b) { return v.stopped && v.stopped[v.row ? v.row[b] : b]; }
__device__ __forceinline__ uint8_t* kv8_block(const Kv8View& v, int b, int page, int head, int blk) {
    return v.blocks + ((size_t)(page + b * v.page_step) * v.n_kv + head) * blk;
}
#endif

// The operators behind the C entry points (arguments checked by the caller); errors recorded.
// staged: K and V rows in pages of 16 tokens, [T / 16][n_kv][16][head_dim] fp16.
qw_status kv8_append(const Kv8View& v, int head_dim, int B, int T, int max_len, const int* start, const int* cu, const void* k,
                     size_t ld_k, const void* val, size_t ld_v, int dtype, bool staged, int* status, cudaStream_t st,
                     int* launches = nullptr);
// Scores of entry b: rows (score_mul * row[b] + score_add) * n_kv .. of the score arrays.
// ws_bytes also decides whether the logits of a decode with scores are kept.
int kv8_sm_count();  // of the device that is current at the first call
// Bytes of a call's query tiles laid out for the scores.
size_t kv8_prep_bytes(int n_kv, int head_dim, int B, int T, int G);
qw_status kv8_attn(const Kv8View& v, int head_dim, const qw_kv8_attn_args& a, int score_mul, int score_add, cudaStream_t st,
                   int* launches = nullptr);
// len_step 0: one length for every entry.
qw_status kv8_evict(const Kv8View& v, int head_dim, int B, int max_len, const int* len, int len_step, int keep, int recent,
                    const int* dst, const float* score, float* score_out, size_t ld_score, int* kept, int* new_len, int* status,
                    cudaStream_t st);
