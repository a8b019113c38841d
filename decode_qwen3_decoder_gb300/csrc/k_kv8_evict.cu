// Eviction from the 8-bit paged KV cache by accumulated attention weight (qw_kv8_evict).
//
// For each (entry, KV head) of L > n_keep tokens: the m = n_keep - n_recent largest scores among
// the first L - n_recent positions are found by a radix select over sortable 32-bit keys (8 bits a
// pass, integer counts, so ties and order are exact), the kept positions are written in
// ascending order by a scan, and the rows and scores move to positions 0 .. n_keep - 1. New
// position j takes the row of kept[j] >= j, so moving page after page in order, with a barrier
// between a batch's reads and its writes, is safe in place.
#include "kv8.cuh"

#include <algorithm>

namespace {

constexpr int EV_T = 512, EV_W = EV_T / 32;

struct Kv8EvictP {
    Kv8View kv;
    const int* len;
    const int* dst;  // destination page table (the entry's own when in place)
    bool in_place;
    int max_len, keep, recent;
    const float* score;
    float* score_out;
    size_t ld_score;
    int* kept;
    int* new_len;
    int* status;
};

// Orders like the value, -0 as 0, NaN above everything.
__device__ __forceinline__ uint32_t ev_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive block scan of one int per thread and its total.
__device__ __forceinline__ int ev_scan(int v, int* ws, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    if (lane == 31) ws[w] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < EV_W; ++i) {
        const int x = ws[i];
        if (i < w) before += x;
        all += x;
    }
    __syncthreads();
    total = all;
    return before + s - v;
}

template <int HD>
__global__ void __launch_bounds__(EV_T) k_kv8_evict(const __grid_constant__ Kv8EvictP p) {
    constexpr int CH = Kv8<HD>::CH, TSTEP = 32 / CH, UPL = KV8_PAGE / TSTEP;
    __shared__ int hist[EV_W][256];
    __shared__ int ws[EV_W];
    __shared__ int s_digit, s_above, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.x, b = blockIdx.y;
    const int L = p.len[b];
    const int* table = p.kv.table + (size_t)b * p.kv.max_pages;
    const int* dst = p.dst + (size_t)b * p.kv.max_pages;
    const float* score = p.score + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
    float* score_out = p.score_out + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
    int* kept = p.kept + ((size_t)b * p.kv.n_kv + head) * p.keep;
    const int n = min(L, p.keep);

    if (tid == 0) s_bad = L < 0 || L > p.max_len || (long long)L > (long long)p.kv.max_pages * KV8_PAGE;
    __syncthreads();
    if (!s_bad) {
        for (int i = tid; i * KV8_PAGE < L; i += EV_T)
            if (table[i] < 0 || table[i] >= p.kv.n_pages || (i * KV8_PAGE < n && (dst[i] < 0 || dst[i] >= p.kv.n_pages)))
                s_bad = 1;
    }
    __syncthreads();
    const bool bad = s_bad;
    if (bad) {
        if (tid == 0) atomicOr(p.status, QW_KV8_BAD_POS);
        for (int j = tid; j < p.keep; j += EV_T) kept[j] = -1;
        if (head == 0 && tid == 0) p.new_len[b] = L;
        return;
    }
    if (L <= p.keep) {
        for (int j = tid; j < p.keep; j += EV_T) kept[j] = j < L ? j : -1;
    } else {
        const int m = p.keep - p.recent, C = L - p.recent;
        uint32_t prefix = 0;
        int need = m;  // of the keys that match the prefix
        for (int shift = 24; shift >= 0 && m > 0; shift -= 8) {
            for (int i = tid; i < EV_W * 256; i += EV_T) (&hist[0][0])[i] = 0;
            __syncthreads();
            for (int j = tid; j < C; j += EV_T) {
                const uint32_t k = ev_key(score[j]);
                if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[warp][(k >> shift) & 255], 1);
            }
            __syncthreads();
            int cnt = 0;
            if (tid < 256)
                for (int w = 0; w < EV_W; ++w) cnt += hist[w][255 - tid];  // thread t: digit 255 - t
            int total;
            const int above = ev_scan(cnt, ws, total);
            if (above < need && above + cnt >= need) {
                s_digit = 255 - tid;
                s_above = above;
            }
            __syncthreads();
            prefix = (prefix << 8) | (uint32_t)s_digit;
            need -= s_above;
            __syncthreads();
        }
        int gt0 = 0, tie0 = 0;
        for (int j0 = 0; j0 < C && m > 0; j0 += EV_T) {
            const int j = j0 + tid;
            const uint32_t k = j < C ? ev_key(score[j]) : 0u;
            const int gt = j < C && k > prefix, tie = j < C && k == prefix;
            int total;
            const int before = ev_scan(gt | (tie << 16), ws, total);
            const int gb = gt0 + (before & 0xFFFF), tb = tie0 + (before >> 16);
            if (gt || (tie && tb < need)) kept[gb + min(tb, need)] = j;
            gt0 += total & 0xFFFF;
            tie0 += total >> 16;
        }
        for (int i = tid; i < p.recent; i += EV_T) kept[m + i] = C + i;
    }
    if (head == 0 && tid == 0) p.new_len[b] = n;
    __syncthreads();
    // ---- scores ----
    if (L > p.keep || score_out != score) {
        for (int j0 = 0; j0 < n; j0 += EV_T) {
            const int j = j0 + tid;
            const float v = j < n ? score[kept[j]] : 0.f;
            __syncthreads();
            if (j < n) score_out[j] = v;
        }
        __syncthreads();
        for (int j = n + tid; j < L; j += EV_T) score_out[j] = 0.f;
    }
    if (L <= p.keep && p.in_place) return;
    // ---- rows: a warp moves one tensor of one destination page ----
    const int which = warp & 1, ch = lane % CH, t0 = lane / CH;
    for (int d0 = 0; d0 * KV8_PAGE < n; d0 += EV_W / 2) {
        const int d = d0 + (warp >> 1);
        const bool on = d * KV8_PAGE < n;
        uint4 code[UPL];
        float sc[UPL];
        if (on) {
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
                const int j = d * KV8_PAGE + t0 + u * TSTEP;
                code[u] = make_uint4(0u, 0u, 0u, 0u);
                sc[u] = 0.f;
                if (j < n) {
                    const int src = kept[j], t = src % KV8_PAGE;
                    const uint8_t* blk = p.kv.blocks + ((size_t)table[src / KV8_PAGE] * p.kv.n_kv + head) * Kv8<HD>::BLK;
                    const int at = which ? kv8_v_pos<HD>(t, ch) : kv8_k_pos<HD>(t, ch);
                    code[u] = *reinterpret_cast<const uint4*>(blk + (which ? Kv8<HD>::VOFF : 0) + t * HD + at * 16);
                    sc[u] = reinterpret_cast<const float*>(blk + Kv8<HD>::SOFF)[which];
                }
            }
        }
        __syncthreads();
        if (on) {
            float amax = 0.f;
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
                float x[16];
                kv8_dec16(code[u], x);
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]) * sc[u]);
            }
            const int e = kv8_exponent(warp_max(amax));
            const float mul = kv8_pow2(-e);
            uint8_t* blk = p.kv.blocks + ((size_t)dst[d] * p.kv.n_kv + head) * Kv8<HD>::BLK;
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
                const int t = t0 + u * TSTEP, at = which ? kv8_v_pos<HD>(t, ch) : kv8_k_pos<HD>(t, ch);
                float x[16];
                kv8_dec16(code[u], x);
                *reinterpret_cast<uint4*>(blk + (which ? Kv8<HD>::VOFF : 0) + t * HD + at * 16) = kv8_enc16(x, sc[u] * mul);
            }
            if (lane == 0) reinterpret_cast<float*>(blk + Kv8<HD>::SOFF)[which] = kv8_pow2(e);
        }
    }
}

}  // namespace

extern "C" qw_status qw_kv8_evict(const qw_kv8* kv, int B, int max_len, const int32_t* dev_len, int n_keep, int n_recent,
                                  const int32_t* dev_dst_table, const float* dev_score, float* dev_score_out,
                                  size_t ld_score, int32_t* dev_kept, int32_t* dev_new_len, int32_t* dev_status,
                                  void* stream) {
    if (qw_status s = kv8_check(kv, B, "evict")) return s;
    if (!dev_len || !dev_score || !dev_score_out || !dev_kept || !dev_new_len || !dev_status)
        return qw_fail(QW_ERR_INVALID_ARG, "evict: NULL argument");
    if (max_len < 1 || (long long)max_len > (long long)kv->max_pages * 16)
        return qw_fail(QW_ERR_INVALID_ARG, "evict: max_len outside [1, 16 max_pages]");
    if (n_keep < 1 || n_recent < 0 || n_recent > n_keep)
        return qw_fail(QW_ERR_INVALID_ARG, "evict: n_keep < 1 or n_recent outside [0, n_keep]");
    if (ld_score < (size_t)max_len) return qw_fail(QW_ERR_INVALID_ARG, "evict: ld_score < max_len");
    if (dev_new_len == dev_len) return qw_fail(QW_ERR_INVALID_ARG, "evict: dev_new_len is dev_len");
    Kv8EvictP p = {kv8_view(kv), dev_len, dev_dst_table ? dev_dst_table : kv->dev_page_table,
                   !dev_dst_table || dev_dst_table == kv->dev_page_table, max_len, n_keep, n_recent, dev_score, dev_score_out,
                   ld_score, dev_kept, dev_new_len, dev_status};
    LaunchCtx c = {(cudaStream_t)stream, false, nullptr};
    const dim3 grid(kv->n_kv_heads, B);
    const cudaError_t e = kv->head_dim == 128 ? launch_k(c, k_kv8_evict<128>, grid, dim3(EV_T), 0, p)
                                              : launch_k(c, k_kv8_evict<64>, grid, dim3(EV_T), 0, p);
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "evict: %s", cudaGetErrorString(e));
}
