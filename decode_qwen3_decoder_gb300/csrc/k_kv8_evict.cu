// Eviction from the 8-bit paged KV cache by accumulated attention weight (qw_kv8_evict).
//
// For each (entry, KV head) of L > n_keep tokens, the m = n_keep - n_recent largest scores among the
// first L - n_recent positions are kept, with the last n_recent; the kept rows and their scores move
// to positions 0 .. n_keep - 1 in order. Bytes bound it: the scores once, the kept rows in and out.
//
// k_kv8_select finds the positions: a radix select over sortable 32-bit keys (8 bits a pass,
// integer counts, so ties and order are exact), then a scan writes them in ascending order. The
// select is a chain of passes, so long entries get a cluster of C CTAs a head, which keep their
// slices of the keys in shared memory and add each other's 256-bin histograms through distributed
// shared memory (2048 bins, one pass less, cost 60 us a pass in remote loads). What bounds it is that
// chain: 15 us for 224 heads of 4k tokens, 27 for 64 of 1k-32k; their scores' bytes are 1.
// k_kv8_move copies rows and scores to their new places, all of them at once, a warp a page: 58 us for
// 28 layers of 4k tokens halved (235 MB of rows; rows are 128 bytes at 32-byte offsets, of which DRAM
// reads 1.4 times the bytes: 245 MB, 4.2 TB/s). A warp for K and one for V took 70 us, more registers
// than 80 a thread 73.
// k_kv8_move_inplace does it where source and destination are the same memory: new position j takes
// the row of kept[j] >= j, so one CTA a head moves batches of ascending pages with a barrier between
// a batch's reads and its writes: with the select, 96 us for 28 layers of 4k tokens halved, 700 for 32k
// (1.9 GB of rows, 2.7 TB/s). (One kernel of clusters for everything took 243 us for 28 layers of
// 4k tokens halved; the two take 74.) k_kv8_evict_one does both for short entries, where a second
// launch would cost more than it moves.
#include "kv8.cuh"

#include <algorithm>

namespace {

constexpr int EV_T = 512, EV_W = EV_T / 32;
constexpr int EV_BINS = 256;
constexpr int EV_CAP = 6144;           // keys of a CTA's slice kept in shared memory; the rest is read again
// CTAs of a long entry's cluster: of 64 entries x heads of 1k-32k tokens 57 us with 8, 68 with 4, 209 with 1
constexpr int EV_C = 8;
// Longest entry (max_len) whose positions one CTA selects: 64 x 4k tokens 56 us, with a cluster 61 (28
// layers of 8 heads: 145 and 188); 64 x 6k 48 and 45
constexpr int EV_ONE_CTA = 6144;
constexpr int EV_ONE_KEEP = 512;       // most kept tokens that the same CTA moves (two rounds of its warps)

struct Kv8EvictP {
    Kv8View kv;
    const int* len;
    int len_step;    // 0: one length for every entry
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

// Barrier of the cluster's CTAs (of the CTA for C = 1), ordering shared and global memory.
template <int C>
__device__ __forceinline__ void ev_sync() {
    if (C == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit word at `p` (this CTA's shared memory) in CTA `rank` of the cluster.
template <int C>
__device__ __forceinline__ int ev_peer(const int* p, int rank) {
    if (C == 1) return *p;
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
    int v;
    asm volatile("{\n\t.reg .b32 t;\n\tmapa.shared::cluster.u32 t, %1, %2;\n\tld.shared::cluster.s32 %0, [t];\n\t}"
                 : "=r"(v)
                 : "r"(a), "r"(rank)
                 : "memory");
    return v;
}

// Writes kept and new_len of (entry b, head); false if the entry is left out.
template <int C>
__device__ __forceinline__ bool select_kept(const Kv8EvictP& p, int rank, int head, int b) {
    __shared__ uint32_t keys[EV_CAP];
    __shared__ int hist[EV_W][EV_BINS];  // a warp its own: equal scores would queue on one bin
    __shared__ int sums[2][EV_BINS];
    __shared__ int ws[EV_W];
    __shared__ int s_digit, s_above, s_bad, pub[2];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int L = p.len[b * p.len_step];
    const int* table = kv8_row(p.kv, p.kv.table, b);
    const int* dst = kv8_row(p.kv, p.dst, b);
    const float* score = p.score + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
    int* kept = p.kept + ((size_t)b * p.kv.n_kv + head) * p.keep;
    const int n = min(L, p.keep);
    const int m = p.keep - p.recent, cand = max(0, L - p.recent);  // m of the first cand positions are kept
    const bool fits = L >= 0 && L <= p.max_len && (long long)L <= (long long)p.kv.max_pages * KV8_PAGE;
    const bool select = fits && L > p.keep && m > 0;
    const int slice = (cand + C - 1) / C, k0 = min(cand, rank * slice), nk = min(cand, k0 + slice) - k0;
    if (tid == 0) s_bad = !fits;
    if (select)
        for (int j = tid; j < min(nk, EV_CAP); j += EV_T) keys[j] = ev_key(score[k0 + j]);
    for (int i = tid; i < EV_W * EV_BINS; i += EV_T) hist[0][i] = 0;
    __syncthreads();
    // the entry's pages: every CTA of the cluster comes to the same answer
    if (fits)
        for (int i = tid; i * KV8_PAGE < L; i += EV_T)
            if (table[i] < 0 || table[i] >= p.kv.n_pages || (i * KV8_PAGE < n && (dst[i] < 0 || dst[i] >= p.kv.n_pages))) s_bad = 1;
    __syncthreads();
    if (s_bad) {
        if (rank == 0) {
            if (tid == 0) atomicOr(p.status, QW_KV8_BAD_POS);
            for (int j = tid; j < p.keep; j += EV_T) kept[j] = -1;  // nothing moves
            if (head == 0 && tid == 0) p.new_len[b] = L;
        }
        return false;
    }
    auto key = [&](int j) { return j < EV_CAP ? keys[j] : ev_key(score[k0 + j]); };
    if (head == 0 && rank == 0 && tid == 0) p.new_len[b] = n;
    if (L <= p.keep) {
        for (int j = rank * EV_T + tid; j < p.keep; j += C * EV_T) kept[j] = j < L ? j : -1;
        return true;
    }
    for (int i = rank * EV_T + tid; i < p.recent; i += C * EV_T) kept[m + i] = cand + i;
    if (!select) return true;
    uint32_t prefix = 0;
    int need = m;  // of the keys that match the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int j = tid; j < nk; j += EV_T) {
            const uint32_t k = key(j);
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[warp][(k >> shift) & 255], 1);
        }
        __syncthreads();
        int* mine = sums[(shift >> 3) & 1];  // two in turn: the other is read until the next barrier
        const int digit = EV_BINS - 1 - tid;  // thread t < 256: the t-th largest digit
        if (tid < EV_BINS) {
            int c = 0;
#pragma unroll
            for (int w = 0; w < EV_W; ++w) {
                c += hist[w][digit];
                hist[w][digit] = 0;
            }
            mine[digit] = c;
        }
        ev_sync<C>();
        int cnt = 0;
        if (tid < EV_BINS)
#pragma unroll
            for (int r = 0; r < C; ++r) cnt += ev_peer<C>(mine + digit, r);
        int total;
        const int above = ev_scan(cnt, ws, total);
        if (above < need && above + cnt >= need) {
            s_digit = digit;
            s_above = above;
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)s_digit;
        need -= s_above;
        __syncthreads();
    }
    // ---- kept positions in order: thread t looks at a run of the slice ----
    const int per = (nk + EV_T - 1) / EV_T, a0 = min(nk, tid * per), a1 = min(nk, a0 + per);
    int gt = 0, tie = 0;
    for (int j = a0; j < a1; ++j) {
        const uint32_t k = key(j);
        gt += k > prefix;
        tie += k == prefix;
    }
    int gt_all, tie_all;
    int gb = ev_scan(gt, ws, gt_all), tb = ev_scan(tie, ws, tie_all);
    if (C > 1) {
        if (tid == 0) {
            pub[0] = gt_all;
            pub[1] = tie_all;
        }
        ev_sync<C>();
        for (int r = 0; r < rank; ++r) {
            gb += ev_peer<C>(pub, r);
            tb += ev_peer<C>(pub + 1, r);
        }
    }
    for (int j = a0; j < a1; ++j) {
        const uint32_t k = key(j);
        const bool t = k == prefix;
        const int at = gb + min(tb, need);  // < m, unless the scores changed meanwhile
        if ((k > prefix || (t && tb < need)) && at < m) kept[at] = k0 + j;
        gb += k > prefix;
        tb += t;
    }
    if (C > 1) ev_sync<C>();  // no CTA leaves while another may read its shared memory
    return true;
}

template <int C>
__global__ void __launch_bounds__(EV_T) k_kv8_select(const __grid_constant__ Kv8EvictP p) {
    pdl_wait();
    pdl_launch();
    select_kept<C>(p, blockIdx.x % C, blockIdx.x / C, blockIdx.y);
}

// One destination page (K and V), by one warp: fetch its rows' codes, then store them under the
// page's own exponents.
template <int HD>
struct RowMove {
    static constexpr int CH = Kv8<HD>::CH, TSTEP = 32 / CH, UPL = KV8_PAGE / TSTEP;
    uint4 code[2][UPL];
    float2 sc[UPL];
    __device__ __forceinline__ void fetch(const Kv8EvictP& p, const int* table, const int* kept, int b, int head, int d, int n, int lane) {
        const int ch = lane % CH, t0 = lane / CH;
        int src[UPL], pg[UPL];
#pragma unroll
        for (int u = 0; u < UPL; ++u) {
            const int j = d * KV8_PAGE + t0 + u * TSTEP;
            src[u] = j < n ? kept[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < UPL; ++u) pg[u] = src[u] >= 0 ? table[src[u] / KV8_PAGE] : 0;
#pragma unroll
        for (int u = 0; u < UPL; ++u) {
            code[0][u] = code[1][u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = make_float2(0.f, 0.f);
            if (src[u] < 0) continue;
            const int t = src[u] % KV8_PAGE;
            const uint8_t* blk = kv8_block(p.kv, b, pg[u], head, Kv8<HD>::BLK);
            code[0][u] = *reinterpret_cast<const uint4*>(blk + t * HD + kv8_k_pos<HD>(t, ch) * 16);
            code[1][u] = *reinterpret_cast<const uint4*>(blk + Kv8<HD>::VOFF + t * HD + kv8_v_pos<HD>(t, ch) * 16);
            sc[u] = *reinterpret_cast<const float2*>(blk + Kv8<HD>::SOFF);
        }
    }
    __device__ __forceinline__ void store(const Kv8EvictP& p, int page, int b, int head, int lane) {
        const int ch = lane % CH, t0 = lane / CH;
        uint8_t* blk = kv8_block(p.kv, b, page, head, Kv8<HD>::BLK);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float amax = 0.f;
#pragma unroll
            for (int u = 0; u < UPL; ++u) amax = fmaxf(amax, kv8_absmax16(code[which][u]) * (which ? sc[u].y : sc[u].x));
            const int e = kv8_exponent(warp_max(amax));
            const float mul = kv8_pow2(-e);
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
                const int t = t0 + u * TSTEP, at = which ? kv8_v_pos<HD>(t, ch) : kv8_k_pos<HD>(t, ch);
                *reinterpret_cast<uint4*>(blk + (which ? Kv8<HD>::VOFF : 0) + t * HD + at * 16) =
                    kv8_recode16(code[which][u], (which ? sc[u].y : sc[u].x) * mul);
            }
            if (lane == 0) reinterpret_cast<float*>(blk + Kv8<HD>::SOFF)[which] = kv8_pow2(e);
        }
    }
};

constexpr int MV_W = 8;
// blockIdx.x < row_ctas: MV_W pages of one (entry, head); above: 4 MV_W * 32 of its scores.
template <int HD>
__global__ void __launch_bounds__(MV_W * 32, 3) k_kv8_move(const __grid_constant__ Kv8EvictP p, int row_ctas, bool scores) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y, b = blockIdx.z;
    const int* kept = p.kept + ((size_t)b * p.kv.n_kv + head) * p.keep;
    pdl_wait();
    pdl_launch();
    const int L = p.len[b * p.len_step], n = min(L, p.keep);
    if (L <= 0 || kept[0] < 0) return;  // empty, or an entry left out
    if ((int)blockIdx.x < row_ctas) {
        const int d = blockIdx.x * MV_W + warp;
        if (d * KV8_PAGE >= n) return;
        RowMove<HD> mv;
        mv.fetch(p, kv8_row(p.kv, p.kv.table, b), kept, b, head, d, n, lane);
        mv.store(p, kv8_row(p.kv, p.dst, b)[d], b, head, lane);
    } else if (scores) {
        const int j0 = ((int)blockIdx.x - row_ctas) * 4 * MV_W * 32 + tid;
        const float* score = p.score + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
        float* out = p.score_out + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * MV_W * 32;
            if (j < L) out[j] = j < n ? score[kept[j]] : 0.f;
        }
    }
}

// Moves the scores and rows of (entry b, head), by one CTA, in an order that is safe within one memory.
template <int HD>
__device__ __forceinline__ void move_ordered(const Kv8EvictP& p, int head, int b, bool scores, bool rows) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int* kept = p.kept + ((size_t)b * p.kv.n_kv + head) * p.keep;
    const int L = p.len[b * p.len_step], n = min(L, p.keep);
    if (scores) {
        const float* score = p.score + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
        float* out = p.score_out + ((size_t)b * p.kv.n_kv + head) * p.ld_score;
        for (int j0 = 0; j0 < n; j0 += EV_T) {
            const int j = j0 + tid;
            const float v = j < n ? score[kept[j]] : 0.f;
            __syncthreads();
            if (j < n) out[j] = v;
        }
        __syncthreads();
        for (int j = n + tid; j < L; j += EV_T) out[j] = 0.f;
    }
    if (!rows) return;
    const int* table = kv8_row(p.kv, p.kv.table, b);
    const int* dst = kv8_row(p.kv, p.dst, b);
    for (int d0 = 0; d0 * KV8_PAGE < n; d0 += EV_W) {
        const int d = d0 + warp;
        RowMove<HD> mv;
        mv.fetch(p, table, kept, b, head, d, n, lane);
        __syncthreads();
        if (d * KV8_PAGE < n) mv.store(p, dst[d], b, head, lane);
    }
}

// What is moved within one memory: rows (p.in_place), scores (score_out == score), or both.
template <int HD>
__global__ void __launch_bounds__(EV_T) k_kv8_move_inplace(const __grid_constant__ Kv8EvictP p) {
    const int head = blockIdx.x, b = blockIdx.y;
    pdl_wait();
    pdl_launch();
    if (p.len[b * p.len_step] <= p.keep || p.kept[((size_t)b * p.kv.n_kv + head) * p.keep] < 0) return;  // nothing to move
    move_ordered<HD>(p, head, b, p.score_out == p.score, p.in_place);
}

template <int HD>
__global__ void __launch_bounds__(EV_T) k_kv8_evict_one(const __grid_constant__ Kv8EvictP p) {
    const int head = blockIdx.x, b = blockIdx.y;
    pdl_wait();
    pdl_launch();
    if (!select_kept<1>(p, 0, head, b)) return;
    __syncthreads();
    const bool same = p.len[b * p.len_step] <= p.keep;  // every token stays: what is in place is left alone
    move_ordered<HD>(p, head, b, !(same && p.score_out == p.score), !(same && p.in_place));
}

template <int HD>
cudaError_t run_evict(const Kv8EvictP& p, int B, cudaStream_t st) {
    LaunchCtx c = {st, true, nullptr};
    // One kernel saves a launch (1 x 200 tokens: 11.8 against 12.3 us with two; 8 x 1k -> 250: 15.9 against
    // 18.4) while every (entry, head) has an SM to itself; 512 of them take 72 against 57 us.
    if (p.max_len <= EV_ONE_CTA && std::min(p.keep, p.max_len) <= EV_ONE_KEEP && B * p.kv.n_kv <= kv8_sm_count())
        return launch_k(c, k_kv8_evict_one<HD>, dim3(p.kv.n_kv, B), dim3(EV_T), 0, p);
    cudaError_t e = p.max_len <= EV_ONE_CTA ? launch_k(c, k_kv8_select<1>, dim3(p.kv.n_kv, B), dim3(EV_T), 0, p)
                                            : launch_kc(c, k_kv8_select<EV_C>, dim3(EV_C * p.kv.n_kv, B), dim3(EV_T), 0, EV_C, p);
    if (e != cudaSuccess) return e;
    const bool alias = p.score_out == p.score;
    if (!p.in_place || !alias) {
        const int pages = (std::min(p.keep, p.max_len) + KV8_PAGE - 1) / KV8_PAGE;
        const int row_ctas = p.in_place ? 0 : (pages + MV_W - 1) / MV_W;
        const int score_ctas = alias ? 0 : (p.max_len + 4 * MV_W * 32 - 1) / (4 * MV_W * 32);
        e = launch_k(c, k_kv8_move<HD>, dim3(row_ctas + score_ctas, p.kv.n_kv, B), dim3(MV_W * 32), 0, p, row_ctas, !alias);
        if (e != cudaSuccess) return e;
    }
    if (p.in_place || alias) e = launch_k(c, k_kv8_move_inplace<HD>, dim3(p.kv.n_kv, B), dim3(EV_T), 0, p);
    return e;
}

}  // namespace

qw_status kv8_evict(const Kv8View& v, int head_dim, int B, int max_len, const int* len, int len_step, int keep, int recent,
                    const int* dst, const float* score, float* score_out, size_t ld_score, int* kept, int* new_len, int* status,
                    cudaStream_t st) {
    Kv8EvictP p = {v, len, len_step, dst ? dst : v.table, !dst || dst == v.table, max_len, keep, recent, score, score_out, ld_score,
                   kept, new_len, status};
    const cudaError_t e = head_dim == 128 ? run_evict<128>(p, B, st) : run_evict<64>(p, B, st);
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "evict: %s", cudaGetErrorString(e));
}

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
    return kv8_evict(kv8_view(kv), kv->head_dim, B, max_len, dev_len, 1, n_keep, n_recent, dev_dst_table, dev_score, dev_score_out,
                     ld_score, dev_kept, dev_new_len, dev_status, (cudaStream_t)stream);
}
