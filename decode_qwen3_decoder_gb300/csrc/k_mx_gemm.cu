// Products of microscaled matrices (qw_mx_linear, qw_mx_swiglu) on the block-scaled tcgen05.mma. mx.cuh
// states the format.
//
// The MMA reads codes and exponents as they lie: kind::mxf8f6f4 (X in e4m3, W in e4m3 or e2m1, 32 columns an
// instruction) or kind::mxf4 (both e2m1, 64 columns), products exact, sums in fp32 in tensor memory. Codes go
// through a ring of TMA tiles with the 128-byte swizzle, 128 bytes a row; e2m1 codes that meet e4m3 are
// spread to 8-byte halves of 16-byte chunks by the copy itself (16U4_ALIGN16B). The exponents' 512-byte tiles go
// to tensor memory by tcgen05.cp, in columns of their ring stage: a stage is refilled only after its MMAs, so no
// exponent is overwritten under an MMA.
//
// What the threads of a CTA do follows from three measurements (8192 x 8192 x 8192, 4 by 4 bits unless said; us):
// - The thread that issues tcgen05.cp waits for nothing the MMAs wait for, and issues none: its waits for shared memory
//   stand behind its copies (a stage of four MMAs 513 cycles alone, 643 to 810 with six copies and a wait in the same
//   thread). Copies from a thread of their own are hidden: 278 with one thread, 176 with two, as without any copy.
// - Waits sleep in the barrier (try_wait with a long limit): polling warps take shared-memory cycles from the MMAs,
//   whose operands and the copies of the next ones need nearly all of them. Polling waits in the three threads 8 by 4
//   bits 348 to 360, sleeping 293.
// - Accumulators are handed back by relaxed arrivals between tcgen05 fences: an arrival that releases all memory to the
//   cluster takes 0.4 us.
// That leaves 640 cycles a stage instead of 512, with every stage's data there when it is asked for: copies write 35 KB into
// shared memory while the MMAs read 32 KB from it. 161 us in 4 by 4 bits (6.8 PFLOP/s), 293 in 8 by 4 (3.8), 340 in 8 by 8.
//
// k_mx_gemm. A pair of CTAs on two SMs (tcgen05.mma.cta_group::2) has a tile of 256 rows of X (M; a TMEM lane a
// row, 128 in each CTA) by 256 of W (N): two neighbouring tiles of 128 for the linear product; the same 128 features
// of gate and up for SwiGLU, so that a thread has both of a feature, and the 32 features of a run, in its
// registers. Each CTA loads its own 128 rows of X and one of the two W tiles, both the exponents of all of W.
// Persistent; 8 epilogue warps read a finished accumulator at once (130 cycles) and convert and store it from registers
// under the next tile's MMAs; the hand-over between tiles takes 750 cycles, an eighth of a tile of 1024 columns. A second
// accumulator would leave no tensor memory for exponents; tiles of 192 columns with two were slower (248 us above).
//
// k_mx_gemm_few. For few rows of X: W's rows are the M (128 of them, of gate and of up for SwiGLU), X's the N
// (16, 64 or 128). A cluster of up to 8 CTAs shares a tile's columns out; each sends its partial sums of an
// equal part of X's rows to the CTA that owns the part (distributed shared memory), which adds them in order.
// Where the tiles alone fill the GPU the CTAs walk them, with two accumulators: W streams on under the output. W's
// bytes bound it: 60000 x 4096 by one row 41 us in 8 bits (6.0 TB/s), 23 in 4 by 4 (5.7), 27 in 8 by 4 (4.8: spread
// codes fill the ring with half as many bytes of memory).
//
// Every wait for a copy, an MMA or a warp is bounded (2 s): then QW_MX_TIMEOUT is set, and the CTA lets its copies and MMAs
// land, frees its tensor memory and ends. Two waits have no bound of their own: the cluster's barriers, which every CTA reaches
// on this way too, and tcgen05.alloc, which waits for CTAs that have the SM's columns. These wait for no CTA that could wait
// for this one's: kernels of the library whose CTAs wait for one another have an SM's shared memory to themselves, or a share
// like that of its columns (MfCfg), so that none of them is on this SM without its columns.
#include <algorithm>
#include <atomic>

#include "mx.cuh"
#include "tc_sm103.cuh"

namespace {

constexpr int MG_THREADS = 352;
constexpr int MG_X = 128 * 128, MG_W = 128 * 128, MG_SF = 1024;  // bytes: operand tiles of a stage, exponents of 128 rows (two atoms)
constexpr int MG_STAGE = MG_X + MG_W + 3 * MG_SF;
constexpr int MG_SF_COL = 256, MG_SF_COLS = 32;  // TMEM columns of the exponents, a stage's
// Linear: a warp stages its output in boxes of 32 rows by 32 columns; SwiGLU's, which is small, is stored from registers.
// Two that take turns; of 4-byte outputs one, whose space a fifth stage needs more (8192 x 1024 by 4096 8 by 4 bits
// 38.7 us, with two boxes and four stages 42.2).
template <int OUT>
struct MgCfg {
    static constexpr bool GLU = OUT == 8 || OUT == 4;
    static constexpr int BOX = GLU ? 0 : 32 * 32 * (OUT == QW_F32 ? 4 : 2);
    static constexpr int BOXES = OUT == QW_F32 ? 1 : 2;
    static constexpr int STAGES = GLU ? 6 : 5;
    static constexpr int SMEM = 1024 + STAGES * MG_STAGE + 8 * BOXES * BOX + 256;
    static_assert(SMEM <= 232448 && MG_SF_COL + STAGES * MG_SF_COLS <= 512, "shared or tensor memory");
};

// How long a wait lasts at most, and for tests the barriers that get an arrival too few (qw_mx_test_stall).
struct MxWaits {
    uint32_t ns;
    int stall;
};
__device__ __forceinline__ uint32_t count_of(const MxWaits& w, int barrier, uint32_t n) { return n + ((w.stall & barrier) != 0); }

struct MxGemmP {
    int T, M, atoms;  // rows of X, rows of W (of gate and of up), atoms of 128 columns
    int tiles_x, tiles_w, units;
    int b_row;   // first row of the tile's second W, after the first's
    int w_step;  // W rows a tile
    void* out;  // linear's output, rows of ld elements
    size_t ld;
    uint8_t *codes, *scales;  // SwiGLU's output
    int oatoms;
    int32_t* status;
    MxWaits waits;
};

// A wait as in tc_sm103.cuh, but the thread sleeps until the phase completes.
__device__ __forceinline__ bool try_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag, const MxWaits& w) {
    if (try_sleep(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!try_sleep(bar, parity))
        if (*abort_flag || globaltimer_ns() - t0 > w.ns) return false;
    return true;
}
// After a wait that gave up: copies and MMAs in flight land within microseconds; a millisecond is enough for all of them.
__device__ __forceinline__ void let_land(volatile int* abort_flag) {
    if (!*abort_flag) return;
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}
__device__ __forceinline__ uint64_t sf_desc(uint32_t a) {  // no swizzle, 8-row groups of 16-byte rows 128 bytes apart
    return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)8 << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {  // a shared address of this CTA in another's
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 32 rows of 16 bytes to 32 lanes by 4 columns, in each of the four lane quarters; in each CTA of a pair from its own
// shared memory.
template <bool PAIR>
__device__ __forceinline__ void sf_copy(uint32_t tmem, uint32_t smem) {
    if (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sf_desc(smem)) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sf_desc(smem)) : "memory");
}
// One arrival at a barrier of this CTA when this thread's copies, of both CTAs of a pair, are complete.
__device__ __forceinline__ void commit_here(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
#define MX_MMA(group, kind)                                                                                          \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                                            \
                 "setp.ne.b32 p, %6, 0;\n\t"                                                                         \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),     \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)                                              \
                 : "memory")
template <bool F4, bool PAIR>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc) {
    if (PAIR) {
        if (F4) MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
        else MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
    } else {
        if (F4) MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
        else MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
    }
}
// Instruction descriptor of the block-scaled kinds: exponent byte of B at bit 4 and of A at bit 29, formats of
// A and B at 7 and 10 (mxf8f6f4: 0 e4m3, 5 e2m1; mxf4: 1 e2m1), N >> 3 at 17, ue8m0 scales at 23, M >> 4 at 24.
constexpr uint32_t idesc_mx(uint32_t fa, uint32_t fb, int M, int N) {
    return (fa << 7) | (fb << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

// A box of 32 rows by 32 columns from a warp's shared memory to the output; rows and columns outside it are clipped.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"((uint64_t)map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}

// A warp's 32 rows (a row a lane) of 32 sums, to columns f .. f + 31 of the output. A lane's 16-byte chunks go to the
// places that the copy's swizzle gives them (rows of 128 or 64 bytes), which no two of 8 lanes share. A copy clips
// whole 16-byte chunks only: the map ends at the last whole one, what is left of M goes element by element. Every use of
// a box commits a group of copies.
template <int DT>
__device__ __forceinline__ void store_box(const CUtensorMap* map, const MxGemmP& p, uint8_t* boxes, uint32_t& uses, int t0, int f, const uint32_t* r) {
    constexpr int ES = DT == QW_F32 ? 4 : 2, ROW = 32 * ES;
    const int lane = threadIdx.x & 31, turn = DT == QW_F32 ? lane & 7 : (lane >> 1) & 3;
    if (t0 >= p.T || f >= p.M) return;
    constexpr int N = MgCfg<DT>::BOXES;
    uint8_t* box = boxes + uses++ % N * 32 * ROW;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N - 1) : "memory");  // this box has been read
    __syncwarp();
#pragma unroll
    for (int c = 0; c < ROW / 16; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = DT == QW_F32 ? r[4 * c + k] : mx_pack2<DT>(__uint_as_float(r[(8 * c + 2 * k) & 31]), __uint_as_float(r[(8 * c + 2 * k + 1) & 31]));
        *reinterpret_cast<uint4*>(box + lane * ROW + (c ^ turn) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    const int whole = p.M & ~(16 / ES - 1);
    if (lane == 0) {
        if (f < whole) tma_store_2d(map, smem_u32(box), f, t0);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (t0 + lane < p.T)
        for (int j = max(whole - f, 0); j < min(p.M - f, 32); ++j) {
            const int b = j * ES;
            const uint8_t* from = box + lane * ROW + ((b / 16) ^ turn) * 16 + b % 16;
            const size_t to = (size_t)(t0 + lane) * p.ld + f + j;
            if (DT == QW_F32) reinterpret_cast<float*>(p.out)[to] = *reinterpret_cast<const float*>(from);
            else reinterpret_cast<uint16_t*>(p.out)[to] = *reinterpret_cast<const uint16_t*>(from);
        }
}

// silu(g) u = g / (1 + e^-g) u. expf is within a unit of its last place (2^-23) wherever g lies; the sum, the quotient (the
// hardware's reciprocal, 2^-23, and the remainder, which an FMA gives exactly) and the product are rounded once each:
// 5 2^-24, as in plain fp32 arithmetic. A code has 4 bits: of 25 million (8192 x 1024 by 3072, 8 by 4 bits) 13 to 19 differ from
// those of 64 bits, the same as there. 44.7 us; with a division 57.3; without the remainder 43.4, and 2^-21.9 in place of
// 2^-22.1 at worst; with 2^t of a rounded t = -g log2 e 40.7, but then t's rounding grows with g to 2^-18.
// A quarter of both, so that the reciprocal is a normal number wherever e^-g is finite; beyond (g < -88.7) it is 0, as is h.
__device__ __forceinline__ float silu_mul(float g, float u) {
    float r;
    const float d = fminf(fmaf(expf(-g), 0.25f, 0.25f), 3.402823466e38f), n = g * 0.25f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float y = n * r;
    return fmaf(fmaf(-d, y, n), r, y) * u;
}

// A thread's run of 32 features of row t: codes and exponent. Features from M on are zeros.
template <int BITS>
__device__ __forceinline__ void store_run(const MxGemmP& p, int t, int f, const uint32_t* g, const uint32_t* u) {
    float h[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = silu_mul(__uint_as_float(g[i]), __uint_as_float(u[i]));
    if (f + 32 > p.M) {
#pragma unroll
        for (int i = 0; i < 32; ++i) h[i] = f + i < p.M ? h[i] : 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(h[i]) & 0x7FFFFFFFu);
    const int byte = mx_exp_byte<BITS>(m);
    const float inv = mx_inv_scale(byte);
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] *= inv;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t q[2];
        mx_enc8<BITS>(h + 8 * i, q);
        if (BITS == 8) w[2 * i] = q[0], w[2 * i + 1] = q[1];
        else w[i] = q[0];
    }
    uint8_t* at = p.codes + (size_t)t * p.oatoms * (MX_ATOM * BITS / 8) + (size_t)f * BITS / 8;
    if (BITS == 8)  // a whole 32-byte sector
        mx_st32(at, w);
    else
        *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    p.scales[mx_scale_word(t, f / MX_ATOM, p.oatoms) + (f / MX_RUN & 3)] = (uint8_t)byte;
}

struct MgMaps {
    CUtensorMap x, a, b;     // codes of X, of the tile's first and second W: boxes of 128 rows
    CUtensorMap sx, sa, sb;  // their exponents: boxes of the 512-byte tiles of a stage
    CUtensorMap out;         // boxes of 32 rows by 32 columns
};

// OUT: QW_F16, QW_BF16, QW_F32 (linear); 8, 4 (SwiGLU with codes of so many bits).
template <int XB, int WB, int OUT>
__global__ void __launch_bounds__(MG_THREADS, 1) k_mx_gemm(const __grid_constant__ MgMaps m, const __grid_constant__ MxGemmP p) {
    constexpr bool F4 = XB == 4;
    using C = MgCfg<OUT>;
    constexpr bool GLU = C::GLU;
    constexpr int AT = F4 ? 2 : 1;                               // atoms of 128 columns a stage
    constexpr uint32_t W_TX = WB == 4 && !F4 ? MG_W / 2 : MG_W;  // a spread tile counts its bytes in memory
    constexpr uint32_t TX = 2 * (MG_X + W_TX), SF_TX = 2 * 3 * AT * MX_TILE_BYTES;  // both CTAs' copies of a stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* boxes = smem + C::STAGES * MG_STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(boxes + 8 * C::BOXES * C::BOX);  // codes here, exponents in tensor memory (the leader's)
    uint64_t* empty = full + C::STAGES;
    uint64_t* sfull = empty + C::STAGES;  // exponents in shared memory (the leader's)
    uint64_t* accf = sfull + C::STAGES;
    uint64_t* acce = accf + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)cta_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int nk = (p.atoms + AT - 1) / AT;  // stages a tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(full + s), count_of(p.waits, QW_MX_STALL_FULL, 2));  // the producer, and the copies of exponents when they are complete
            mbar_init(smem_u32(empty + s), count_of(p.waits, QW_MX_STALL_EMPTY, 1));
            mbar_init(smem_u32(sfull + s), count_of(p.waits, QW_MX_STALL_SFULL, 1));
        }
        mbar_init(smem_u32(accf), count_of(p.waits, QW_MX_STALL_ACCF, 1));
        mbar_init(smem_u32(acce), count_of(p.waits, QW_MX_STALL_ACCE, 16));  // the epilogue warps of both CTAs
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&m.x);
        tma_prefetch_desc(rank ? &m.b : &m.a);
        tma_prefetch_desc(&m.sx);
        tma_prefetch_desc(&m.sa);
        tma_prefetch_desc(&m.sb);
        if (!GLU) tma_prefetch_desc(&m.out);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's copies complete on the leader's barriers
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch();

    if (warp == 8) {
        if (lane == 0) {
            uint32_t g = 0;
            for (int u = pair; u < p.units && !*abort_flag; u += pairs) {
                const int tw = u % p.tiles_w, tx = 2 * (u / p.tiles_w) + rank;  // tiles of 128 rows of X
                const int wa = tw * p.w_step, wb = wa + p.b_row;
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const int s = g % C::STAGES;
                    if (!wait_phase(smem_u32(empty + s), ((g / C::STAGES) & 1u) ^ 1u, abort_flag, p.waits)) {
                        *abort_flag = 1;
                        break;
                    }
                    const uint32_t st = smem_u32(smem + s * MG_STAGE), sf = st + MG_X + MG_W;
                    const uint32_t bar = map_to(smem_u32(full + s), 0), sbar = map_to(smem_u32(sfull + s), 0);
                    if (rank == 0) {
                        mbar_expect_tx(smem_u32(sfull + s), SF_TX);
                        mbar_expect_tx(smem_u32(full + s), TX);
                    }
                    // rows and tiles past a matrix's end arrive as zeros
                    tma_load_2d_pair(sf, &m.sx, sbar, 0, tx * p.atoms + kb * AT);
                    tma_load_2d_pair(sf + MG_SF, &m.sa, sbar, 0, (wa >> 7) * p.atoms + kb * AT);
                    tma_load_2d_pair(sf + 2 * MG_SF, &m.sb, sbar, 0, (wb >> 7) * p.atoms + kb * AT);
                    tma_load_2d_pair(st, &m.x, bar, kb * 128, tx * 128);
                    tma_load_2d_pair(st + MG_X, rank ? &m.b : &m.a, bar, kb * 128, rank ? wb : wa);
                }
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_mx(F4 ? 1 : 0, F4 ? 1 : WB == 4 ? 5 : 0, 256, 256);
            uint32_t g = 0;
            int i = 0;
            bool ok = true;
            for (int u = pair; u < p.units && ok; u += pairs, ++i) {
                ok = wait_phase(smem_u32(acce), ((uint32_t)i & 1u) ^ 1u, abort_flag, p.waits);
                for (int kb = 0; kb < nk && ok; ++kb, ++g) {
                    const int s = g % C::STAGES;
                    ok = wait_phase(smem_u32(full + s), (g / C::STAGES) & 1u, abort_flag, p.waits);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * MG_STAGE);
                    const uint32_t ta = tmem + MG_SF_COL + s * MG_SF_COLS, tb = ta + 8;
                    const int at = min(AT, p.atoms - kb * AT);
                    const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + MG_X);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // 32 bytes of a row: 32 columns with the exponents' byte k, or 64 with bytes 2 k % 4 and the next
                        const int a = F4 ? k / 2 : 0;
                        const uint32_t id = F4 ? (uint32_t)(k & 1) * 2 : (uint32_t)k;
                        if (a < at)
                            mma_mx<F4, true>(tmem, ad + 2 * k, bd + 2 * k, idesc | (id << 4) | (id << 29), ta + 4 * a, tb + 8 * a, kb > 0 || k > 0);
                    }
                    umma_commit_pair(smem_u32(empty + s));
                }
                if (ok) umma_commit_pair(smem_u32(accf));
            }
            if (!ok) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp == 10) {
        // exponents to tensor memory
        if (lane == 0 && rank == 0) {
            const uint32_t total = (uint32_t)((p.units - pair + pairs - 1) / pairs) * nk;
            for (uint32_t g = 0; g < total; ++g) {
                const int s = g % C::STAGES;
                if (!wait_phase(smem_u32(sfull + s), (g / C::STAGES) & 1u, abort_flag, p.waits)) {
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t sf = smem_u32(smem + s * MG_STAGE) + MG_X + MG_W, to = tmem + MG_SF_COL + s * MG_SF_COLS;
#pragma unroll
                for (int a = 0; a < AT; ++a) {
                    sf_copy<true>(to + 4 * a, sf + a * MX_TILE_BYTES);
                    sf_copy<true>(to + 8 + 8 * a, sf + MG_SF + a * MX_TILE_BYTES);
                    sf_copy<true>(to + 8 + 8 * a + 4, sf + 2 * MG_SF + a * MX_TILE_BYTES);
                }
                commit_here(smem_u32(full + s));
            }
        }
        __syncwarp();
    } else {
        // warps w and w + 4 read the lanes 32 (w % 4) ..: the first half of the features and the second
        const int half = warp >> 2;
        const uint32_t row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t free_bar = map_to(smem_u32(acce), 0);
        uint32_t uses = 0;
        int i = 0;
        for (int u = pair; u < p.units; u += pairs, ++i) {
            const int tw = u % p.tiles_w, tx = 2 * (u / p.tiles_w) + rank;
            const int t = tx * 128 + (warp & 3) * 32 + lane;
            int ok = 0;
            if (lane == 0) ok = wait_phase(smem_u32(accf), (uint32_t)i & 1u, abort_flag, p.waits);
            if (!__shfl_sync(0xffffffffu, ok, 0)) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            // into registers at once: the next tile's MMAs run while this one is converted and stored
            uint32_t r[4][32];
            if (GLU) {
                TMEM_LD32(row + half * 64, r[0]);
                TMEM_LD32(row + 128 + half * 64, r[1]);
                TMEM_LD32(row + half * 64 + 32, r[2]);
                TMEM_LD32(row + 128 + half * 64 + 32, r[3]);
            } else {
                TMEM_LD32(row + half * 128, r[0]);
                TMEM_LD32(row + half * 128 + 32, r[1]);
                TMEM_LD32(row + half * 128 + 64, r[2]);
                TMEM_LD32(row + half * 128 + 96, r[3]);
            }
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            // only tensor memory is handed over, which the tcgen05 fences order
            if (lane == 0) asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(free_bar) : "memory");
            if constexpr (GLU) {
                if (t < p.T) {
                    store_run<OUT>(p, t, tw * 128 + half * 64, r[0], r[1]);
                    store_run<OUT>(p, t, tw * 128 + half * 64 + 32, r[2], r[3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    store_box<OUT>(&m.out, p, boxes + warp * C::BOXES * C::BOX, uses, t - lane, tw * 256 + half * 128 + 32 * k, r[k]);
            }
        }
        if (!GLU && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, QW_MX_TIMEOUT);
    let_land(abort_flag);
    cluster_sync();  // no copy, MMA or arrival of the pair still targets this CTA
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---- few rows of X --------------------------------------------------------------------------------------------

struct MfP {
    int T, M, atoms, oatoms;
    int tiles_w, lsplits;         // log2 of the CTAs that share a tile
    const uint8_t *sx, *sa, *sb;  // exponents of X, W (gate) and up
    int dtype, bits;              // of the output
    void* out;
    size_t ld;
    uint8_t *codes, *scales;
    int32_t* status;
    MxWaits waits;
};
struct MfMaps {
    CUtensorMap x, a, b;
};

constexpr int MF_THREADS = 224;
template <bool F4, bool GLU, int BN>
struct MfCfg {
    static constexpr int NW = GLU ? 2 : 1;  // tiles of W
    static constexpr int AT = F4 ? 2 : 1;   // atoms of 128 columns a stage
    static constexpr int STAGE = NW * MG_W + BN * 128 + (NW + 1) * MG_SF;
    // two CTAs an SM, or one with more rows of X. One row by 60000 x 4096 in 8 bits: 41 us; with 3 stages and three CTAs 52
    static constexpr int STAGES = BN == 16 ? (GLU ? 3 : 5) : GLU ? 5 : BN == 64 ? 4 : 6;
    static constexpr int SF_COLS = (NW + 1) * AT * 4, SF_COL = 2 * NW * BN;  // after two accumulators
    static constexpr int COLS_USED = SF_COL + STAGES * SF_COLS;
    static constexpr int COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    // CTAs of a cluster wait for one another, so none may wait for tensor memory that another cluster holds: a CTA asks for
    // as large a share of the SM's shared memory (228 KB, 1 of it taken) as of its tensor memory. Whatever shares an
    // SM then has its columns.
    static constexpr int NEED = 1024 + STAGES * STAGE + 256, SHARE = COLS * 456 - 1024;
    static constexpr int SMEM = NEED > SHARE ? NEED : SHARE;
    static constexpr int PER_SM = 233472 / (SMEM + 1024);  // CTAs that share an SM
    static_assert(COLS_USED <= COLS && (PER_SM == 1 || PER_SM == 2) && PER_SM * COLS <= 512 && SMEM <= 232448, "shared or tensor memory");
    static_assert(NW * BN * 512 <= STAGES * STAGE, "partial sums");
};

// A lane's feature f of rows t .. t + min(n, N) - 1; 8 at a time, so that their loads, reductions and stores overlap.
// GLU: the warp has a run of 32 features, lane l the l-th.
template <int DT, int N>
__device__ __forceinline__ void store_few(const MfP& p, int t, int n, int f, const float* v) {
    const size_t at = (size_t)t * p.ld + f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n && f < p.M) {
            if (DT == QW_F32) reinterpret_cast<float*>(p.out)[at + i * p.ld] = v[i];
            else reinterpret_cast<uint16_t*>(p.out)[at + i * p.ld] = (uint16_t)mx_pack2<DT>(v[i], 0.f);
        }
}
template <bool GLU, int N>
__device__ __forceinline__ void finish_few(const MfP& p, int t, int n, int f, const float* a, const float* b) {
    if (!GLU) {
        if (p.dtype == QW_F32) store_few<QW_F32, N>(p, t, n, f, a);
        else if (p.dtype == QW_BF16) store_few<QW_BF16, N>(p, t, n, f, a);
        else store_few<QW_F16, N>(p, t, n, f, a);
        return;
    }
    const int lane = threadIdx.x & 31;
    float h[8] = {};
    int byte[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = f < p.M ? silu_mul(a[i], b[i]) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h[i]) & 0x7FFFFFFFu);
        byte[i] = p.bits == 8 ? mx_exp_byte<8>(m) : mx_exp_byte<4>(m);
        h[i] *= mx_inv_scale(byte[i]);
    }
    const size_t row = (size_t)p.oatoms * (MX_ATOM * p.bits / 8);
    uint8_t* at = p.codes + (size_t)t * row;
    uint32_t q[2];
    if (p.bits == 8) {
        mx_enc8<8>(h, q);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) at[i * row + f] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
    } else {
        mx_enc8<4>(h, q);
        const uint32_t next = __shfl_down_sync(0xffffffffu, q[0], 1);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n && (lane & 1) == 0) at[i * row + f / 2] = (uint8_t)((q[0] >> (4 * i) & 15u) | (next >> (4 * i) & 15u) << 4);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane == i && i < n) p.scales[mx_scale_word(t + i, f / MX_ATOM, p.oatoms) + (f / MX_RUN & 3)] = (uint8_t)byte[i];
}

template <int XB, int WB, bool GLU, int BN>
__global__ void __launch_bounds__(MF_THREADS) k_mx_gemm_few(const __grid_constant__ MfMaps m, const __grid_constant__ MfP p) {
    constexpr bool F4 = XB == 4;
    using C = MfCfg<F4, GLU, BN>;
    constexpr int AT = C::AT, NW = C::NW;
    constexpr uint32_t W_TX = WB == 4 && !F4 ? MG_W / 2 : MG_W;  // a spread tile counts its bytes in memory
    constexpr int SF = NW * MG_W + BN * 128;                     // exponents of W, up and X in a stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE);
    uint64_t* empty = full + C::STAGES;
    uint64_t* sfull = empty + C::STAGES;
    uint64_t* accf = sfull + C::STAGES;   // [2] accumulator complete
    uint64_t* acce = accf + 2;            // [2] accumulator read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = 1 << p.lsplits, z = S > 1 ? (int)cta_rank() : 0;
    const int tw0 = blockIdx.x >> p.lsplits, step = S > 1 ? p.tiles_w : gridDim.x;  // this CTA's tiles; one if it shares it
    const int nk_all = (p.atoms + AT - 1) / AT;
    const int kb0 = (nk_all * z) >> p.lsplits, nk = ((nk_all * (z + 1)) >> p.lsplits) - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(full + s), count_of(p.waits, QW_MX_STALL_FULL, 2));
            mbar_init(smem_u32(empty + s), count_of(p.waits, QW_MX_STALL_EMPTY, 1));
            mbar_init(smem_u32(sfull + s), count_of(p.waits, QW_MX_STALL_SFULL, 1));
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(accf + b), count_of(p.waits, QW_MX_STALL_ACCF, 1));
            mbar_init(smem_u32(acce + b), count_of(p.waits, QW_MX_STALL_ACCE, 4));
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch_desc(&m.a);
        tma_prefetch_desc(&m.x);
        if (GLU) tma_prefetch_desc(&m.b);
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(C::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch();

    if (warp == 4) {
        if (lane == 0) {
            uint32_t g = 0;
            for (int tw = tw0; tw < p.tiles_w && !*abort_flag; tw += step)
                for (int j = 0; j < nk; ++j, ++g) {
                    const int s = g % C::STAGES, kb = kb0 + j;
                    if (!wait_phase(smem_u32(empty + s), ((g / C::STAGES) & 1u) ^ 1u, abort_flag, p.waits)) {
                        *abort_flag = 1;
                        break;
                    }
                    const uint32_t st = smem_u32(smem + s * C::STAGE), bar = smem_u32(full + s), sbar = smem_u32(sfull + s);
                    const uint32_t n = (uint32_t)min(AT, p.atoms - kb * AT) * MX_TILE_BYTES;
                    mbar_expect_tx(sbar, (NW + 1) * n);
                    mbar_expect_tx(bar, NW * W_TX + BN * 128);
                    const size_t at = (size_t)kb * AT;
                    bulk_load(st + SF, p.sa + ((size_t)tw * p.atoms + at) * MX_TILE_BYTES, n, sbar);
                    if (GLU) bulk_load(st + SF + MG_SF, p.sb + ((size_t)tw * p.atoms + at) * MX_TILE_BYTES, n, sbar);
                    bulk_load(st + SF + NW * MG_SF, p.sx + at * MX_TILE_BYTES, n, sbar);
                    tma_load_2d(st, &m.a, bar, kb * 128, tw * 128);
                    if (GLU) tma_load_2d(st + MG_W, &m.b, bar, kb * 128, tw * 128);
                    tma_load_2d(st + NW * MG_W, &m.x, bar, kb * 128, 0);
                }
        }
        __syncwarp();
    } else if (warp == 5) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_mx(F4 ? 1 : WB == 4 ? 5 : 0, F4 ? 1 : 0, 128, BN);
            uint32_t g = 0;
            int i = 0;
            bool ok = true;
            for (int tw = tw0; tw < p.tiles_w && ok; tw += step, ++i) {
                const int buf = i & 1;
                ok = wait_phase(smem_u32(acce + buf), ((uint32_t)(i >> 1) & 1u) ^ 1u, abort_flag, p.waits);
                const uint32_t d = tmem + buf * NW * BN;
                for (int j = 0; j < nk && ok; ++j, ++g) {
                    const int s = g % C::STAGES;
                    ok = wait_phase(smem_u32(full + s), (g / C::STAGES) & 1u, abort_flag, p.waits);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * C::STAGE), sf = tmem + C::SF_COL + s * C::SF_COLS;
                    const int at = min(AT, p.atoms - (kb0 + j) * AT);
                    const uint64_t xd = sw128_desc(st + NW * MG_W);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // as in k_mx_gemm
                        const int a = F4 ? k / 2 : 0;
                        const uint32_t id = F4 ? (uint32_t)(k & 1) * 2 : (uint32_t)k;
                        if (a >= at) continue;
#pragma unroll
                        for (int w = 0; w < NW; ++w)
                            mma_mx<F4, false>(d + w * BN, sw128_desc(st + w * MG_W) + 2 * k, xd + 2 * k, idesc | (id << 4) | (id << 29),
                                              sf + (w * AT + a) * 4, sf + (NW * AT + a) * 4, j > 0 || k > 0);
                    }
                    umma_commit(smem_u32(empty + s));
                }
                if (ok) umma_commit(smem_u32(accf + buf));
            }
            if (!ok) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp == 6) {
        if (lane == 0) {
            const uint32_t total = (uint32_t)((p.tiles_w - tw0 + step - 1) / step) * nk;
            for (uint32_t g = 0; g < total; ++g) {
                const int s = g % C::STAGES;
                if (!wait_phase(smem_u32(sfull + s), (g / C::STAGES) & 1u, abort_flag, p.waits)) {
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t from = smem_u32(smem + s * C::STAGE) + SF, to = tmem + C::SF_COL + s * C::SF_COLS;
#pragma unroll
                for (int w = 0; w <= NW; ++w)
#pragma unroll
                    for (int a = 0; a < AT; ++a) sf_copy<false>(to + (w * AT + a) * 4, from + w * MG_SF + a * MX_TILE_BYTES);
                umma_commit(smem_u32(full + s));
            }
        }
        __syncwarp();
    }
    const int fl = warp * 32 + lane, ncols = p.T;
    const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    if (warp < 4) {
        int i = 0;
        for (int tw = tw0; tw < p.tiles_w; tw += step, ++i) {
            const int buf = i & 1, f = tw * 128 + fl;
            int got = 0;
            if (lane == 0) got = wait_phase(smem_u32(accf + buf), (uint32_t)(i >> 1) & 1u, abort_flag, p.waits);
            ok = __shfl_sync(0xffffffffu, got, 0);
            if (!ok) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            if (S > 1) break;  // the sums of the others first
            const uint32_t acc = row + buf * NW * BN;
            for (int c0 = 0; c0 < ncols; c0 += 16) {
                uint32_t r[NW][16];
#pragma unroll
                for (int w = 0; w < NW; ++w) TMEM_LD16(acc + w * BN + c0, r[w]);
                tmem_wait_ld();
                if (c0 + 16 >= ncols) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(acce + buf)) : "memory");
                }
                const float *a = reinterpret_cast<const float*>(r[0]), *b = reinterpret_cast<const float*>(r[NW - 1]);
                if (ncols == 1) finish_few<GLU, 1>(p, 0, 1, f, a, b);
                else finish_few<GLU, 8>(p, c0, ncols - c0, f, a, b);
                if (c0 + 8 < ncols) finish_few<GLU, 8>(p, c0 + 8, ncols - c0 - 8, f, a + 8, b + 8);
            }
        }
    }
    if (S > 1) {
        // partial sums [splits][own rows of X][NW][128], over the ring once every CTA of the cluster has done its MMAs
        const int lown = (BN == 16 ? 4 : BN == 64 ? 6 : 7) - p.lsplits, own = 1 << lown, f = tw0 * 128 + fl;
        const uint32_t red = smem_u32(smem);
        cluster_sync();
        if (warp < 4 && ok) {
            for (int c0 = 0; c0 < ncols; c0 += 16) {
                uint32_t r[NW][16];
#pragma unroll
                for (int g = 0; g < NW; ++g) TMEM_LD16(row + g * BN + c0, r[g]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int c = c0 + j;
                    if (j && c >= ncols) continue;
                    const uint32_t to = map_to(red + (((z << lown) + (c & (own - 1))) * NW * 128 + fl) * 4, (uint32_t)(c >> lown));
#pragma unroll
                    for (int g = 0; g < NW; ++g) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + g * 512), "r"(r[g][j]) : "memory");
                }
            }
        }
        cluster_sync();
        if (warp < 4 && ok) {
            const float* part = reinterpret_cast<const float*>(smem);
            const int mine = min(own, ncols - z * own);
            if (ncols == 1) {
                if (mine == 1) {
                    float v[NW] = {};
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int g = 0; g < NW; ++g) v[g] += part[((s << lown) * NW + g) * 128 + fl];
                    finish_few<GLU, 1>(p, 0, 1, f, v, v + NW - 1);
                }
            } else {
                for (int c = 0; c < mine; c += 8) {
                    float v[NW][8] = {};
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int g = 0; g < NW; ++g)
                                if (c + i < mine) v[g][i] += part[(((s << lown) + c + i) * NW + g) * 128 + fl];
                    finish_few<GLU, 8>(p, z * own + c, mine - c, f, v[0], v[NW - 1]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, QW_MX_TIMEOUT);
    let_land(abort_flag);
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::COLS) : "memory");
    }
}

// ---- host ------------------------------------------------------------------------------------------------

std::atomic<uint32_t> wait_ns{(uint32_t)kTcWaitNs};
std::atomic<int> stall{0};
MxWaits waits() { return {wait_ns.load(std::memory_order_relaxed), stall.load(std::memory_order_relaxed)}; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled find_encode() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return (EncodeTiled)f;
}

// Tiles of `box` rows by 128 bytes of shared memory. spread: 4-bit codes to 16-byte chunks of 16.
bool encode(CUtensorMap* map, const qw_mx& m, bool spread, unsigned box) {
    static const EncodeTiled enc = find_encode();
    if (!enc) return false;
    const cuuint64_t bytes = mx_row_bytes(m.bits, m.cols);
    const cuuint64_t dims[2] = {spread ? 2 * bytes : bytes, (cuuint64_t)m.rows}, strides[1] = {bytes};
    const cuuint32_t boxes[2] = {128, box}, es[2] = {1, 1};
    return enc(map, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.dev_codes, dims,
               strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stage's exponents: `box` of the 512-byte tiles.
bool encode_scales(CUtensorMap* map, const qw_mx& m, unsigned box) {
    static const EncodeTiled enc = find_encode();
    if (!enc) return false;
    const cuuint64_t tiles = ((cuuint64_t)m.rows + 127) / 128 * mx_atoms(m.cols);
    const cuuint64_t dims[2] = {MX_TILE_BYTES / 4, tiles}, strides[1] = {MX_TILE_BYTES};
    const cuuint32_t boxes[2] = {MX_TILE_BYTES / 4, box}, es[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, m.dev_scales, dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of 32 rows by 32 columns of an output.
bool encode_out(CUtensorMap* map, void* out, int rows, int cols, size_t ld, int dtype) {
    static const EncodeTiled enc = find_encode();
    if (!enc) return false;
    const cuuint64_t es = dtype == QW_F32 ? 4 : 2;
    const cuuint64_t whole = std::max<cuuint64_t>(cols / (16 / es), 1) * (16 / es);  // 16-byte chunks
    const cuuint64_t dims[2] = {whole, (cuuint64_t)rows}, strides[1] = {ld * es};
    const cuuint32_t boxes[2] = {32, 32}, steps[2] = {1, 1};
    const CUtensorMapDataType type = dtype == QW_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    return enc(map, type, 2, out, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
               es == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of X that k_mx_gemm_few's tiles have.
int few_box(int T) { return T <= 16 ? 16 : T <= 64 ? 64 : 128; }

// The current device and its SMs; a kernel's shared memory is allowed once a device (these calls cost a microsecond
// between them, a quarter of a small product).
struct Device {
    int id, sms;
};
Device device() {
    static std::atomic<int> sms[64];
    Device d = {0, 0};
    if (cudaGetDevice(&d.id) != cudaSuccess) return {-1, 1};
    if (d.id < 64) d.sms = sms[d.id].load(std::memory_order_relaxed);
    if (d.sms == 0) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.id) != cudaSuccess) return {-1, 1};
        if (d.id < 64) sms[d.id].store(d.sms, std::memory_order_relaxed);
    }
    return d;
}
template <typename K>
cudaError_t allow_smem(K kern, int bytes, const Device& d, std::atomic<unsigned long long>& done) {
    const unsigned long long bit = d.id >= 0 && d.id < 64 ? 1ull << d.id : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int XB, int WB, int OUT>
cudaError_t launch_gemm(const MgMaps& m, const MxGemmP& p, cudaStream_t st) {
    constexpr int SMEM = MgCfg<OUT>::SMEM;
    static std::atomic<unsigned long long> done;
    const Device d = device();
    const cudaError_t e = allow_smem(k_mx_gemm<XB, WB, OUT>, SMEM, d, done);
    if (e != cudaSuccess) return e;
    return launch_kc({st, true, nullptr}, k_mx_gemm<XB, WB, OUT>, dim3(2 * std::min(p.units, std::max(d.sms / 2, 1))), dim3(MG_THREADS),
                     SMEM, 2, m, p);
}

// Clusters of 2^l CTAs, each with an SM to itself, that the device holds at once; asked once for a device and size. A cluster
// lies within one of the GPU's groups of SMs: 15 of 8, 36 of 4 and 76 of 2 fit on 152 SMs.
template <typename K>
int clusters_of_sms(K kern, int smem, int l, const Device& d, std::atomic<int>* known) {
    std::atomic<int>* at = d.id >= 0 && d.id < 64 ? known + 4 * d.id + l : nullptr;
    int n = at ? at->load(std::memory_order_relaxed) : 0;
    if (n) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << l);
    cfg.blockDim = dim3(MF_THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << l;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (at) at->store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int XB, int WB, bool GLU, int BN>
cudaError_t launch_few_split(const MfMaps& m, MfP& p, cudaStream_t st) {
    using C = MfCfg<XB == 4, GLU, BN>;
    const auto kern = k_mx_gemm_few<XB, WB, GLU, BN>;
    static std::atomic<unsigned long long> done;
    static std::atomic<int> known[64 * 4];
    const int nk = XB == 4 ? (p.atoms + 1) / 2 : p.atoms;
    const Device d = device();
    const cudaError_t e = allow_smem(kern, C::SMEM, d, done);
    if (e != cudaSuccess) return e;
    const int slots = d.sms * C::PER_SM;
    // the widest cluster that all tiles get at once and whose CTAs have two stages at least: one row by 4096 x 4096 5.0 us with 8
    // CTAs a tile, 7.4 with two, 11 with one; by 4096 x 1024 3.5 with four, 3.9 with 8 of one stage, 4.5 with one. Clusters that
    // come second cost most of another turn: 128 rows by 2048 x 12288 with 8 a tile (16 clusters where 15 fit) 16.6 us, with four
    // 10.3. Where two CTAs share an SM, which the query does not count, a cluster takes half as many SMs; at once run 36 of 8,
    // 74 of 4 (two of the 76 that it counts find no place) and 152 of 2: one row by 37 x 128 rows of 4096 columns with 8 a tile
    // 8.1, with four 5.5, by 74 x 128 with four 6.3, by 75 x 128 10.3, with two 7.7
    p.lsplits = 0;
    for (int l = 1; l <= 3 && (long long)p.tiles_w << l <= slots && 2 << l <= nk; ++l) {
        const int at_once = C::PER_SM == 1 ? clusters_of_sms(kern, C::SMEM, l, d, known)
                            : l == 1       ? 2 * clusters_of_sms(kern, C::SMEM, 1, d, known)
                                           : clusters_of_sms(kern, C::SMEM, l - 1, d, known) - (l == 2 ? 2 : 0);
        if (p.tiles_w <= at_once) p.lsplits = l;
    }
    const LaunchCtx c = {st, true, nullptr};
    return p.lsplits ? launch_kc(c, kern, dim3(p.tiles_w << p.lsplits), dim3(MF_THREADS), C::SMEM, 1u << p.lsplits, m, p)
                     : launch_k(c, kern, dim3(std::min(p.tiles_w, slots)), dim3(MF_THREADS), C::SMEM, m, p);
}

template <int XB, int WB, bool GLU>
cudaError_t launch_few_rows(const MfMaps& m, MfP& p, cudaStream_t st) {
    if constexpr (!GLU)
        if (few_box(p.T) == 128) return launch_few_split<XB, WB, GLU, 128>(m, p, st);
    return few_box(p.T) == 64 ? launch_few_split<XB, WB, GLU, 64>(m, p, st) : launch_few_split<XB, WB, GLU, 16>(m, p, st);
}

template <bool GLU>
cudaError_t launch_few_formats(int xb, int wb, const MfMaps& m, MfP& p, cudaStream_t st) {
    return xb == 4   ? launch_few_rows<4, 4, GLU>(m, p, st)
           : wb == 4 ? launch_few_rows<8, 4, GLU>(m, p, st)
                     : launch_few_rows<8, 8, GLU>(m, p, st);
}

// Whether k_mx_gemm_few serves a product of nk stages and tiles of W. Measured against k_mx_gemm (us, 8 by 4 bits): linear, 64 rows
// by 4096 x 4096 8.1 and 13.5, by 151936 x 1024 25 and 38; 128 rows by 1024 x 8192 9.0 and 22.9, by 4096 x 2048 8.3 and 9.0,
// by 4096 x 1024 7.6 and 6.6. SwiGLU, whose runs lie across lanes here: 16 rows by 3072 x 1024 6.1 and 7.5; 64 rows by 4096 x 4096
// 12.3 and 14.9, by 3072 x 1024 9.3 and 7.5, by 6144 x 2048 (two CTAs a tile) 13.5 and 10.2.
bool few(const qw_mx& x, const qw_mx& w, bool glu) {
    const size_t nk = x.bits == 4 ? (mx_atoms(x.cols) + 1) / 2 : mx_atoms(x.cols);
    if (glu) return x.rows <= 16 || (x.rows <= 64 && nk >= 32 && 4 * mx_atoms(w.rows) <= (size_t)device().sms);
    return x.rows <= 64 || (x.rows <= 128 && nk >= 16);
}

bool product_few(const qw_mx& x, const qw_mx& wa, const qw_mx& wb, bool glu, int32_t* status, MfP& p, MfMaps& m) {
    p = MfP{};
    p.T = x.rows;
    p.M = wa.rows;
    p.atoms = (int)mx_atoms(x.cols);
    p.oatoms = (int)mx_atoms(wa.rows);
    p.tiles_w = p.oatoms;
    p.sx = (const uint8_t*)x.dev_scales;
    p.sa = (const uint8_t*)wa.dev_scales;
    p.sb = (const uint8_t*)wb.dev_scales;
    p.status = status;
    p.waits = waits();
    const bool spread = wa.bits == 4 && x.bits == 8;
    return encode(&m.x, x, false, few_box(p.T)) && encode(&m.a, wa, spread, 128) && (!glu || encode(&m.b, wb, spread, 128));
}

template <int OUT>
cudaError_t launch_formats(int xb, int wb, const MgMaps& m, const MxGemmP& p, cudaStream_t st) {
    return xb == 4   ? launch_gemm<4, 4, OUT>(m, p, st)
           : wb == 4 ? launch_gemm<8, 4, OUT>(m, p, st)
                     : launch_gemm<8, 8, OUT>(m, p, st);
}

qw_status formats_check(const qw_mx* x, const qw_mx* w, const char* what) {
    if (x->cols != w->cols) return qw_fail(QW_ERR_INVALID_ARG, "%s: x has %d columns, the weights %d", what, x->cols, w->cols);
    if (x->bits == 4 && w->bits == 8)
        return qw_fail(QW_ERR_UNSUPPORTED, "%s: 4-bit x with 8-bit weights (8 by 4, 4 by 4 and 8 by 8 are built)", what);
    return QW_OK;
}

// Parameters and tensor maps that both products share; wb: the tiles' second matrix (linear: w itself).
bool product(const qw_mx& x, const qw_mx& wa, const qw_mx& wb, bool glu, int32_t* status, MxGemmP& p, MgMaps& m) {
    p = MxGemmP{};
    p.T = x.rows;
    p.M = wa.rows;
    p.atoms = (int)mx_atoms(x.cols);
    p.oatoms = (int)mx_atoms(wa.rows);
    p.w_step = glu ? 128 : 256;
    p.b_row = glu ? 0 : 128;
    p.tiles_x = (int)(((long long)p.T + 255) / 256);
    p.tiles_w = (int)(((long long)p.M + p.w_step - 1) / p.w_step);
    p.units = p.tiles_x * p.tiles_w;
    p.status = status;
    p.waits = waits();
    const bool spread = wa.bits == 4 && x.bits == 8;
    const unsigned at = x.bits == 4 ? 2 : 1;
    if (!encode(&m.x, x, false, 128) || !encode(&m.a, wa, spread, 128) || !encode_scales(&m.sx, x, at) || !encode_scales(&m.sa, wa, at)) return false;
    m.b = m.a;
    m.sb = m.sa;
    return !glu || (encode(&m.b, wb, spread, 128) && encode_scales(&m.sb, wb, at));
}

qw_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? QW_OK : qw_fail(QW_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Tiles are numbered in an int.
bool too_many(int T, int M) { return (double)(T / 256 + 1) * (M / 128 + 1) > 2147483647.0; }

}  // namespace

extern "C" qw_status qw_mx_test_stall(int barriers, int wait_us) {
    if (barriers < 0 || barriers > 31) return qw_fail(QW_ERR_INVALID_ARG, "mx_test_stall: barriers %d", barriers);
    if (wait_us != 0 && (wait_us < 100 || wait_us > 2000000)) return qw_fail(QW_ERR_INVALID_ARG, "mx_test_stall: wait_us %d", wait_us);
    stall.store(barriers, std::memory_order_relaxed);
    wait_ns.store(wait_us ? wait_us * 1000u : (uint32_t)kTcWaitNs, std::memory_order_relaxed);
    return QW_OK;
}

extern "C" qw_status qw_mx_linear(const qw_mx* x, const qw_mx* w, void* dev_out, size_t ld_out, int dtype,
                                  int32_t* dev_status, void* stream) {
    const char* what = "mx_linear";
    if (qw_status s = mx_check(x, what, "x")) return s;
    if (qw_status s = mx_check(w, what, "w")) return s;
    if (qw_status s = formats_check(x, w, what)) return s;
    if (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) return qw_fail(QW_ERR_INVALID_ARG, "%s: dtype %d", what, dtype);
    if (!dev_status || ((uintptr_t)dev_status & 3)) return qw_fail(QW_ERR_INVALID_ARG, "%s: status NULL or not 4-byte aligned", what);
    if (x->rows == 0 || w->rows == 0) return QW_OK;
    if (!dev_out) return qw_fail(QW_ERR_INVALID_ARG, "%s: NULL out", what);
    if (ld_out < (size_t)w->rows) return qw_fail(QW_ERR_INVALID_ARG, "%s: row stride of out below w's rows", what);
    if (((uintptr_t)dev_out & 15) || ld_out % (dtype == QW_F32 ? 4 : 8))
        return qw_fail(QW_ERR_INVALID_ARG, "%s: rows of out not 16-byte aligned", what);
    if (too_many(x->rows, w->rows)) return qw_fail(QW_ERR_UNSUPPORTED, "%s: more than 2^31 tiles", what);
    const MxSpan rows = mx_rows_span(dev_out, x->rows, w->rows, ld_out, dtype);
    if (mx_meet(*x, rows) || mx_meet(*w, rows)) return qw_fail(QW_ERR_INVALID_ARG, "%s: out overlaps x or w", what);
    if (few(*x, *w, false)) {
        MfP p;
        MfMaps m;
        if (!product_few(*x, *w, *w, false, dev_status, p, m)) return qw_fail(QW_ERR_CUDA, "%s: tensor map", what);
        p.dtype = dtype;
        p.out = dev_out;
        p.ld = ld_out;
        return done(launch_few_formats<false>(x->bits, w->bits, m, p, (cudaStream_t)stream), what);
    }
    MxGemmP p;
    MgMaps m;
    if (!product(*x, *w, *w, false, dev_status, p, m) || !encode_out(&m.out, dev_out, p.T, p.M, ld_out, dtype))
        return qw_fail(QW_ERR_CUDA, "%s: tensor map", what);
    p.out = dev_out;
    p.ld = ld_out;
    const cudaStream_t st = (cudaStream_t)stream;
    return done(dtype == QW_F16    ? launch_formats<QW_F16>(x->bits, w->bits, m, p, st)
                : dtype == QW_BF16 ? launch_formats<QW_BF16>(x->bits, w->bits, m, p, st)
                                   : launch_formats<QW_F32>(x->bits, w->bits, m, p, st),
                what);
}

extern "C" qw_status qw_mx_swiglu(const qw_mx* x, const qw_mx* w_gate, const qw_mx* w_up, const qw_mx* out,
                                  int32_t* dev_status, void* stream) {
    const char* what = "mx_swiglu";
    if (qw_status s = mx_check(x, what, "x")) return s;
    if (qw_status s = mx_check(w_gate, what, "w_gate")) return s;
    if (qw_status s = mx_check(w_up, what, "w_up")) return s;
    if (w_gate->rows < 1) return qw_fail(QW_ERR_INVALID_ARG, "%s: w_gate has no rows", what);
    if (qw_status s = mx_check(out, what, "out")) return s;
    if (qw_status s = formats_check(x, w_gate, what)) return s;
    if (w_up->rows != w_gate->rows || w_up->cols != w_gate->cols || w_up->bits != w_gate->bits)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: w_gate and w_up differ in shape or bits", what);
    if (out->rows != x->rows || out->cols != w_gate->rows)
        return qw_fail(QW_ERR_INVALID_ARG, "%s: out is not [rows of x][rows of w_gate]", what);
    if (!dev_status || ((uintptr_t)dev_status & 3)) return qw_fail(QW_ERR_INVALID_ARG, "%s: status NULL or not 4-byte aligned", what);
    if (x->rows == 0) return QW_OK;
    if (too_many(x->rows, w_gate->rows)) return qw_fail(QW_ERR_UNSUPPORTED, "%s: more than 2^31 tiles", what);
    if (mx_meet(*out, *x) || mx_meet(*out, *w_gate) || mx_meet(*out, *w_up)) return qw_fail(QW_ERR_INVALID_ARG, "%s: out overlaps an input", what);
    if (few(*x, *w_gate, true)) {
        MfP p;
        MfMaps m;
        if (!product_few(*x, *w_gate, *w_up, true, dev_status, p, m)) return qw_fail(QW_ERR_CUDA, "%s: tensor map", what);
        p.bits = out->bits;
        p.codes = (uint8_t*)out->dev_codes;
        p.scales = (uint8_t*)out->dev_scales;
        return done(launch_few_formats<true>(x->bits, w_gate->bits, m, p, (cudaStream_t)stream), what);
    }
    MxGemmP p;
    MgMaps m;
    if (!product(*x, *w_gate, *w_up, true, dev_status, p, m)) return qw_fail(QW_ERR_CUDA, "%s: tensor map", what);
    p.codes = (uint8_t*)out->dev_codes;
    p.scales = (uint8_t*)out->dev_scales;
    const cudaStream_t st = (cudaStream_t)stream;
    return done(out->bits == 8 ? launch_formats<8>(x->bits, w_gate->bits, m, p, st) : launch_formats<4>(x->bits, w_gate->bits, m, p, st),
                what);
}
