// K9b -- the product of two e4m3 matrices with block scales on tcgen05:
//
//   C [M, N] = sum over K blocks b of 128 of
//              a_scale[m, b] b_scale[n / 128, b] sum_{k in b} A[m, k] B[n, k]
//
// A [M, K] (rows: tokens), B [N, K] (rows: output features, as a linear layer keeps
// its weight), both K-contiguous; C bf16 or fp32.
//
// The scales change with every K block, so the tensor cores cannot accumulate over K
// on their own: each block's 128 x BN product goes to its own TMEM buffer (four
// K = 32 MMAs, one 128-byte swizzled row of each operand), and the epilogue warps
// read it, multiply by the block's scale and add it into fp32 registers while the
// next block's MMAs fill another buffer.
//
// Roles: warp 0 loads by TMA, warps 1 and 3 issue the MMAs (1 owns the TMEM), warp 2
// fetches the scales, warps 4 and up are the epilogue.  Every wait is bounded; one that
// expires raises the error word and an abort flag that the other roles check.
//
// Two operand orders.  Many tokens: tokens are the MMA's 128 rows and features its BN
// columns.  At most 64 tokens: features are the 128 rows and the tokens the 16, 32 or
// 64 columns, so that no row of the tile is empty while the weights stream by.
//
// Where the tiles leave SMs idle the K range is split over the CTAs of a cluster: each
// writes its fp32 part to its own shared memory, and after a cluster barrier every CTA
// adds a share of the tile over the cluster in rank order (the sum's order is fixed).
//
// Measured.  16384 x 8512 x 2048, bf16: 244 us = 2.34 PFLOP/s in short runs, 295 where the
// power limit holds the clock at 1.4 GHz; the MMAs alone need 174 at the rate of a 128 x
// 256 x 128-byte block in 512 clocks.  What bounds it is the round trip of a K block's
// product through its two buffers (MMAs, commit, TMEM reads, scaling, hand-back: tensor
// pipe 70 % active), with the clock beside it; L2 is at 39 %, DRAM lower.
// 4 x 8512 x 2048: 6.4 us for 17.5 MB of weights, of it about 4 launch and first loads;
// 333 x 2048 x 4112, fp32: 13.8 us, one wave of 96 tiles of 33 K blocks.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cstring>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "umma.cuh"

namespace gdn {

__device__ unsigned int g_fp8_err;

namespace fp8 {
constexpr int BM = 128, BK = 128;
constexpr uint32_t MAX_POLLS = 1u << 24;
// ring of scales: SG K blocks of the 128 rows (or columns) of tokens and of two blocks of
// features, a token's SG scales side by side
constexpr int NSC = 3, SG = 4, SC_SLOT = 130 * SG;

template <int BN_, bool SWAP_, bool PAIR_ = false> struct Shape {
    static constexpr int BN = BN_;
    static constexpr bool SWAP = SWAP_;
    static constexpr bool PAIR = PAIR_;                                 // two CTAs on one tile of 256 rows
    static constexpr int ROWS = PAIR ? 2 * BM : BM;                     // of a tile
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;                   // rows of B that one CTA loads
    static constexpr int A_ST = BM * BK, B_ST = B_ROWS * BK, ST = A_ST + B_ST;
    // Epilogue: 32 rows a warp, and 64 columns a thread (32 or 16 in the swapped order; 128
    // of a pair, whose 8 warps keep 128 sums and a read in flight in registers:
    // 16384 x 8512 x 2048 in 250 us, with 16 warps of 64 columns 470).
    static constexpr int EPC = SWAP ? (BN < 32 ? BN : 32) : PAIR ? 128 : 64;
    static constexpr int EPI_WARPS = 4 * BN / EPC;
    static constexpr int OUT_WARP = SWAP ? 0 : 64 * EPC;                 // result rows of a warp, bf16
    static constexpr int OUT = OUT_WARP * EPI_WARPS;
    static constexpr int NS = (226304 - OUT) / ST < 8 ? (226304 - OUT) / ST : 8;
    // A buffer's round trip (MMAs 512 clocks, commit, reads 350, hand-back) is longer than
    // two K blocks' MMAs, and 512 columns hold two products of 256.  So a pair's K block is
    // two products of 128 columns, each with two buffers and warps of its own: half the MMA
    // time in the same round trip.
    static constexpr int HALVES = PAIR ? 2 : 1, HN = BN / HALVES;
    static constexpr int NT = 512 / BN < 4 ? 512 / BN : 4;            // TMEM buffers of each half
    static constexpr uint32_t TMEM_COLS = NT * BN;                      // 64 .. 512, a power of two
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int OFF_OUT = NS * ST;
    static constexpr int OFF_SC = OFF_OUT + OUT;
    static constexpr int OFF_BAR = OFF_SC + NSC * SC_SLOT * 4;
    static constexpr int SMEM = OFF_BAR + 384 + 1024;                   // barriers; alignment slack
    static constexpr int PART_LD = SWAP ? BM : BN + 4;                  // split: row length of the fp32 part
    static_assert(PAIR || (SWAP ? BN * BM : BM * (BN + 4)) * 4 <= OFF_OUT, "the split's part fits in the stages");
    static_assert(SMEM <= 232448, "227 KB per block");
};
}  // namespace fp8

struct Fp8Maps {
    CUtensorMap a, b;   // MMA rows (box 128 x 128 bytes) and columns (box 128 bytes x B_ROWS, of a pair half that)
    CUtensorMap c;      // the result, boxes of 128 bytes x 32 rows (where its rows are 16-byte aligned)
};

namespace {

// kind::f8f6f4, e4m3 operands (format 0), fp32 result; both operands K-major.
// With PAIR the MMA's rows and its B operand are spread over two CTAs at the same
// shared-memory offsets.
template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// An arrival on `bar` (of both CTAs of a pair) when this thread's MMAs so far are done.
template <bool PAIR> __device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                umma::smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        umma::mma_commit(bar);
}

template <bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(umma::smem_u32(dst)),
                     "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        umma::tmem_alloc(dst, cols);
    }
}
template <bool PAIR> __device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        umma::tmem_dealloc(addr, cols);
}

// Address of the cluster's CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t at_rank(const void *p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(umma::smem_u32(p)), "r"(rank));
    return a;
}
template <bool PAIR> __device__ __forceinline__ void arrive_at(uint32_t bar) {
    if constexpr (PAIR) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
    else asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A tile into this CTA's shared memory whose bytes are counted on the barrier at cluster
// address `bar`, which may be the other CTA's of the pair.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(umma::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}

// Registers move from the loading warps to the epilogue: 4 warps x 72 + 8 x 216 is what
// 12 warps x 168 were launched with.
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// A 4-byte asynchronous copy to shared memory, zero where `in` is false (src is then any
// valid address); an arrival on `bar` once this thread's earlier copies have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;   // no clobber: loads overlap
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    memcpy(&u.x, &a, 4);
    memcpy(&u.y, &b, 4);
    *reinterpret_cast<uint2 *>(p) = u;
}

// One 16-byte chunk of a result row.
template <typename T> __device__ __forceinline__ void store_chunk(uint8_t *p, const float2 *x);
template <> __device__ __forceinline__ void store_chunk<__nv_bfloat16>(uint8_t *p, const float2 *x) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[e].x, x[e].y);
        memcpy(w + e, &b, 4);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store_chunk<float>(uint8_t *p, const float2 *x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}

// The tiles of a CTA: i, its row of tiles r (fastest) and column c.
struct Tile {
    int i, r, c;
    __device__ __forceinline__ Tile(int first, int rows) : i(first), r(first % rows), c(first / rows) {}
    __device__ __forceinline__ void next(int step, int rows) {
        i += step;
        r += step;
        while (r >= rows) { r -= rows; ++c; }
    }
};

}  // namespace

template <class Sh, typename Tout>
__global__ void __launch_bounds__(Sh::THREADS, 1)
gemm_fp8_kernel(const __grid_constant__ Fp8Maps maps, int M, int N, int K, const float *__restrict__ a_scale,
                const float *__restrict__ b_scale, Tout *__restrict__ C, long long ldc, int split, int bulk_n) {
    using namespace fp8;
    constexpr int BN = Sh::BN, NS = Sh::NS, NT = Sh::NT, EPC = Sh::EPC;
    constexpr bool SWAP = Sh::SWAP, PAIR = Sh::PAIR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = umma::align_smem<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + Sh::OFF_BAR), *empty = full + NS;
    constexpr int HALVES = Sh::HALVES, HN = Sh::HN;
    uint64_t *tfull = empty + NS, *tempty = tfull + HALVES * NT, *sfull = tempty + HALVES * NT, *sempty = sfull + NSC;
    uint64_t *mma_done = sempty + NSC;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(mma_done + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rows = SWAP ? N : M, cols = SWAP ? M : N;              // of the MMA's operands
    const int tiles_r = (rows + Sh::ROWS - 1) / Sh::ROWS, tiles_c = (cols + BN - 1) / BN;
    const int kbs = (K + BK - 1) / BK;
    const int n_tiles = tiles_r * tiles_c;
    // split > 1: one tile per cluster, rank `part` takes K blocks [k_lo, k_hi)
    const int part = split > 1 ? (int)(blockIdx.x % split) : 0;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;   // of the pair; 0 leads
    const int per_tile = PAIR ? 2 : split;
    const int first = blockIdx.x / per_tile, step = gridDim.x / per_tile;
    const int k_lo = (int)((long long)kbs * part / split), k_hi = (int)((long long)kbs * (part + 1) / split);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            umma::mbar_init(full + i, 1);
            umma::mbar_init(empty + i, HALVES);
        }
        for (int i = 0; i < HALVES * NT; ++i) {
            umma::mbar_init(tfull + i, 1);
            umma::mbar_init(tempty + i, (PAIR ? 2 : 1) * Sh::EPI_WARPS / HALVES);
        }
        for (int i = 0; i < NSC; ++i) {
            umma::mbar_init(sfull + i, 32);
            umma::mbar_init(sempty + i, Sh::EPI_WARPS);
        }
        umma::mbar_init(mma_done, 1);
        umma::mbar_init(mma_done + 1, 1);
        *abort_flag = 0;
        umma::fence_mbar_init();
    }
    if (warp == 1) tmem_alloc<PAIR>(tslot, Sh::TMEM_COLS);
    umma::tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // the other CTA's barriers are ready
    umma::tc_fence_after();
    const uint32_t tbase = *tslot;

    // A wait that expires raises the abort flag, and every later one gives up soon after:
    // the loads stop, the other roles run through their loops on whatever there is, and
    // nothing is stored.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (umma::mbar_try_wait(bar, parity)) return true;
        for (uint32_t i = 1; i < MAX_POLLS; ++i) {
            if (umma::mbar_try_wait(bar, parity)) return true;
            if ((i & 63u) == 63u && *abort_flag) return false;
        }
        atomicOr(&g_fp8_err, 1u);
        *abort_flag = 1;
        return false;
    };

    constexpr bool MOVE_REGS = Sh::EPC == 128;
    if (warp < 4) {
    if constexpr (MOVE_REGS) regs_dec<72>();
    // Loading and issuing warps walk their loops with all lanes and elect one for the
    // instruction itself: loops of a lone lane lose the uniform registers that descriptors
    // and barriers are addressed with.
    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        int st = 0, issued = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (Tile t(first, tiles_r); ok && t.i < n_tiles; t.next(step, tiles_r)) {
            const int tr = t.r, tc = t.c;
            for (int kb = k_lo; kb < k_hi; ++kb) {
                if (!(ok = __all_sync(0xffffffffu, wait(empty + st, ph)))) break;
                if (elect_one()) {
                    uint8_t *buf = sm + st * Sh::ST;
                    if constexpr (PAIR) {
                        // both halves are counted on the leader's barrier
                        const uint32_t bar = at_rank(full + st, 0);
                        if (rank == 0) umma::mbar_expect_tx(full + st, 2 * Sh::ST);
                        tma_load_pair(buf, &maps.a, BK * kb, 0, Sh::ROWS * tr + BM * rank, bar);
                        // this CTA's 64 rows of B for each half of the columns
                        for (int h = 0; h < 2; ++h)
                            tma_load_pair(buf + Sh::A_ST + h * (Sh::B_ST / 2), &maps.b, BK * kb, 0,
                                          BN * tc + HN * h + HN / 2 * rank, bar);
                    } else {
                        umma::mbar_expect_tx(full + st, Sh::ST);
                        umma::tma_load_3d(buf, &maps.a, BK * kb, 0, BM * tr, full + st);
                        umma::tma_load_3d(buf + Sh::A_ST, &maps.b, BK * kb, 0, BN * tc, full + st);
                    }
                }
                __syncwarp();
                if (issued < NS) ++issued;
                if (++st == NS) { st = 0; ph ^= 1; }
            }
        }
        // after an abort, loads still in flight land before the CTA leaves
        if (*abort_flag && rank == 0)
            for (int i = 0; i < issued; ++i) {
                if (--st < 0) { st = NS - 1; ph ^= 1; }
                umma::mbar_wait_bounded(full + st, ph ^ 1, MAX_POLLS);
            }
    } else if ((warp == 1 || warp == 3) && rank == 0) {
        // -------------------------------------------------------------- MMA issuers
        // Two warps, so that one waits for its operands and its buffer while the other's MMAs
        // are issued: they take the K blocks in turn, or of a pair's the two halves.  Every
        // product has a buffer of its own, so their order does not matter.
        constexpr uint32_t idesc = umma::idesc_f16(Sh::ROWS, HN, false, false);   // format 0 is e4m3 in this kind
        const uint64_t d0 = umma::sw128_desc(umma::smem_u32(sm), 16, 1024);
        constexpr int TURN = HALVES == 2 ? 1 : 2;   // K blocks from one of this warp's to its next
        const int half = HALVES == 2 && warp == 3;
        int skip = HALVES == 1 && warp == 3, st = skip, ts = skip;
        uint32_t ph = 0, tph = 1;
        bool any = false;
        for (int t = first; t < n_tiles; t += step) {
            int kb = k_lo + skip;
            for (; kb < k_hi; kb += TURN) {
                wait(tempty + half * NT + ts, tph);
                wait(full + st, ph);
                __syncwarp();
                umma::tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = d0 + (uint32_t)st * (Sh::ST >> 4);
                    const uint64_t bd = ad + ((Sh::A_ST + half * (Sh::B_ST / 2)) >> 4);
#pragma unroll
                    for (int ks = 0; ks < BK / 32; ++ks)   // 32 bytes of K: start address + 2 (units of 16)
                        mma_e4m3<PAIR>(tbase + (half * NT + ts) * HN, ad + 2 * ks, bd + 2 * ks, idesc, ks > 0);
                    commit<PAIR>(empty + st);
                    commit<PAIR>(tfull + half * NT + ts);
                }
                __syncwarp();
                any = true;
                if ((st += TURN) >= NS) { st -= NS; ph ^= 1; }
                if ((ts += TURN) >= NT) { ts -= NT; tph ^= 1; }
            }
            if (TURN == 2) skip = kb - k_hi;   // an odd number of K blocks: the other warp begins the next tile
        }
        // after an abort the epilogue may not have waited for the last MMAs: they
        // complete before the tensor memory is released
        if (any && *abort_flag && elect_one()) {
            commit<PAIR>(mma_done + (warp == 3));
            umma::mbar_wait_bounded(mma_done + (warp == 3), 0, MAX_POLLS);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------- scales
        // They come from L2, whose latency is several K blocks' MMAs: 4-byte asynchronous
        // copies into a ring, in flight for many blocks at once.
        int ss = 0;
        uint32_t sph = 1;
        for (Tile t(first, tiles_r); t.i < n_tiles; t.next(step, tiles_r)) {
            const int tr = t.r, tc = t.c;
            // tokens of the tile (rows, or columns in the swapped order) and blocks of features
            constexpr int TOK = SWAP ? BN : BM, PER = TOK < 32 ? 1 : TOK / 32;
            const int m0 = SWAP ? BN * tc : Sh::ROWS * tr + BM * rank, nb0 = SWAP ? tr : (BN * tc) >> 7;
            const int nb = nb0 + lane;   // lanes 0, 1: the tile's one or two blocks of 128 features
            const bool has_b = lane < (SWAP || BN <= 128 ? 1 : 2) && (long long)nb * 128 < N;
            for (int kb = k_lo; kb < k_hi; kb += SG) {
                wait(sempty + ss, sph);
                const uint32_t dst = umma::smem_u32(sm + Sh::OFF_SC) + ss * SC_SLOT * 4;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int j = 32 * i + lane, m = m0 + j;
                    const float *src = a_scale + (m < M ? (size_t)m * kbs + kb : 0);
#pragma unroll
                    for (int g = 0; g < SG; ++g)
                        if (j < TOK) copy4(dst + 4 * (SG * j + g), src + (m < M && kb + g < k_hi ? g : 0), m < M && kb + g < k_hi);
                }
                const float *src = b_scale + (has_b ? (size_t)nb * kbs + kb : 0);
#pragma unroll
                for (int g = 0; g < SG; ++g)
                    if (lane < 2) copy4(dst + 4 * (SG * (128 + lane) + g), src + (has_b && kb + g < k_hi ? g : 0), has_b && kb + g < k_hi);
                copies_arrive(sfull + ss);
                if (++ss == NSC) { ss = 0; sph ^= 1; }
            }
        }
        copies_wait();
    }
    } else {
        if constexpr (MOVE_REGS) regs_inc<216>();
        // ----------------------------------------------------------------- epilogue
        // TMEM lane quadrant warp % 4: one row of the tile per lane; each four warps take
        // the next EPC columns
        const int qd = warp & 3, c0 = EPC * ((warp - 4) >> 2);
        const int half = c0 / HN;   // buffers and barriers of this warp's product
        const uint32_t trow = tbase + ((uint32_t)(32 * qd) << 16) + half * NT * HN + c0 % HN;
        int ts = 0, ss = 0;
        uint32_t tph = 0, sph = 0;
        uint64_t *const tf = tfull + half * NT;
        const uint32_t te = PAIR ? at_rank(tempty + half * NT, 0) : umma::smem_u32(tempty);   // the issuers' copy
        float2 acc[EPC / 2];
        const float *scales = reinterpret_cast<const float *>(sm + Sh::OFF_SC);
        for (Tile t(first, tiles_r); t.i < n_tiles; t.next(step, tiles_r)) {
            const int tr = t.r, tc = t.c;
            const int row0 = Sh::ROWS * tr + BM * rank + 32 * qd, row = row0 + lane, col0 = BN * tc + c0;
#pragma unroll
            for (int j = 0; j < EPC / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int kb = k_lo; kb < k_hi; ++kb) {
                const int sg = (kb - k_lo) & (SG - 1);
                const float *sc = scales + ss * SC_SLOT;
                if (sg == 0) {
                    // SG K blocks' scales of this row times its columns' (one block of 128), or
                    // in the swapped order of the rows, to be multiplied by each column's
                    wait(sfull + ss, sph);
                    s4 = *reinterpret_cast<const float4 *>(sc + SG * (SWAP ? 128 : 128 + (c0 >> 7)));
                    if constexpr (!SWAP) {
                        const float4 r4 = *reinterpret_cast<const float4 *>(sc + SG * (32 * qd + lane));
                        s4.x *= r4.x; s4.y *= r4.y; s4.z *= r4.z; s4.w *= r4.w;
                    }
                }
                const float s = s4.x;
                s4 = make_float4(s4.y, s4.z, s4.w, 0.f);
                wait(tf + ts, tph);
                __syncwarp();
                umma::tc_fence_after();
                // 32 columns at a time, the next ones on their way while these are added
                constexpr int W = EPC < 32 ? EPC : 32, NW = EPC / W;
                uint32_t v[NW > 1 ? 2 : 1][W];
                auto load = [&](int i) {
                    if constexpr (W == 32) umma::tmem_ld32_nowait(trow + ts * HN + i * W, v[NW > 1 ? i & 1 : 0]);
                    else umma::tmem_ld16_nowait(trow + ts * HN + i * W, v[0]);
                };
                load(0);
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    umma::tmem_ld_wait();
                    if (i + 1 < NW) load(i + 1);
                    else {   // the buffer is read: the next product may take it
                        umma::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_at<PAIR>(te + 8 * ts);
                    }
                    const uint32_t *x = v[NW > 1 ? i & 1 : 0];
#pragma unroll
                    for (int j = 0; j < W; j += 2) {
                        float2 f = make_float2(s, s);
                        if constexpr (SWAP)
                            f = make_float2(sc[SG * (c0 + i * W + j) + sg] * s, sc[SG * (c0 + i * W + j + 1) + sg] * s);
                        float2 &d = acc[(i * W + j) / 2];
                        d = ffma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), f, d);
                    }
                }
                if (++ts == NT) { ts = 0; tph ^= 1; }
                if (sg == SG - 1 || kb + 1 == k_hi) {
                    __syncwarp();
                    if (lane == 0) arrive(sempty + ss);
                    if (++ss == NSC) { ss = 0; sph ^= 1; }
                }
            }
            if (*abort_flag) continue;
            auto el = [&](int j) { return j & 1 ? acc[j / 2].y : acc[j / 2].x; };
            if (split > 1) {
                // this rank's part, in the stages (every load and MMA of the tile is done)
                float *buf = reinterpret_cast<float *>(sm);
                if constexpr (SWAP) {
#pragma unroll
                    for (int j = 0; j < EPC; ++j) buf[(c0 + j) * Sh::PART_LD + 32 * qd + lane] = el(j);
                } else {
                    float *p = buf + (32 * qd + lane) * Sh::PART_LD + c0;
#pragma unroll
                    for (int j = 0; j < EPC; j += 4)
                        *reinterpret_cast<float4 *>(p + j) = make_float4(el(j), el(j + 1), el(j + 2), el(j + 3));
                }
            } else if constexpr (SWAP) {
                if (row < N) {
#pragma unroll
                    for (int j = 0; j < EPC; ++j)
                        if (col0 + j < M) C[(col0 + j) * ldc + row] = from_f32<Tout>(el(j));
                }
            } else if (bulk_n > 0) {
                // rows of this warp through shared memory (128-byte rows, swizzled), then one
                // bulk store per 128 bytes of columns.  It leaves out rows and columns outside its
                // map, but columns in whole 16 bytes only, so the map ends at the last whole ones
                // and what is behind them goes by itself.
                constexpr int SC = 128 / (int)sizeof(Tout);        // columns of a 128-byte row
                constexpr int GROUPS = Sh::OUT_WARP / 4096;        // of them in the buffer
                uint8_t *buf = sm + Sh::OFF_OUT + (warp - 4) * Sh::OUT_WARP;
#pragma unroll
                for (int j0 = 0; j0 < EPC; j0 += SC * GROUPS) {
                    if (lane == 0) umma::bulk_wait_read<0>();      // the last store has read the buffer
                    __syncwarp();
#pragma unroll
                    for (int gq = 0; gq < GROUPS && j0 + gq * SC < EPC; ++gq)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            store_chunk<Tout>(buf + gq * 4096 + umma::sw128_offset(lane, k), acc + (j0 + gq * SC + k * (SC / 8)) / 2);
                    umma::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int gq = 0; gq < GROUPS && j0 + gq * SC < EPC; ++gq)
                            if (col0 + j0 + gq * SC < bulk_n && row0 < M)
                                umma::tma_store_3d(&maps.c, col0 + j0 + gq * SC, 0, row0, buf + gq * 4096);
                        umma::bulk_commit();
                    }
                }
                if (bulk_n < N && col0 + EPC > bulk_n && row < M) {
                    Tout *crow = C + row * ldc + col0;
#pragma unroll
                    for (int j = 0; j < EPC; ++j)
                        if (col0 + j >= bulk_n && col0 + j < N) crow[j] = from_f32<Tout>(el(j));
                }
            } else if (row < M) {
                Tout *crow = C + row * ldc + col0;
#pragma unroll
                for (int j = 0; j < EPC; ++j)
                    if (col0 + j < N) crow[j] = from_f32<Tout>(el(j));
            }
        }
        if (bulk_n > 0 && lane == 0) umma::bulk_wait_all();
    }
    umma::tc_fence_before();
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        const int tr = first % tiles_r, tc = first / tiles_r;
        // the tile four elements at a time in the order of C's rows; rank `part` adds its
        // share, all ranks' loads of an element in flight together
        constexpr int V = (SWAP ? BM : BN) / 4, OUTER = SWAP ? BN : BM;
        constexpr int total = V * OUTER;
        const int lo = total * part / split, hi = total * (part + 1) / split;
        uint32_t from[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) from[p] = at_rank(sm, p < split ? p : 0);
        const bool vec = (reinterpret_cast<uintptr_t>(C) & 15) == 0 && ldc % (16 / (int)sizeof(Tout)) == 0;
        const bool whole = *abort_flag == 0;   // after an abort the parts are not complete: write nothing
        for (int i = lo + tid; whole && i < hi; i += Sh::THREADS) {
            const int o = i / V, in = 4 * (i % V);
            const long long m = SWAP ? (long long)BN * tc + o : (long long)BM * tr + o;
            const long long n = SWAP ? (long long)BM * tr + in : (long long)BN * tc + in;
            if (m >= M || n >= N) continue;
            float4 v[8];
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < split) v[p] = ld_cluster(from[p] + (uint32_t)(o * Sh::PART_LD + in) * 4);
#pragma unroll
            for (int p = 1; p < 8; ++p)
                if (p < split) {
                    v[0].x += v[p].x; v[0].y += v[p].y; v[0].z += v[p].z; v[0].w += v[p].w;
                }
            Tout *dst = C + m * ldc + n;
            if (vec && n + 4 <= N) store4(dst, v[0]);
            else {
                const float x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) dst[e] = from_f32<Tout>(x[e]);
            }
        }
        __syncwarp();
        cluster_sync();   // no CTA leaves while another still reads its part
    } else if constexpr (PAIR) {
        cluster_sync();   // the leader's MMAs read both CTAs' memory
    } else {
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc<PAIR>(tbase, Sh::TMEM_COLS);
}

namespace {

// The kernel's shared-memory limit, set once per device.
template <class Sh, typename Tout, typename Kernel> cudaError_t allow_smem(Kernel *kernel) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

// Clusters of two CTAs of this kernel that the current device runs at once (asked once
// per device and kernel).
template <typename Kernel>
cudaError_t resident_pairs(Kernel *kernel, cudaLaunchConfig_t cfg, int sms, int *pairs) {
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!cache[dev]) {
        int n = 0;
        cfg.gridDim = dim3(2 * (sms / 2));
        if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        cache[dev] = n;
    }
    *pairs = cache[dev];
    return cudaSuccess;
}

template <class Sh, typename Tout>
cudaError_t launch_shape(int M, int N, int K, const void *A, long long lda, const float *a_scale, const void *B,
                         long long ldb, const float *b_scale, void *C, long long ldc, int split, int sms,
                         cudaStream_t stream) {
    Fp8Maps m;
    std::memset(&m, 0, sizeof m);
    cudaError_t e;
    e = make_tma_mat_u8(reinterpret_cast<TmaMap *>(&m.a), Sh::SWAP ? B : A, K, Sh::SWAP ? N : M, Sh::SWAP ? ldb : lda,
                        fp8::BM);
    if (e != cudaSuccess) return e;
    e = make_tma_mat_u8(reinterpret_cast<TmaMap *>(&m.b), Sh::SWAP ? A : B, K, Sh::SWAP ? M : N, Sh::SWAP ? lda : ldb,
                        Sh::PAIR ? Sh::B_ROWS / 2 : Sh::B_ROWS);
    if (e != cudaSuccess) return e;
    // columns that bulk stores write: whole 16 bytes, where the rows are aligned to them
    constexpr int VEC = 16 / (int)sizeof(Tout);
    const int bulk_n = !Sh::SWAP && (reinterpret_cast<uintptr_t>(C) & 15) == 0 && ldc % VEC == 0 ? N / VEC * VEC : 0;
    if (bulk_n > 0 && (e = make_tma_mat_out(reinterpret_cast<TmaMap *>(&m.c), C, sizeof(Tout) == 2, bulk_n, M, ldc)) !=
                          cudaSuccess)
        return e;
    auto *kernel = gemm_fp8_kernel<Sh, Tout>;
    if ((e = allow_smem<Sh, Tout>(kernel)) != cudaSuccess) return e;
    const long long rows = Sh::SWAP ? N : M, cols = Sh::SWAP ? M : N;
    const long long tiles = ((rows + Sh::ROWS - 1) / Sh::ROWS) * ((cols + Sh::BN - 1) / Sh::BN);
    const int cluster = Sh::PAIR ? 2 : split;
    if (tiles * split > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(Sh::THREADS);
    cfg.dynamicSmemBytes = Sh::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (Sh::PAIR) {
        // as many pairs as run at once: not every SM has a partner
        int pairs = 0;
        if ((e = resident_pairs(kernel, cfg, sms, &pairs)) != cudaSuccess) return e;
        cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    }
    if ((e = cudaLaunchKernelEx(&cfg, kernel, m, M, N, K, a_scale, b_scale, static_cast<Tout *>(C), ldc, split, bulk_n)) !=
        cudaSuccess)
        return e;
    return launched();
}

template <typename Tout>
cudaError_t launch_typed(int M, int N, int K, const void *A, long long lda, const float *a_scale, const void *B,
                         long long ldb, const float *b_scale, void *C, long long ldc, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int kbs = (K + fp8::BK - 1) / fp8::BK;
    auto tiles = [&](long long rows, long long cols, int height, int bn) {
        return ((rows + height - 1) / height) * ((cols + bn - 1) / bn);
    };
    // K split where tiles leave half of the SMs idle, over at most 4 CTAs with two K blocks
    // each (4 x 2048 x 4096: 10.6 us whole, 6.2 over 4; over 8, whose clusters fit fewer at
    // once, 9.5)
    auto split_for = [&](long long n) {
        int s = 1;
        while (s < 4 && n * s * 2 <= sms && kbs >= 4 * s) s *= 2;
        return s;
    };
#define GDN_FP8(BN, SWAP, S)                                                                                       \
    launch_shape<fp8::Shape<BN, SWAP>, Tout>(M, N, K, A, lda, a_scale, B, ldb, b_scale, C, ldc, S, sms, stream)
    if (M <= 64) {
        const int s = split_for(tiles(N, M, 128, 64));
        if (M <= 16) return GDN_FP8(16, true, s);
        if (M <= 32) return GDN_FP8(32, true, s);
        return GDN_FP8(64, true, s);
    }
    // Otherwise the shape whose waves take least, by the microseconds a K block takes (in
    // hundredths): 31 at 64 columns, 34 at 128, 53 at a pair's 256 x 256 (512 x 4096 x 4096:
    // 23.6, 14.6 and 19.3 us; 2048 x 2048 x 4096: 40, 24 and 20 us)
    auto cost = [&](long long n, int at_once, int block) { return (n + at_once - 1) / at_once * block; };
    const long long t64 = tiles(M, N, 128, 64);
    const long long c64 = cost(t64, sms, 31), c128 = cost(tiles(M, N, 128, 128), sms, 34);
    const long long c256 = cost(tiles(M, N, 256, 256), sms / 2, 53);
    if (c64 <= c128 && c64 <= c256) return GDN_FP8(64, false, split_for(t64));
    if (c128 <= c256) return GDN_FP8(128, false, 1);
    return launch_shape<fp8::Shape<256, false, true>, Tout>(M, N, K, A, lda, a_scale, B, ldb, b_scale, C, ldc, 1, sms,
                                                            stream);
#undef GDN_FP8
}

}  // namespace

cudaError_t launch_gemm_fp8(int M, int N, int K, const void *A, long long lda, const float *a_scale, const void *B,
                            long long ldb, const float *b_scale, void *C, long long ldc, bool out_bf16,
                            cudaStream_t stream) {
    return out_bf16 ? launch_typed<__nv_bfloat16>(M, N, K, A, lda, a_scale, B, ldb, b_scale, C, ldc, stream)
                    : launch_typed<float>(M, N, K, A, lda, a_scale, B, ldb, b_scale, C, ldc, stream);
}

// One CTA waits, through the product's bounded wait, for a barrier phase that
// nothing completes.
__global__ void fp8_wait_selftest_kernel(uint32_t max_polls) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        umma::mbar_init(&bar, 1);
        umma::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !umma::mbar_wait_bounded(&bar, 0, max_polls)) atomicOr(&g_fp8_err, 1u);
}

cudaError_t fp8_wait_selftest(uint32_t max_polls, cudaStream_t s) {
    fp8_wait_selftest_kernel<<<1, 32, 0, s>>>(max_polls);
    return cudaGetLastError();
}

cudaError_t fp8_error_word(unsigned *v, bool clear, cudaStream_t s) { return read_error_word(g_fp8_err, v, clear, s); }

}  // namespace gdn
