// The state-space mixer's prefill for bf16 tensors on tcgen05, in chunks of 64 tokens.
// With L_t the sum of log-decays from the chunk's start through t, R_s the sum after s
// to its end, and S the state before the chunk:
//
//   y_t  = e^{L_t} C_t S + sum_{s <= t} (C_t . B_s) e^{L_t - L_s} D_s x_s + D x_t
//   S   <- e^{L_end} S + sum_s (e^{R_s} D_s) B_s x_s^T
//
// ssm_prep convolves and activates B and C once per group (H / G heads share them), and
// writes them as fp16 operand tiles with the scalars of every head.  ssm_chain runs one
// CTA per 128 state columns (two heads of 64 or one of 128) of a sequence: it convolves
// its x columns, and keeps the fp32 state in registers.
//
// Precision.  The state is held to fp32: its update takes both operands as fp16 pairs
// hi + lo (22 bits; the product lo lo, 2^-22 of the whole, is left out), three MMAs into
// one fp32 accumulator.  y is rounded to bf16, so its products take one fp16 operand
// each (2^-11 against the result's 2^-9).  fp16's narrow range does not show: every row
// of B and C is scaled by its own power of two, x and the state by one per chunk and
// head, D_s by one per chunk, and the powers are multiplied back in fp32.
//
// Tokens past a sequence's end are zeros in the tiles and zeroed in x: a tile never
// holds another sequence's rows, so its NaN stays there.
#include <cuda.h>
#include <cuda_runtime.h>

#include "ssm.cuh"
#include "umma.cuh"

namespace gdn {

__device__ unsigned int g_ssm_err;

using ssm::seq_range;

namespace stc {
constexpr int Q = 64;             // tokens per chunk
constexpr int REC = 336;          // floats of one (chunk, head) record
// record: L log2 e [64] | u [64] | u e^R [64] | 2^ec e^L [64] | 2^ec umax [64] | e^L_end, umax
constexpr int R_L = 0, R_U = 64, R_W = 128, R_YI = 192, R_YW = 256, R_DEC = 320, R_UMAX = 321;
constexpr float kLog2e = 1.44269504088896341f;
constexpr uint32_t MAX_POLLS = 1u << 24;
constexpr int THREADS = 512;
// one 64-column block of a tile: B hi | C | B lo, each 64 rows of 128 bytes.  In this
// order C is followed by B lo and preceded by B hi, so an M = 128 operand that starts
// at C (or at B hi) has the chunk's C in its rows 0..63 (or 64..127); the other rows
// are finite values whose products nobody reads.
constexpr int KB = 24576;
constexpr int OFF_C = 8192, OFF_LO = 16384;
}  // namespace stc

namespace {

// The chunks of sequence n occupy slots first(n), first(n) + 1, ...: floor(cu / 64) + n
// leaves room for every sequence's ragged last chunk without a prefix sum.
__device__ __forceinline__ int first_slot(int begin, int n) { return begin / stc::Q + n; }

// 2^k with the largest |x| of a set (its bits) scaled into [2^top, 2^{top + 1}), and
// the inverse; both stay normal numbers.
__device__ __forceinline__ void scale_pow2(uint32_t max_bits, int top, float &scale, float &inv) {
    const int e = (int)(max_bits >> 23);
    const int s = min(max(254 + top - e, 1), 253);
    scale = __uint_as_float((uint32_t)s << 23);
    inv = __uint_as_float((uint32_t)(254 - s) << 23);
}

__device__ __forceinline__ float silu_fast(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     umma::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(umma::smem_u32(bar))
                 : "memory");
}

struct PrepArgs {
    const bf16 *B, *C, *dt, *hist;
    long long ld_B, ld_C, ld_dt;
    const float *conv_w, *conv_b, *A, *b_dt;
    const int32_t *cu;
    int n_seq, n_tok, H, G, hp;
    uint8_t *tiles;   // [slot][G][N / 64][KB]
    float *rec;       // [slot][H][REC]
};

}  // namespace

// One CTA per (slot, group).
template <int N>
__global__ void __launch_bounds__(256) ssm_prep_kernel(const PrepArgs a) {
    using namespace stc;
    __shared__ float eb[Q], ec[Q];        // inverse scales of the rows of B and C
    __shared__ float dts[Q][33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x, g = blockIdx.y;
    // the sequence whose first slot is the last one at or before this slot
    int lo = 0, hi = a.n_seq, begin, end;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        seq_range(a.cu, a.n_seq, a.n_tok, mid, begin, end);
        if (first_slot(begin, mid) <= slot) lo = mid; else hi = mid;
    }
    seq_range(a.cu, a.n_seq, a.n_tok, lo, begin, end);
    const int t0 = begin + (slot - first_slot(begin, lo)) * Q;
    if (t0 < begin || t0 >= end) return;
    const int len = min(Q, end - t0);
    const int gn = a.G * N, chans = a.hp + 2 * gn;

    // ---- B and C: 8 channels x 8 consecutive tokens per thread; a row of B (or C) lies
    // in N / 8 neighbouring lanes
    constexpr int VEC = N / 8;                    // lanes of a row
    constexpr int LANES = 2 * VEC;                // threads across B | C
    constexpr int RUN = Q / (256 / LANES);        // tokens of a thread
    {
        const int v = tid % LANES, isC = v / VEC, c = (v % VEC) * 8;
        const int r0 = (tid / LANES) * RUN;
        const int ch = a.hp + isC * gn + g * N + c;
        const bf16 *src = (isC ? a.C : a.B) + g * N + c;
        const long long ld = isC ? a.ld_C : a.ld_B;
        float w[8][4], bias[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 w4 = __ldg(reinterpret_cast<const float4 *>(a.conv_w) + ch + e);
            w[e][0] = w4.x; w[e][1] = w4.y; w[e][2] = w4.z; w[e][3] = w4.w;
            bias[e] = a.conv_b ? __ldg(a.conv_b + ch + e) : 0.f;
        }
        float win[4][8];
        auto row = [&](int t, float (&x)[8]) {
            if (t >= begin && t < end) load8(src + t * ld, x);
            else if (t < begin && a.hist) load8(a.hist + ((size_t)lo * 3 + (t - begin + 3)) * chans + ch, x);
            else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
        };
#pragma unroll
        for (int j = 0; j < 3; ++j) row(t0 + r0 - 3 + j, win[j]);
        uint8_t *tile = a.tiles + ((size_t)slot * a.G + g) * (N / 64) * KB + (c / 64) * KB;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const int r = r0 + i;
            row(t0 + r, win[(3 + i) & 3]);
            float x[8];
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = bias[e];
#pragma unroll
                for (int j = 0; j < 4; ++j) s = fmaf(w[e][j], win[(i + j) & 3][e], s);
                x[e] = r < len ? ssm::silu(s) : 0.f;
                m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
            }
#pragma unroll
            for (int o = 1; o < VEC; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            float s, inv;
            scale_pow2(m, 3, s, inv);   // |B'|, |C'| < 16: scores stay below 128 x 256
            if (v % VEC == 0) (isC ? ec : eb)[r] = inv;
            uint32_t h[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float u0 = x[2 * e] * s, u1 = x[2 * e + 1] * s;
                const __half2 p = __floats2half2_rn(u0, u1);
                const float2 f = __half22float2(p);
                h[e] = *reinterpret_cast<const uint32_t *>(&p);
                l[e] = umma::pack_half2(u0 - f.x, u1 - f.y);
            }
            const int chunk = (c % 64) / 8;
            umma::st_chunk(tile + (isC ? OFF_C : 0), r, chunk, make_uint4(h[0], h[1], h[2], h[3]));
            if (!isC) umma::st_chunk(tile + OFF_LO, r, chunk, make_uint4(l[0], l[1], l[2], l[3]));
        }
    }
    // ---- the heads' records, one warp per head, two tokens per lane
    const int heads = a.H / a.G;
    for (int h0 = 0; h0 < heads; h0 += 32) {
        __syncthreads();
        const int hn = min(32, heads - h0);
        for (int i = tid; i < len * 32; i += 256) {
            const int r = i >> 5, k = i & 31;
            if (k < hn) dts[r][k] = to_f32(a.dt[(t0 + r) * a.ld_dt + g * heads + h0 + k]);
        }
        __syncthreads();
        for (int k = warp; k < hn; k += 8) {
            const int h = g * heads + h0 + k;
            const float rate = expf(__ldg(a.A + h)), bias = __ldg(a.b_dt + h);
            float d[2], la[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                d[i] = r < len ? softplus_acc(dts[r][k] + bias) : 0.f;
                la[i] = r < len ? clamp_log_decay(-rate * d[i]) : 0.f;
            }
            // prefix sums through each token, suffix sums after it (summed from the end,
            // so that the small ones, which matter, are exact to fp32)
            float pre[2] = {la[0], la[1]}, suf[2] = {la[0], la[1]};
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float p = __shfl_up_sync(0xffffffffu, pre[i], o);
                    if (lane >= o) pre[i] += p;
                    const float s = __shfl_down_sync(0xffffffffu, suf[i], o);
                    if (lane + o < 32) suf[i] += s;
                }
            }
            const float half0 = __shfl_sync(0xffffffffu, pre[0], 31), half1 = __shfl_sync(0xffffffffu, suf[1], 0);
            pre[1] += half0;
            suf[0] += half1;
            // sums after the token: the next token's inclusive suffix
            float aft0 = __shfl_down_sync(0xffffffffu, suf[0], 1), aft1 = __shfl_down_sync(0xffffffffu, suf[1], 1);
            if (lane == 31) { aft0 = half1; aft1 = 0.f; }
            const float total = __shfl_sync(0xffffffffu, suf[0], 0);
            float u[2] = {d[0] * eb[lane], d[1] * eb[lane + 32]};
            const uint32_t m = __reduce_max_sync(0xffffffffu, max(__float_as_uint(u[0]) & 0x7fffffffu,
                                                                    __float_as_uint(u[1]) & 0x7fffffffu));
            float s, inv;
            scale_pow2(m, -1, s, inv);   // u < 1
            float *rec = a.rec + ((size_t)slot * a.H + h) * REC;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                u[i] *= s;
                rec[R_L + r] = pre[i] * kLog2e;
                rec[R_U + r] = u[i];
                rec[R_W + r] = u[i] * expf(i ? aft1 : aft0);
                rec[R_YI + r] = ec[r] * expf(pre[i]);
                rec[R_YW + r] = ec[r] * inv;
            }
            if (lane == 0) {
                rec[R_DEC] = expf(total);
                rec[R_UMAX] = inv;
            }
        }
    }
}

namespace {
struct ChainArgs {
    const bf16 *x, *z, *hist;
    long long ld_x, ld_z;
    const float *conv_w, *conv_b, *D, *S0;
    const int32_t *cu;
    const uint8_t *tiles;
    const float *rec;
    bf16 *out;
    float *S_final;
    float *seg_state;   // [n_seq][blocks][n_seg - 1][N][128], then decays [n_seq][blocks][n_seg - 1][2]
    float *seg_decay;
    float *s0_copy;     // [n_seq][H][N][P] when S_final may be S0
    int n_seq, n_tok, H, G, P, blocks_per_group, seg_chunks, n_seg;
};
}  // namespace

namespace stc {
template <int N> struct Smem {
    static constexpr int TILE = (N / 64) * KB;
    static constexpr int OFF_X = 2 * TILE;             // x'' fp16, token rows x 128 columns (two 64-column blocks)
    static constexpr int OFF_XH = OFF_X + 16384;       // weighted x, hi and lo
    static constexpr int OFF_XL = OFF_XH + 16384;
    static constexpr int OFF_W = OFF_XL + 16384;       // decayed scores, 128 rows (two halves) x 64
    static constexpr int OFF_S = OFF_W + 16384;        // state fp16, N rows x 128 columns
    static constexpr int OFF_REC = OFF_S + 2 * N * 128;   // [2 stages][2 halves][REC]
    static constexpr int OFF_CW = OFF_REC + 4 * REC * 4;  // conv weights [5][128]
    static constexpr int OFF_MAX = OFF_CW + 5 * 128 * 4;  // maxima: x [16 warps][2], state [16 warps]
    static constexpr int OFF_BAR = OFF_MAX + 48 * 4;
    static constexpr int SIZE = OFF_BAR + 128 + 1024;     // barriers, TMEM slot, abort flag; alignment slack
};
static_assert(Smem<128>::SIZE <= 232448, "227 KB per block");
}  // namespace stc

// STATE_ONLY: segment k of a split sequence, from zero (segment 0: from S0) to its
// final state in seg_state.  Otherwise the whole mixer over the segment.
template <int N, bool STATE_ONLY>
__global__ void __launch_bounds__(stc::THREADS, 1) ssm_chain_kernel(const ChainArgs a) {
    using namespace stc;
    using Sm = Smem<N>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = umma::align_smem<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + Sm::OFF_BAR);
    uint64_t *bar_sc = full + 2, *bar_u = full + 3, *bar_y = full + 4;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(full + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    float *cw = reinterpret_cast<float *>(sm + Sm::OFF_CW);
    uint32_t *xmax = reinterpret_cast<uint32_t *>(sm + Sm::OFF_MAX), *smax = xmax + 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, cg = warp >> 2;
    const int blk = blockIdx.x, n = blockIdx.y, seg = blockIdx.z;
    // columns: heads h0 + half * (P == 64); the second half of a group's last block may be empty
    const int R = a.H / a.G, g = blk / a.blocks_per_group, bi = blk % a.blocks_per_group;
    const int col0 = bi * 128, gcols = R * a.P;                       // columns within the group
    const bool live1 = col0 + 64 < gcols;
    const int head0 = g * R + col0 / a.P, head1 = live1 ? g * R + (col0 + 64) / a.P : head0;
    const long long xcol = (long long)g * gcols + col0;               // first channel of the block
    const int chans = a.H * a.P + 2 * a.G * N;
    int begin, end;
    seq_range(a.cu, a.n_seq, a.n_tok, n, begin, end);
    const int all_chunks = (end - begin + Q - 1) / Q;
    const int c_lo = seg * a.seg_chunks, c_hi = min(c_lo + a.seg_chunks, all_chunks);
    const int chunks = max(0, c_hi - c_lo);
    const int last_seg = all_chunks > 0 ? (all_chunks - 1) / a.seg_chunks : 0;
    // state pass: every segment but a sequence's last; else the segments it has
    if (STATE_ONLY ? (seg >= last_seg && !(seg == 0 && a.s0_copy)) : seg > last_seg) return;
    const int slot0 = first_slot(begin, n) + c_lo;

    // ---- the state of this thread: row 32 q + lane, columns 32 cg .. + 31 of the block
    const int srow = 32 * q + lane, sc0 = 32 * cg;
    const bool owner = srow < N && (cg < 2 || live1);
    const int shead = cg < 2 ? head0 : head1;
    const int spc = a.P == 64 ? sc0 & 63 : sc0;                       // column within the head
    const size_t sbase = (((size_t)n * a.H + shead) * N + srow) * a.P + spc;
    float S[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) S[j] = 0.f;
    auto load_state = [&](const float *p) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + j);
            S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
        }
    };
    auto store_state = [&](float *p) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(p + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    };
    const size_t seg_base = ((size_t)n * gridDim.x + blk) * (a.n_seg - 1);   // of this chain's segments
    auto seg_ptr = [&](int k) { return a.seg_state + ((seg_base + k) * N + srow) * 128 + sc0; };
    if (owner) {
        if (STATE_ONLY || seg == 0) {
            if (seg == 0 && a.S0) {
                const bool copied = !STATE_ONLY && a.s0_copy;
                load_state((copied ? a.s0_copy : a.S0) + sbase);
                if (STATE_ONLY && a.s0_copy) store_state(a.s0_copy + sbase);
            }
        } else {
            // the segments before this one joined: I <- decay I + state
            load_state(seg_ptr(0));
            for (int k = 1; k < seg; ++k) {
                const float d = __ldg(a.seg_decay + (seg_base + k) * 2 + (cg >> 1));
                const float *p = seg_ptr(k);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(p + j);
                    S[j] = fmaf(d, S[j], v.x); S[j + 1] = fmaf(d, S[j + 1], v.y);
                    S[j + 2] = fmaf(d, S[j + 2], v.z); S[j + 3] = fmaf(d, S[j + 3], v.w);
                }
            }
        }
    }
    if (STATE_ONLY && seg >= last_seg) return;   // only the copy of S0 was wanted

    if (warp == 0) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) umma::mbar_init(full + i, 1);
        *abort_flag = 0;
        umma::fence_mbar_init();
    }
    for (int i = tid; i < 5 * 128; i += THREADS) {
        const int j = i >> 7, c = i & 127;
        const bool in = c < 64 || live1;
        float v = 0.f;
        if (in && j < 4) v = __ldg(a.conv_w + (xcol + c) * 4 + j);
        if (in && j == 4 && a.conv_b) v = __ldg(a.conv_b + xcol + c);
        cw[i] = v;
    }
    umma::tc_fence_before();
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tb = *tslot;
    const uint32_t T_SC = tb, T_YI = tb + 128, T_YW = tb + 256, T_U = tb + 384;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;

    auto wait = [&](uint64_t *bar, uint32_t parity) {
        for (uint32_t i = 0; i < MAX_POLLS; ++i) {
            if (umma::mbar_try_wait(bar, parity)) return;
            if ((i & 255u) == 255u && *abort_flag) return;
        }
        *abort_flag = 1;
        atomicOr(&g_ssm_err, 1u);
    };
    auto issue = [&](int c) {   // tiles and records of chunk c into stage c & 1
        const int b = c & 1;
        const size_t slot = (size_t)slot0 + c;
        umma::mbar_expect_tx(full + b, Sm::TILE + 2 * REC * 4);
        bulk_load(sm + b * Sm::TILE, a.tiles + (slot * a.G + g) * Sm::TILE, Sm::TILE, full + b);
        bulk_load(sm + Sm::OFF_REC + b * 2 * REC * 4, a.rec + (slot * a.H + head0) * REC, REC * 4, full + b);
        bulk_load(sm + Sm::OFF_REC + (b * 2 + 1) * REC * 4, a.rec + (slot * a.H + head1) * REC, REC * 4, full + b);
    };
    if (tid == 0)
        for (int c = 0; c < 2 && c < chunks; ++c) issue(c);

    // ---- raw x of this thread: tokens 4 warp .. + 3 and the three before, columns 4 lane .. + 3
    const int xc = 4 * lane, half = lane >> 4;
    const bool xlive = half == 0 || live1;
    uint2 raw[7];
    auto fetch = [&](int c) {
        const int t = begin + (c_lo + c) * Q + 4 * warp - 3;
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            raw[j] = make_uint2(0, 0);
            if (!xlive) continue;
            if (t + j >= begin) {
                if (t + j < end) raw[j] = __ldg(reinterpret_cast<const uint2 *>(a.x + (t + j) * a.ld_x + xcol + xc));
            } else if (a.hist) {
                raw[j] = __ldg(reinterpret_cast<const uint2 *>(a.hist + ((size_t)n * 3 + (t + j - begin + 3)) * chans +
                                                               xcol + xc));
            }
        }
    };
    if (chunks > 0) fetch(0);

    const float dskip0 = !STATE_ONLY && a.D ? __ldg(a.D + head0) : 0.f;
    const float dskip1 = !STATE_ONLY && a.D ? __ldg(a.D + head1) : 0.f;
    float decay0 = 1.f, decay1 = 1.f;   // of the whole segment (state pass)
    const uint32_t sX = umma::smem_u32(sm + Sm::OFF_X), sXH = umma::smem_u32(sm + Sm::OFF_XH);
    const uint32_t sXL = umma::smem_u32(sm + Sm::OFF_XL), sW = umma::smem_u32(sm + Sm::OFF_W);
    const uint32_t sS = umma::smem_u32(sm + Sm::OFF_S), sT = umma::smem_u32(sm);

    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        const uint32_t ph = (uint32_t)c & 1u, ph_full = (uint32_t)(c >> 1) & 1u;
        const int t0 = begin + (c_lo + c) * Q, len = min(Q, end - t0);
        const float *rec0 = reinterpret_cast<const float *>(sm + Sm::OFF_REC) + b * 2 * REC, *rec1 = rec0 + REC;

        // ---- convolution and activation of x
        float xh[4][4];
        uint32_t m = 0;
        {
            float4 w[5];
#pragma unroll
            for (int j = 0; j < 5; ++j) w[j] = *reinterpret_cast<const float4 *>(cw + 128 * j + xc);
            float f[7][4];
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                f[j][0] = bf16lo(raw[j].x); f[j][1] = bf16hi(raw[j].x);
                f[j][2] = bf16lo(raw[j].y); f[j][3] = bf16hi(raw[j].y);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = 4 * warp + i < len;
                const float s0 = fmaf(w[3].x, f[i + 3][0], fmaf(w[2].x, f[i + 2][0], fmaf(w[1].x, f[i + 1][0], fmaf(w[0].x, f[i][0], w[4].x))));
                const float s1 = fmaf(w[3].y, f[i + 3][1], fmaf(w[2].y, f[i + 2][1], fmaf(w[1].y, f[i + 1][1], fmaf(w[0].y, f[i][1], w[4].y))));
                const float s2 = fmaf(w[3].z, f[i + 3][2], fmaf(w[2].z, f[i + 2][2], fmaf(w[1].z, f[i + 1][2], fmaf(w[0].z, f[i][2], w[4].z))));
                const float s3 = fmaf(w[3].w, f[i + 3][3], fmaf(w[2].w, f[i + 2][3], fmaf(w[1].w, f[i + 1][3], fmaf(w[0].w, f[i][3], w[4].w))));
                xh[i][0] = in ? silu_fast(s0) : 0.f;
                xh[i][1] = in ? silu_fast(s1) : 0.f;
                xh[i][2] = in ? silu_fast(s2) : 0.f;
                xh[i][3] = in ? silu_fast(s3) : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(xh[i][e]) & 0x7fffffffu);
            }
        }
        if (c + 1 < chunks) fetch(c + 1);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((lane & 15) == 0) xmax[half * 16 + warp] = m;
        if (!STATE_ONLY) {
            uint32_t ms = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) ms = max(ms, __float_as_uint(S[j]) & 0x7fffffffu);
            ms = __reduce_max_sync(0xffffffffu, ms);
            if (lane == 0) smax[warp] = ms;       // columns of half cg / 2: warps 8 (cg / 2) .. + 7
        }
        __syncthreads();   // the previous chunk is done with the tiles, the stage of chunk c - 1 and x
        if (tid == 0 && c >= 1 && c + 1 < chunks) issue(c + 1);

        // ---- scales; operands into shared memory
        float xs, xinv, xinv0, xinv1, ss = 0.f, sinv0 = 0.f, sinv1 = 0.f;
        {
            uint32_t m0 = 0, m1 = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) { m0 = max(m0, xmax[i]); m1 = max(m1, xmax[16 + i]); }
            float s0, s1;
            scale_pow2(m0, 13, s0, xinv0);
            scale_pow2(m1, 13, s1, xinv1);
            xs = half ? s1 : s0;
            xinv = cg < 2 ? xinv0 : xinv1;        // of the state columns of this thread
            if (!STATE_ONLY) {
                m0 = m1 = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) { m0 = max(m0, smax[i]); m1 = max(m1, smax[8 + i]); }
                scale_pow2(m0, 13, s0, sinv0);
                scale_pow2(m1, 13, s1, sinv1);
                ss = cg < 2 ? s0 : s1;
            }
        }
        wait(full + b, ph_full);
        {
            const float *rw = (half ? rec1 : rec0) + R_W;
            const uint32_t off = half * 8192 + 8 * (lane & 1);
            const int chunk = (lane & 15) >> 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * warp + i;
                const uint32_t at = off + umma::sw128_offset(r, chunk);
                const float wr = rw[r];
                uint32_t hi2[2], lo2[2], x2[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u0 = xh[i][2 * e] * xs, u1 = xh[i][2 * e + 1] * xs;
                    x2[e] = umma::pack_half2(u0, u1);
                    const float v0 = u0 * wr, v1 = u1 * wr;
                    const __half2 p = __floats2half2_rn(v0, v1);
                    const float2 pf = __half22float2(p);
                    hi2[e] = *reinterpret_cast<const uint32_t *>(&p);
                    lo2[e] = umma::pack_half2(v0 - pf.x, v1 - pf.y);
                }
                if (!STATE_ONLY) *reinterpret_cast<uint2 *>(sm + Sm::OFF_X + at) = make_uint2(x2[0], x2[1]);
                *reinterpret_cast<uint2 *>(sm + Sm::OFF_XH + at) = make_uint2(hi2[0], hi2[1]);
                *reinterpret_cast<uint2 *>(sm + Sm::OFF_XL + at) = make_uint2(lo2[0], lo2[1]);
            }
            if (!STATE_ONLY && srow < N) {
                uint8_t *p = sm + Sm::OFF_S + (cg >> 1) * (N * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    umma::st_chunk(p, srow, (cg & 1) * 4 + j,
                                   make_uint4(umma::pack_half2(S[8 * j] * ss, S[8 * j + 1] * ss),
                                              umma::pack_half2(S[8 * j + 2] * ss, S[8 * j + 3] * ss),
                                              umma::pack_half2(S[8 * j + 4] * ss, S[8 * j + 5] * ss),
                                              umma::pack_half2(S[8 * j + 6] * ss, S[8 * j + 7] * ss)));
            }
        }
        umma::fence_proxy_async_smem();
        umma::tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            umma::tc_fence_after();
            const uint32_t tile = sT + b * Sm::TILE;
            constexpr int KS = N / 16;   // K steps over the state dim
            if (!STATE_ONLY) {
                const uint32_t id = umma::idesc_f16(128, 64, false, false);
#pragma unroll
                for (int j = 0; j < 2; ++j)   // scores: C in rows 64 j .. 64 j + 63
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const uint32_t kb = tile + (k / 4) * KB + (k % 4) * 32;
                        umma::mma_f16(T_SC + 64 * j, umma::sw128_desc(kb + (j ? 0 : OFF_C), 16, 1024),
                                      umma::sw128_desc(kb, 16, 1024), id, k > 0);
                    }
                umma::mma_commit(bar_sc);
            }
            {
                const uint32_t id = umma::idesc_f16(128, 128, true, true);
                constexpr uint32_t LBO = N == 128 ? KB : 0;   // N = 64: rows 64.. repeat rows 0..
                const uint32_t as[3] = {tile, tile, tile + OFF_LO}, bs[3] = {sXH, sXL, sXH};
#pragma unroll
                for (int p = 0; p < 3; ++p)
#pragma unroll
                    for (int k = 0; k < Q / 16; ++k)
                        umma::mma_f16(T_U, umma::sw128_desc(as[p] + k * 2048, LBO, 1024),
                                      umma::sw128_desc(bs[p] + k * 2048, 8192, 1024), id, p > 0 || k > 0);
                umma::mma_commit(bar_u);
            }
            if (!STATE_ONLY) {
                const uint32_t id = umma::idesc_f16(128, 64, false, true);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const uint32_t kb = tile + (k / 4) * KB + (k % 4) * 32;
                        umma::mma_f16(T_YI + 64 * j, umma::sw128_desc(kb + (j ? 0 : OFF_C), 16, 1024),
                                      umma::sw128_desc(sS + j * (N * 128) + k * 2048, 16, 1024), id, k > 0);
                    }
            }
        }
        const int hv = q >> 1, t = 32 * (q & 1) + lane;      // rows of y: half and token of this thread
        const float *recv = hv ? rec1 : rec0;
        if (!STATE_ONLY) {
            // ---- decayed scores: 16 of them per thread
            wait(bar_sc, ph);
            umma::tc_fence_after();
            uint32_t sc[16];
            umma::tmem_ld16_nowait(T_SC + lane_off + 64 * hv + 16 * cg, sc);
            umma::tmem_ld_wait();
            const float Lt = recv[R_L + t];
            float wv[16];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
                const float4 l4 = *reinterpret_cast<const float4 *>(recv + R_L + 16 * cg + 4 * s4);
                const float4 u4 = *reinterpret_cast<const float4 *>(recv + R_U + 16 * cg + 4 * s4);
                const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = 16 * cg + 4 * s4 + e;
                    wv[4 * s4 + e] = s <= t ? __uint_as_float(sc[4 * s4 + e]) * us[e] * exp2f(Lt - ls[e]) : 0.f;
                }
            }
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = umma::pack_half2(wv[2 * e], wv[2 * e + 1]);
            umma::st_chunk(sm + Sm::OFF_W, srow, 2 * cg, make_uint4(p[0], p[1], p[2], p[3]));
            umma::st_chunk(sm + Sm::OFF_W, srow, 2 * cg + 1, make_uint4(p[4], p[5], p[6], p[7]));
            umma::fence_proxy_async_smem();
            umma::tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                umma::tc_fence_after();
                const uint32_t id = umma::idesc_f16(128, 128, false, true);
#pragma unroll
                for (int k = 0; k < Q / 16; ++k)
                    umma::mma_f16(T_YW, umma::sw128_desc(sW + k * 32, 16, 1024),
                                  umma::sw128_desc(sX + k * 2048, 8192, 1024), id, k > 0);
                umma::mma_commit(bar_y);
            }
        }
        // ---- state
        wait(bar_u, ph);
        umma::tc_fence_after();
        {
            const float *rs = cg < 2 ? rec0 : rec1;
            const float dec = rs[R_DEC], add = rs[R_UMAX] * xinv;
            float v[32];
            umma::tmem_ld32(T_U + lane_off + sc0, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) S[j] = fmaf(dec, S[j], add * v[j]);
            if (STATE_ONLY) { decay0 *= rec0[R_DEC]; decay1 *= rec1[R_DEC]; }
        }
        if (!STATE_ONLY) {
            // ---- output: token t of half hv, columns 64 hv + 16 cg .. + 15
            const bool store = t < len && (hv == 0 || live1);
            const long long tok = t0 + t;
            const int oc = 64 * hv + 16 * cg;
            float zf[2][8];
            if (a.z && store) {
                load8(a.z + tok * a.ld_z + xcol + oc, zf[0]);
                load8(a.z + tok * a.ld_z + xcol + oc + 8, zf[1]);
            }
            wait(bar_y, ph);
            umma::tc_fence_after();
            uint32_t yi[16], yw[16];
            umma::tmem_ld16_nowait(T_YI + lane_off + oc, yi);
            umma::tmem_ld16_nowait(T_YW + lane_off + oc, yw);
            umma::tmem_ld_wait();
            if (store) {
                const float fi = recv[R_YI + t] * (hv ? sinv1 : sinv0), fx = hv ? xinv1 : xinv0;
                const float fw = recv[R_YW + t] * fx, fd = (hv ? dskip1 : dskip0) * fx;
                bf16 *o = a.out + tok * (long long)(a.H * a.P) + xcol + oc;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 xx = *reinterpret_cast<const uint4 *>(sm + Sm::OFF_X + hv * 8192 +
                                                                      umma::sw128_offset(t, 2 * cg + k));
                    const __half2 *x2 = reinterpret_cast<const __half2 *>(&xx);
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 xf = __half22float2(x2[e]);
                        float y0 = fmaf(__uint_as_float(yi[8 * k + 2 * e]), fi,
                                        fmaf(__uint_as_float(yw[8 * k + 2 * e]), fw, xf.x * fd));
                        float y1 = fmaf(__uint_as_float(yi[8 * k + 2 * e + 1]), fi,
                                        fmaf(__uint_as_float(yw[8 * k + 2 * e + 1]), fw, xf.y * fd));
                        if (a.z) {
                            y0 *= silu_fast(zf[k][2 * e]);
                            y1 *= silu_fast(zf[k][2 * e + 1]);
                        }
                        const __nv_bfloat162 p = __floats2bfloat162_rn(y0, y1);
                        w[e] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                    reinterpret_cast<uint4 *>(o)[k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            umma::tc_fence_before();
        }
    }
    if (owner && !*abort_flag) {
        if (STATE_ONLY) {
            store_state(seg_ptr(seg));
            if (lane == 0 && q == 0 && (cg & 1) == 0)
                a.seg_decay[(seg_base + seg) * 2 + (cg >> 1)] = cg < 2 ? decay0 : decay1;
        } else if (seg == last_seg && a.S_final) {
            store_state(a.S_final + sbase);
        }
    }
    umma::tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0)   // copies in flight land before the CTA leaves (bounded)
        for (int b = 0; b < 2 && b < chunks; ++b)
            umma::mbar_wait_bounded(full + b, (uint32_t)(((chunks - 1 - b) / 2)) & 1u, 1u << 16);
    if (warp == 0) umma::tmem_dealloc(tb, 512);
}

namespace {

size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    int blocks_per_group, blocks, slots, seg_chunks, n_seg;
    size_t tiles, rec, seg_state, seg_decay, s0_copy, bytes;
};

// Segments: a chain (128 columns of a sequence) is sequential over its chunks, so with
// fewer chains than SMs the sequence is cut and a first pass finds the segments' states.
Plan plan_for(const SsmArgs &a, int sms) {
    Plan p;
    const int R = a.H / a.G;
    p.blocks_per_group = (R * a.P + 127) / 128;
    p.blocks = a.G * p.blocks_per_group;
    p.slots = a.n_tok / stc::Q + a.n_seq;
    const long long chains = (long long)p.blocks * a.n_seq;
    const int longest = a.cu_seqlens ? a.n_tok : a.n_tok / a.n_seq;
    const int max_chunks = (longest + stc::Q - 1) / stc::Q;
    p.n_seg = 1;
    if (chains * 2 <= sms) {
        const int k = (int)(sms / chains);
        p.n_seg = max_chunks / 4 < k ? max_chunks / 4 : k;
        if (p.n_seg < 1) p.n_seg = 1;
    }
    p.seg_chunks = (max_chunks + p.n_seg - 1) / p.n_seg;
    if (p.seg_chunks < 1) p.seg_chunks = 1;
    p.n_seg = max_chunks > 0 ? (max_chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
    p.tiles = round256((size_t)p.slots * a.G * (a.N / 64) * stc::KB);
    p.rec = round256((size_t)p.slots * a.H * stc::REC * 4);
    p.seg_state = round256((size_t)chains * (p.n_seg - 1) * a.N * 128 * 4);
    p.seg_decay = round256((size_t)chains * (p.n_seg - 1) * 2 * 4);
    p.s0_copy = p.n_seg > 1 ? round256((size_t)a.n_seq * a.H * a.N * a.P * 4) : 0;
    p.bytes = p.tiles + p.rec + p.seg_state + p.seg_decay + p.s0_copy;
    return p;
}

template <int N>
cudaError_t launch_tc(const SsmArgs &a, char *ws, int sms) {
    const Plan p = plan_for(a, sms);
    PrepArgs pa = {};
    pa.B = static_cast<const bf16 *>(a.B);
    pa.C = static_cast<const bf16 *>(a.C);
    pa.dt = static_cast<const bf16 *>(a.dt);
    pa.hist = static_cast<const bf16 *>(a.hist);
    pa.ld_B = a.ld_B; pa.ld_C = a.ld_C; pa.ld_dt = a.ld_dt;
    pa.conv_w = a.conv_w; pa.conv_b = a.conv_b; pa.A = a.A; pa.b_dt = a.b_dt;
    pa.cu = a.cu_seqlens;
    pa.n_seq = a.n_seq; pa.n_tok = a.n_tok; pa.H = a.H; pa.G = a.G; pa.hp = a.H * a.P;
    pa.tiles = reinterpret_cast<uint8_t *>(ws);
    pa.rec = reinterpret_cast<float *>(ws + p.tiles);
    ChainArgs ca = {};
    ca.x = static_cast<const bf16 *>(a.x);
    ca.z = static_cast<const bf16 *>(a.z);
    ca.hist = pa.hist;
    ca.ld_x = a.ld_x; ca.ld_z = a.ld_z;
    ca.conv_w = a.conv_w; ca.conv_b = a.conv_b; ca.D = a.D; ca.S0 = a.S0;
    ca.cu = a.cu_seqlens;
    ca.tiles = pa.tiles;
    ca.rec = pa.rec;
    ca.out = static_cast<bf16 *>(a.out);
    ca.S_final = a.S_final;
    ca.seg_state = reinterpret_cast<float *>(ws + p.tiles + p.rec);
    ca.seg_decay = reinterpret_cast<float *>(ws + p.tiles + p.rec + p.seg_state);
    // segment 0 reads the initial state while the last one writes the final one
    ca.s0_copy = p.n_seg > 1 && a.S0 && a.S0 == a.S_final
                     ? reinterpret_cast<float *>(ws + p.tiles + p.rec + p.seg_state + p.seg_decay) : nullptr;
    ca.n_seq = a.n_seq; ca.n_tok = a.n_tok; ca.H = a.H; ca.G = a.G; ca.P = a.P;
    ca.blocks_per_group = p.blocks_per_group;
    ca.seg_chunks = p.seg_chunks;
    ca.n_seg = p.n_seg;
    cudaError_t e;
    if (a.n_tok > 0) {
        ssm_prep_kernel<N><<<dim3(p.slots, a.G), 256, 0, a.stream>>>(pa);
        if ((e = launched()) != cudaSuccess) return e;
    }
    constexpr int SMEM = stc::Smem<N>::SIZE;
    if ((e = cudaFuncSetAttribute(ssm_chain_kernel<N, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) !=
        cudaSuccess)
        return e;
    if (p.n_seg > 1) {
        if ((e = cudaFuncSetAttribute(ssm_chain_kernel<N, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) !=
            cudaSuccess)
            return e;
        ssm_chain_kernel<N, true><<<dim3(p.blocks, a.n_seq, p.n_seg - 1), stc::THREADS, SMEM, a.stream>>>(ca);
        if ((e = launched()) != cudaSuccess) return e;
    }
    ssm_chain_kernel<N, false><<<dim3(p.blocks, a.n_seq, p.n_seg), stc::THREADS, SMEM, a.stream>>>(ca);
    return launched();
}

}  // namespace

bool ssm_tc_supported(const SsmArgs &a) { return a.in_bf16 && a.out_bf16; }

size_t ssm_tc_workspace_bytes(const SsmArgs &a, int sms) { return plan_for(a, sms).bytes; }

cudaError_t launch_ssm_tc(const SsmArgs &a, void *ws, int sms) {
    return a.N == 128 ? launch_tc<128>(a, static_cast<char *>(ws), sms) : launch_tc<64>(a, static_cast<char *>(ws), sms);
}

// One CTA waits, through the chain's poll, for a barrier phase that nothing completes.
__global__ void ssm_wait_selftest_kernel(uint32_t max_polls) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        umma::mbar_init(&bar, 1);
        umma::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !umma::mbar_wait_bounded(&bar, 0, max_polls)) atomicOr(&g_ssm_err, 1u);
}

cudaError_t ssm_wait_selftest(uint32_t max_polls, cudaStream_t s) {
    ssm_wait_selftest_kernel<<<1, 32, 0, s>>>(max_polls);
    return cudaGetLastError();
}

cudaError_t ssm_error_word(unsigned *v, bool clear, cudaStream_t s) { return read_error_word(g_ssm_err, v, clear, s); }

}  // namespace gdn
