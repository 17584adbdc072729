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
// of B, of C and of the decayed scores is scaled by its own power of two, the weights of
// the state's x by one per chunk, x and the state by one per chunk and head, and the
// powers are multiplied back in fp32.
//
// Tokens past a sequence's end are zeros in the tiles and zeroed in x: a tile never
// holds another sequence's rows, so its NaN stays there.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <limits>

#include "ssm.cuh"
#include "umma.cuh"

namespace gdn {

__device__ unsigned int g_ssm_err;

using ssm::seq_range;

namespace stc {
constexpr int Q = 64;             // tokens per chunk
constexpr int PREP_THREADS = 512;
constexpr int MIN_SEG = 3;        // chunks of a segment
constexpr int REC = 420;          // floats of one (chunk, head) record
// record, with u = 2^eb D below 1, w and r powers of two: L log2 e [64] | u [64] | w u e^R [64] |
// 2^ec e^L [64] | 2^ec umax / r [64] | u e^{L_31 - L} of the first 32 tokens |
// L log2 e + log2 r [64] | e^L_end, its relative remainder, L_end, umax / w
constexpr int R_L = 0, R_U = 64, R_W = 128, R_YI = 192, R_YW = 256, R_UH = 320, R_LR = 352, R_END = 416;
constexpr float kLog2e = 1.44269504088896341f;
constexpr uint32_t MAX_POLLS = 1u << 24;
// 16 warps compute; one more issues the MMAs and one the copies (and two idle: registers
// move between groups of four warps, 16 x 104 + 4 x 64 of the 20 x 96 at launch)
constexpr int CWARPS = 16, MMA_WARP = 16, COPY_WARP = 17, THREADS = 32 * 20;
constexpr int COMPUTE_REGS = 104, SERVE_REGS = 64;
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

// 2^x and 1 / x on the special-function unit, 2 units in the last place each;
// subnormal results and arguments are flushed (decays below 2^-126 are nothing).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x E / (1 + E), E = e^x, of a pair with one reciprocal, 1 / a = b / (a b): the special-
// function unit (16 results a clock) is what the chain has least of.  E is kept below 2^60
// so that the product is finite, which changes nothing: there E / (1 + E) rounds to 1.  Far
// below zero E goes to 0, and x E with it (-inf: NaN, as in the formula).
__device__ __forceinline__ float2 silu2(float2 x) {
    const float2 l = fmul2(x, make_float2(stc::kLog2e, stc::kLog2e));
    const float2 e = make_float2(ex2(fminf(l.x, 60.f)), ex2(fminf(l.y, 60.f)));
    const float2 d = fadd2(e, make_float2(1.f, 1.f));
    const float r = rcp(d.x * d.y);
    return fmul2(x, fmul2(e, fmul2(make_float2(r, r), make_float2(d.y, d.x))));
}

__device__ __forceinline__ float2 half2_float2(uint32_t h) {
    __half2 p;
    *reinterpret_cast<uint32_t *>(&p) = h;
    return __half22float2(p);
}
__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint32_t pack(float2 v) { return umma::pack_half2(v.x, v.y); }
// The scales are those of the finite values: an infinity or a NaN stays what it is at any
// scale, and must not cost its neighbours theirs.  fmaxf leaves out NaN; infinities are
// rare and left out when one was met.
__device__ __forceinline__ float amax2(float m, float2 v) { return fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))); }
constexpr uint32_t kInf = 0x7f800000u;
constexpr float kNan = std::numeric_limits<float>::quiet_NaN();
__device__ __forceinline__ float finite_abs(float x) { return __float_as_uint(fabsf(x)) < kInf ? fabsf(x) : 0.f; }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Shared memory by 32-bit address: a row's chunks are one exclusive or apart.
__device__ __forceinline__ void sts64(uint32_t p, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(p), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}

template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

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
    int2 *cuts;       // [n_seq]: segments of the sequence, first of its rows
    int4 *rows;       // [cap]: sequence (-1: none), segment from 1 on, and the sequence's cut
    int slots;
    int cap, even;    // rows of segments (0: none); an even share of the chunks
};

// Chunks of the segments behind the first, which is half as long.
__device__ __forceinline__ int seg_chunks_of(int chunks, int parts) {
    return parts < 3 ? max(chunks, 1) : (2 * chunks + 2 * parts - 2) / (2 * parts - 1);
}

// Which sequences are cut, by one block: those of more than 1.6 even shares, into one
// segment and as many more as their part of the rows, of MIN_SEG chunks at least; none of
// them where the longest of the first launch and of the second together are no shorter.
__device__ void cut_sequences(const PrepArgs &a) {
    constexpr int WARPS = stc::PREP_THREADS / 32;
    __shared__ int sums[5][WARPS];
    const int n = threadIdx.x, lane = n & 31, warp = n >> 5;
    int chunks = 0;
    if (n < a.n_seq) {
        int begin, end;
        ssm::seq_range(a.cu, a.n_seq, a.n_tok, n, begin, end);
        chunks = (end - begin + stc::Q - 1) / stc::Q;
    }
    const bool is_long = 5LL * chunks > 8LL * a.even;
    const int part = __reduce_add_sync(0xffffffffu, is_long ? chunks : 0);
    if (lane == 0) sums[0][warp] = part;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < WARPS; ++w) all += sums[0][w];
    int more = is_long ? (int)min((long long)a.cap * chunks / all, (long long)chunks / stc::MIN_SEG - 1) : 0;
    if (more < 2) more = 0;   // two segments would run one after the other
    // longest whole, of the first launch (a state's chunk takes half as long) and of the second
    const int s = seg_chunks_of(chunks, 1 + more), first = more ? (s + 1) / 2 : chunks;
    const int l = __reduce_max_sync(0xffffffffu, chunks), f = __reduce_max_sync(0xffffffffu, max(first, more ? (s * 17) / 32 : 0));
    const int r2 = __reduce_max_sync(0xffffffffu, more ? s : 0);
    if (lane == 0) {
        sums[1][warp] = l;
        sums[2][warp] = f;
        sums[3][warp] = r2;
    }
    __syncthreads();
    int whole = 0, one = 0, two = 0;
    for (int w = 0; w < WARPS; ++w) {
        whole = max(whole, sums[1][w]);
        one = max(one, sums[2][w]);
        two = max(two, sums[3][w]);
    }
    if (one + two + 2 >= whole) more = 0;
    int upto = more;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[4][warp] = upto;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) upto += sums[4][w];
        total += sums[4][w];
    }
    if (n < a.n_seq) a.cuts[n] = make_int2(1 + more, upto - more);
    for (int k = 0; k < more; ++k) a.rows[upto - more + k] = make_int4(n, 1 + k, 1 + more, upto - more);
    for (int r = total + n; r < a.cap; r += stc::PREP_THREADS) a.rows[r] = make_int4(-1, 0, 0, 0);
}

}  // namespace

// One CTA per (slot, group).
template <int N>
__global__ void __launch_bounds__(stc::PREP_THREADS, 2) ssm_prep_kernel(const PrepArgs a) {
    using namespace stc;
    __shared__ float eb[Q], ec[Q];        // inverse scales of the rows of B and C
    __shared__ float dts[Q][33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x, g = blockIdx.y;
    if (slot == a.slots) {   // one more block
        if (g == 0) cut_sequences(a);
        return;
    }
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

    // ---- B and C: 4 channels x RUN consecutive tokens per thread; a row of B (or C) lies in
    // N / 4 neighbouring lanes.  Few registers, so that two CTAs hide each other's latency.
    constexpr int VEC = N / 4;                    // lanes of a row
    constexpr int LANES = 2 * VEC;                // threads across B | C
    constexpr int RUN = Q / (PREP_THREADS / LANES);   // tokens of a thread
    {
        const int v = tid % LANES, isC = v / VEC, c = (v % VEC) * 4;
        const int r0 = (tid / LANES) * RUN;
        const int ch = a.hp + isC * gn + g * N + c;
        const bf16 *src = (isC ? a.C : a.B) + g * N + c;
        const long long ld = isC ? a.ld_C : a.ld_B;
        float2 w[4][2], bias[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // [tap][channel pair]
        {
            float4 w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w4[e] = __ldg(reinterpret_cast<const float4 *>(a.conv_w) + ch + e);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[0][e] = make_float2(w4[2 * e].x, w4[2 * e + 1].x);
                w[1][e] = make_float2(w4[2 * e].y, w4[2 * e + 1].y);
                w[2][e] = make_float2(w4[2 * e].z, w4[2 * e + 1].z);
                w[3][e] = make_float2(w4[2 * e].w, w4[2 * e + 1].w);
            }
            if (a.conv_b) {
                const float4 b4 = __ldg(reinterpret_cast<const float4 *>(a.conv_b + ch));
                bias[0] = make_float2(b4.x, b4.y);
                bias[1] = make_float2(b4.z, b4.w);
            }
        }
        auto row = [&](int t) -> uint2 {
            if (t >= begin && t < end) return __ldg(reinterpret_cast<const uint2 *>(src + t * ld));
            if (t < begin && a.hist)
                return __ldg(reinterpret_cast<const uint2 *>(a.hist + ((size_t)lo * 3 + (t - begin + 3)) * chans + ch));
            return make_uint2(0, 0);
        };
        uint2 raw[RUN + 3];
#pragma unroll
        for (int j = 0; j < RUN + 3; ++j) raw[j] = row(t0 + r0 - 3 + j);
        uint8_t *tile = a.tiles + ((size_t)slot * a.G + g) * (N / 64) * KB + (c / 64) * KB + (isC ? OFF_C : 0);
        const uint32_t sub = 8 * ((c / 4) & 1);
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const int r = r0 + i;
            float2 x[2];
            float mf = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 s = bias[e];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = e ? raw[i + j].y : raw[i + j].x;
                    s = ffma2(w[j][e], make_float2(bf16lo(u), bf16hi(u)), s);
                }
                s = silu2(s);
                x[e] = r < len ? s : make_float2(0.f, 0.f);
                mf = fmaxf(mf, fmaxf(finite_abs(x[e].x), finite_abs(x[e].y)));
            }
            uint32_t m = __float_as_uint(mf);
            if constexpr (VEC == 32) m = __reduce_max_sync(0xffffffffu, m);
            else {
#pragma unroll
                for (int o = 1; o < VEC; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            float s, inv;
            // B' < 2^14: its pairs keep 22 bits of an element down to 2^-15 of the row's largest;
            // C' < 16: scores stay below 128 x 2^18
            scale_pow2(m, isC ? 3 : 13, s, inv);
            if (v % VEC == 0) (isC ? ec : eb)[r] = inv;
            uint2 hi, lo2;
            const float2 u0 = fmul2(x[0], make_float2(s, s)), u1 = fmul2(x[1], make_float2(s, s));
            hi.x = pack(u0);
            hi.y = pack(u1);
            uint8_t *p = tile + umma::sw128_offset(r, (c % 64) / 8) + sub;
            *reinterpret_cast<uint2 *>(p) = hi;
            if (!isC) {
                const float2 h0 = half2_float2(hi.x), h1 = half2_float2(hi.y);
                lo2.x = umma::pack_half2(u0.x - h0.x, u0.y - h0.y);
                lo2.y = umma::pack_half2(u1.x - h1.x, u1.y - h1.y);
                *reinterpret_cast<uint2 *>(p + OFF_LO) = lo2;
            }
        }
    }
    // ---- the heads' records, one warp per head, two tokens per lane
    const int heads = a.H / a.G;
    for (int h0 = 0; h0 < heads; h0 += 32) {
        __syncthreads();
        const int hn = min(32, heads - h0);
        for (int i = tid; i < len * 32; i += PREP_THREADS) {
            const int r = i >> 5, k = i & 31;
            if (k < hn) dts[r][k] = to_f32(a.dt[(t0 + r) * a.ld_dt + g * heads + h0 + k]);
        }
        __syncthreads();
        for (int k = warp; k < hn; k += PREP_THREADS / 32) {
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
            const float suf0 = suf[0];   // from the token to the end of the first half
            pre[1] += half0;
            suf[0] += half1;
            // sums after the token: the next token's inclusive suffix
            float aft0 = __shfl_down_sync(0xffffffffu, suf[0], 1), aft1 = __shfl_down_sync(0xffffffffu, suf[1], 1);
            if (lane == 31) { aft0 = half1; aft1 = 0.f; }
            const float total = __shfl_sync(0xffffffffu, suf[0], 0);
            float u[2] = {d[0] * eb[lane], d[1] * eb[lane + 32]};
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(finite_abs(u[0]), finite_abs(u[1]))));
            float s, inv;
            scale_pow2(m, -1, s, inv);   // u < 1
            float w[2];
            int lr[2];   // log2 u - L, rounded up
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u[i] *= s;
                w[i] = u[i] * expf(i ? aft1 : aft0);
                pre[i] *= kLog2e;
                lr[i] = max(__float2int_ru(__log2f(finite_abs(u[i])) - pre[i]), -30000);
            }
            // Row t of the decayed scores is made of u_s e^{L_t - L_s}; its own power of two r
            // brings the largest of them, 2^{L_t + max_{s <= t} (log2 u_s - L_s)}, to 2^-12 ..
            // 2^-10, so that a score times it is below 2^15 (r at most 2^100: what is smaller
            // than that against the chunk's u is nothing).
            // The maxima of both halves side by side in one word, |L| < 12000.
            uint32_t top = __byte_perm(lr[0], lr[1], 0x5410);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t p = __shfl_up_sync(0xffffffffu, top, o);
                if (lane >= o) top = __vmaxs2(top, p);
            }
            lr[0] = (short)(top & 0xffff);
            lr[1] = max((short)(top >> 16), (short)(__shfl_sync(0xffffffffu, top, 31) & 0xffff));
            // The state's operands: the largest u e^R to 1/2 .. 1, whatever u was before a decay.
            const uint32_t mw = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(finite_abs(w[0]), finite_abs(w[1]))));
            float sw, invw;
            scale_pow2(mw, -1, sw, invw);
            float *rec = a.rec + ((size_t)slot * a.H + h) * REC;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                const float k = fminf(-10.f - ceilf(pre[i] + lr[i]), 100.f);
                rec[R_L + r] = pre[i];
                rec[R_U + r] = u[i];
                rec[R_W + r] = w[i] * sw;
                rec[R_YI + r] = ec[r] * exp2f(pre[i]);
                rec[R_YW + r] = ec[r] * inv * __uint_as_float((uint32_t)(127 - (int)k) << 23);
                rec[R_LR + r] = pre[i] + k;
            }
            // e^{L_31 - L_s}, the sum after s inside the first half
            const float in_half = __shfl_down_sync(0xffffffffu, suf0, 1);
            rec[R_UH + lane] = u[0] * expf(lane == 31 ? 0.f : in_half);
            if (lane == 0) {
                const float2 a = ssm::decay_pair(-total);
                *reinterpret_cast<float4 *>(rec + R_END) = make_float4(a.x, ssm::relative_rest(a), total, inv * invw);
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
    float *seg_state;   // [cap][blocks][N][128]: of segment k of a sequence in row first + k
    float *seg_decay;   // [cap][blocks][2]: log
    const int2 *cuts;   // as in PrepArgs
    const int4 *rows;
    int n_seq, n_tok, H, G, P, blocks_per_group;
    int cap;            // rows of segments; 0: no sequence is cut
};
struct ChainMaps {
    CUtensorMap z, out;   // [N_tok][H P], boxes of 64 columns x 64 tokens
};
}  // namespace

namespace stc {
template <int N> struct Smem {
    static constexpr int TILE = (N / 64) * KB;
    static constexpr int OFF_X = 2 * TILE;             // x'' fp16, token rows x 128 columns (two 64-column blocks)
    static constexpr int OFF_XH = OFF_X + 16384;       // weighted x, hi and lo
    static constexpr int OFF_XL = OFF_XH + 16384;
    static constexpr int OFF_S = OFF_XL + 16384;       // state fp16, N rows x 128 columns
    static constexpr int OFF_Z = OFF_S + 2 * N * 128;  // [2 stages]: z, then out in its place, 64 rows x 128 columns
    static constexpr int OFF_REC = OFF_Z + 2 * 16384;  // [2 stages][2 halves][REC]
    static constexpr int OFF_CW = OFF_REC + 4 * REC * 4;  // conv weights [5][128]
    static constexpr int OFF_MAX = OFF_CW + 5 * 128 * 4;  // bits of the largest |.|, [3 chunks][x, x, state, state]
    static constexpr int OFF_ODD = OFF_MAX + 12 * 4;      // per column the first token whose x is not finite; any
    static constexpr int OFF_BAR = OFF_ODD + 132 * 4;
    static constexpr int SIZE = OFF_BAR + 128 + 1024;     // barriers, TMEM slot, abort flag; alignment slack
};
static_assert(Smem<128>::SIZE <= 232448, "227 KB per block");
}  // namespace stc

// One CTA per 128 columns of a sequence's segment.  STATE_ONLY: only the state, from zero,
// into seg_state with the sum of its log-decays.  Otherwise the whole mixer over the
// segment.
template <int N, bool STATE_ONLY>
__device__ __forceinline__ void chain_segment(const ChainArgs &a, const ChainMaps &maps, const int n, const int seg,
                                              const int2 cut) {
    using namespace stc;
    using Sm = Smem<N>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = umma::align_smem<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + Sm::OFF_BAR);
    uint64_t *bar_sc = full + 2, *bar_u = full + 3, *bar_y = full + 4, *full_z = full + 5;
    uint64_t *bar_x = full + 7, *bar_w = full + 8;   // the computing warps' operands, and decayed scores, are there
    uint64_t *bar_m = full + 9;   // a chunk's meeting
    uint32_t *tslot = reinterpret_cast<uint32_t *>(full + 10);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    float *cw = reinterpret_cast<float *>(sm + Sm::OFF_CW);
    uint32_t *mx = reinterpret_cast<uint32_t *>(sm + Sm::OFF_MAX);
    int *odd = reinterpret_cast<int *>(sm + Sm::OFF_ODD);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, cg = warp >> 2;
    const int blk = blockIdx.x;
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
    const int seg_chunks = seg_chunks_of(all_chunks, cut.x), first = cut.x < 3 ? seg_chunks : (seg_chunks + 1) / 2;
    const int c_lo = seg == 0 ? 0 : first + (seg - 1) * seg_chunks;
    const int c_hi = min(seg == 0 ? first : c_lo + seg_chunks, all_chunks);
    const int chunks = max(0, c_hi - c_lo);
    const int last_seg = all_chunks > first ? (all_chunks - first - 1) / seg_chunks + 1 : 0;
    if (STATE_ONLY ? seg >= last_seg : seg > last_seg) return;   // a last segment's state has no reader
    const int slot0 = first_slot(begin, n) + c_lo;

    // ---- the state of a computing thread: row 32 q + lane, columns 32 cg .. + 31 of the block
    const bool computes = warp < CWARPS;
    const int srow = 32 * q + lane, sc0 = 32 * (cg & 3);
    const bool owner = computes && srow < N && (cg < 2 || live1);
    const int shead = cg < 2 ? head0 : head1;
    const int spc = a.P == 64 ? sc0 & 63 : sc0;                       // column within the head
    const size_t sbase = (((size_t)n * a.H + shead) * N + srow) * a.P + spc;
    auto seg_at = [&](int k) { return (size_t)(cut.y + k) * gridDim.x + blk; };
    auto seg_ptr = [&](int k) { return a.seg_state + (seg_at(k) * N + srow) * 128 + sc0; };

    if (warp == MMA_WARP) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < 10; ++i) umma::mbar_init(full + i, i < 7 ? 1 : i < 9 || STATE_ONLY ? CWARPS : CWARPS + 1);
        *abort_flag = 0;
        umma::fence_mbar_init();
    }
    if (tid < 12) mx[tid] = 0;
    if (tid <= 128) odd[tid] = tid < 128 ? INT_MAX : 0;
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
    const uint32_t sT = umma::smem_u32(sm);

    // A wait that expires raises the abort flag: later ones give up soon after, no more
    // copies are started, and the state is not stored.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        for (uint32_t i = 0; i < MAX_POLLS; ++i) {
            if (umma::mbar_try_wait(bar, parity)) return;
            if ((i & 255u) == 255u && *abort_flag) return;
        }
        *abort_flag = 1;
        atomicOr(&g_ssm_err, 1u);
    };
    // Once a chunk the computing warps and the copying one meet: the previous chunk is done
    // with shared memory, and the maxima are there.  A warp arrives when its own part is,
    // and waits where it needs the others'.
    auto arrive = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_m);
    };

    if (!computes) {
        regs_dec<SERVE_REGS>();
        if (warp == MMA_WARP) {
            // ------------------------------------------------------------ MMA issuer
            // The tensor pipe takes MMAs about as fast as it runs them, so their issuer
            // waits along; it has nothing else to do.
            const uint64_t d_tile = umma::sw128_desc(sT, 16, 1024);
            const uint64_t d_tile_mn = umma::sw128_desc(sT, N == 128 ? KB : 0, 1024);   // N = 64: rows 64.. repeat 0..
            const uint64_t d_x = umma::sw128_desc(sT + Sm::OFF_X, 8192, 1024);
            const uint64_t d_s = umma::sw128_desc(sT + Sm::OFF_S, 16, 1024);
            constexpr int KS = N / 16;   // K steps over the state dim
            auto scores = [&](int c) {   // C in rows 64 j .. 64 j + 63
                const uint64_t dt = d_tile + (uint32_t)((c & 1) * (Sm::TILE >> 4));
                wait(full + (c & 1), (uint32_t)(c >> 1) & 1u);
                __syncwarp();
                if (elect_one()) {
                    constexpr uint32_t id = umma::idesc_f16(128, 64, false, false);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const uint32_t kb = ((k / 4) * KB + (k % 4) * 32) >> 4;
                            umma::mma_f16(T_SC + 64 * j, dt + (kb + (j ? 0 : OFF_C >> 4)), dt + kb, id, k > 0);
                        }
                    umma::mma_commit(bar_sc);
                }
                __syncwarp();
            };
            if (!STATE_ONLY && chunks > 0) scores(0);
            for (int c = 0; c < chunks; ++c) {
                const uint32_t st = (uint32_t)((c & 1) * (Sm::TILE >> 4));
                // the states' chunks alternate between two buffers
                const int second = STATE_ONLY ? c & 1 : 0;
                wait(second ? bar_w : bar_x, (uint32_t)(STATE_ONLY ? c >> 1 : c) & 1u);
                __syncwarp();
                umma::tc_fence_after();
                if (elect_one()) {
                    constexpr uint32_t idu = umma::idesc_f16(128, 128, true, true);
                    const uint64_t da = d_tile_mn + st;
                    const uint64_t dxh = d_x + (((second ? Sm::OFF_Z : Sm::OFF_XH) - Sm::OFF_X) >> 4), dxl = dxh + (16384 >> 4);
#pragma unroll
                    for (int p = 0; p < 3; ++p)   // hi hi, hi lo, lo hi
#pragma unroll
                        for (int k = 0; k < Q / 16; ++k)
                            umma::mma_f16(second ? T_YW : T_U, da + (((p == 2 ? OFF_LO : 0) + k * 2048) >> 4),
                                          (p == 1 ? dxl : dxh) + ((k * 2048) >> 4), idu, p > 0 || k > 0);
                    umma::mma_commit(second ? bar_y : bar_u);
                    if (!STATE_ONLY) {
                        constexpr uint32_t id = umma::idesc_f16(128, 64, false, true);
                        const uint64_t dt = d_tile + st;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int k = 0; k < KS; ++k) {
                                const uint32_t kb = ((k / 4) * KB + (k % 4) * 32) >> 4;
                                umma::mma_f16(T_YI + 64 * j, dt + (kb + (j ? 0 : OFF_C >> 4)),
                                              d_s + ((j * (N * 128) + k * 2048) >> 4), id, k > 0);
                            }
                    }
                }
                __syncwarp();
                if (!STATE_ONLY) {
                    wait(bar_w, (uint32_t)c & 1u);
                    __syncwarp();
                    umma::tc_fence_after();
                    if (elect_one()) {
                        constexpr uint32_t id = umma::idesc_f16(128, 64, false, true);
#pragma unroll
                        for (int j = 0; j < 2; ++j)   // rows 64 j .. of the decayed scores, columns of half j
#pragma unroll
                            for (int k = 0; k < Q / 16; ++k)
                                umma::mma_f16_ts(T_YW + 64 * j, T_SC + (j ? 0 : 64) + 8 * k,
                                                 d_x + ((j * 8192 + k * 2048) >> 4), id, k > 0);
                        umma::mma_commit(bar_y);
                    }
                    __syncwarp();
                }
                if (!STATE_ONLY && c + 1 < chunks) {
                    wait(bar_y, (uint32_t)c & 1u);   // the decayed scores are used up
                    umma::tc_fence_after();
                    scores(c + 1);
                }
            }
        } else if (warp == COPY_WARP) {
            // ---------------------------------------------------------------- copies
            const uint8_t *tile = a.tiles + ((size_t)slot0 * a.G + g) * Sm::TILE;
            const float *rec = a.rec + ((size_t)slot0 * a.H + head0) * REC;
            const size_t tile_step = (size_t)a.G * Sm::TILE, rec_step = (size_t)a.H * REC;
            auto issue = [&](int c) {   // tiles and records of chunk c, in turn, into stage c & 1
                uint64_t *bar = full + (c & 1);
                uint8_t *r = sm + Sm::OFF_REC + (c & 1) * 2 * REC * 4;
                umma::mbar_expect_tx(bar, Sm::TILE + 2 * REC * 4);
                bulk_load(sm + (c & 1) * Sm::TILE, tile, Sm::TILE, bar);
                bulk_load(r, rec, REC * 4, bar);
                bulk_load(r + REC * 4, rec + (head1 - head0) * REC, REC * 4, bar);
                tile += tile_step;
                rec += rec_step;
            };
            auto issue_z = [&](int c) {
                uint8_t *p = sm + Sm::OFF_Z + (c & 1) * 16384;
                const int t = begin + (c_lo + c) * Q;
                umma::mbar_expect_tx(full_z + (c & 1), live1 ? 16384 : 8192);
                umma::tma_load_3d(p, &maps.z, (int)xcol, 0, t, full_z + (c & 1));
                if (live1) umma::tma_load_3d(p + 8192, &maps.z, (int)xcol + 64, 0, t, full_z + (c & 1));
            };
            auto store_out = [&](int c) {
                const uint8_t *p = sm + Sm::OFF_Z + (c & 1) * 16384;
                const int t = begin + (c_lo + c) * Q;
                umma::tma_store_3d(&maps.out, (int)xcol, 0, t, p);
                if (live1) umma::tma_store_3d(&maps.out, (int)xcol + 64, 0, t, p + 8192);
                umma::bulk_commit();
            };
            const bool one = elect_one();
            if (one && chunks > 0) {
                issue(0);
                if (!STATE_ONLY && a.z) issue_z(0);
                if (chunks > 1) {
                    issue(1);
                    if (!STATE_ONLY && a.z) issue_z(1);
                }
            }
            // chunk c's products, which follow its records' last reader, have read its tile
            for (int c = 0; STATE_ONLY && c + 2 < chunks; ++c) {
                wait(c & 1 ? bar_y : bar_u, (uint32_t)(c >> 1) & 1u);
                if (one && *abort_flag == 0) issue(c + 2);
                __syncwarp();
            }
            float carry = 0.f;   // of this lane's half
            for (int c = 0; !STATE_ONLY && c < chunks; ++c) {
                if (c >= 1) wait(bar_y, (uint32_t)(c - 1) & 1u);
                // the decays that the state takes, in place, before the meeting: this warp has time
                wait(full + (c & 1), (uint32_t)(c >> 1) & 1u);
                if (lane < 2) {
                    float *e = reinterpret_cast<float *>(sm + Sm::OFF_REC) + ((c & 1) * 2 + lane) * REC + R_END;
                    carry += e[1];
                    e[0] = ssm::next_decay(e[0], carry);
                    umma::fence_proxy_async_smem();   // before the stage is loaded again
                }
                arrive();
                wait(bar_m, (uint32_t)c & 1u);
                if (one) {
                    const bool go = *abort_flag == 0;
                    if (c >= 1 && c + 1 < chunks && go) issue(c + 1);
                    if (c >= 2) {
                        // out of chunk c - 2, gated before this meeting, leaves; its tile takes z of chunk c
                        store_out(c - 2);
                        umma::bulk_wait_read<0>();
                        if (a.z && go) issue_z(c);
                    }
                }
                __syncwarp();
            }
            if (!STATE_ONLY && chunks > 0) {
                arrive();
                wait(bar_m, (uint32_t)chunks & 1u);
                if (one) {   // the last two tiles (the last only if it is whole); the copies end before the CTA does
                    if (chunks > 1) store_out(chunks - 2);
                    if (begin + (c_lo + chunks) * Q <= end) store_out(chunks - 1);
                    umma::bulk_wait_all();
                }
                __syncwarp();
            }
            // after an abort, copies in flight land before the CTA leaves (bounded)
            if (one && *abort_flag)
                for (int b = 0; b < 2 && b < chunks; ++b) {
                    umma::mbar_wait_bounded(full + b, (uint32_t)((chunks - 1 - b) / 2) & 1u, 1u << 16);
                    if (!STATE_ONLY && a.z)
                        umma::mbar_wait_bounded(full_z + b, (uint32_t)((chunks - 1 - b) / 2) & 1u, 1u << 16);
                }
        }
    } else {
        regs_inc<COMPUTE_REGS>();
        const uint32_t lane_off = (uint32_t)(32 * q) << 16;
        float2 S[16];
        float carry = 0.f;   // of the decays that join segments, or of a states' pass
#pragma unroll
        for (int j = 0; j < 16; ++j) S[j] = make_float2(0.f, 0.f);
        if (owner) {
            // the initial state, or the segments before this one joined: I <- decay I + state
            const bool joined = !STATE_ONLY && seg > 0;
            const float *p = joined ? seg_ptr(0) : seg > 0 || !a.S0 ? nullptr : a.S0 + sbase;
            for (int k = 0; p && k < (joined ? seg : 1); ++k) {
                if (k > 0) p = seg_ptr(k);
                float d = 0.f;
                if (k > 0) {
                    const float2 e = ssm::decay_pair(-__ldg(a.seg_decay + seg_at(k) * 2 + (cg >> 1)));
                    carry += ssm::relative_rest(e);
                    d = ssm::next_decay(e.x, carry);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(p + 2 * j);
                    S[j] = ffma2(make_float2(d, d), S[j], make_float2(v.x, v.y));
                    S[j + 1] = ffma2(make_float2(d, d), S[j + 1], make_float2(v.z, v.w));
                }
            }
        }

        // ---- raw x of this thread: tokens 4 warp .. + 3 and the three before, columns 4 lane .. + 3
        const int xc = 4 * lane, half = lane >> 4;
        const bool xlive = half == 0 || live1;
        uint2 raw[7];
        auto fetch = [&](int c) {
            const int t = begin + (c_lo + c) * Q + 4 * warp - 3;
            const bf16 *p = a.x + t * a.ld_x + xcol + xc;
            if (t >= begin && t + 7 <= end && live1) {
#pragma unroll
                for (int j = 0; j < 7; ++j) raw[j] = __ldg(reinterpret_cast<const uint2 *>(p + j * a.ld_x));
                return;
            }
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                raw[j] = make_uint2(0, 0);
                if (!xlive) continue;
                if (t + j >= begin) {
                    if (t + j < end) raw[j] = __ldg(reinterpret_cast<const uint2 *>(p + j * a.ld_x));
                } else if (a.hist) {
                    raw[j] = __ldg(reinterpret_cast<const uint2 *>(
                        a.hist + ((size_t)n * 3 + (t + j - begin + 3)) * chans + xcol + xc));
                }
            }
        };
        // convolution and activation of the fetched tokens of chunk c, and the largest |x| of
        // each half into m3[half]
        float2 xh[4][2];
        auto convolve = [&](int c, uint32_t *m3) {
            const int len = min(Q, end - (begin + (c_lo + c) * Q));
            float2 w[5][2], f[7][2];
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(cw + 128 * j + xc);
                w[j][0] = make_float2(v.x, v.y);
                w[j][1] = make_float2(v.z, v.w);
            }
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                f[j][0] = make_float2(bf16lo(raw[j].x), bf16hi(raw[j].x));
                f[j][1] = make_float2(bf16lo(raw[j].y), bf16hi(raw[j].y));
            }
            float m = 0.f;
            float2 chk = make_float2(0.f, 0.f);   // stays 0 while all are finite
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = 4 * warp + i < len;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float2 v = w[4][e];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v = ffma2(w[j][e], f[i + j][e], v);
                    v = silu2(v);
                    xh[i][e] = in ? v : make_float2(0.f, 0.f);
                    m = amax2(m, xh[i][e]);
                    chk = ffma2(xh[i][e], make_float2(0.f, 0.f), chk);
                }
            }
            if (__any_sync(0xffffffffu, chk.x + chk.y != 0.f)) {
                // A product's zero for a token before it would make NaN of such a value, so
                // it is left out here, and its column written over behind the last chunk.
                m = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &v = e & 1 ? xh[i][e >> 1].y : xh[i][e >> 1].x;
                        if (!(fabsf(v) <= FLT_MAX)) {
                            v = 0.f;
                            atomicMin(odd + xc + e, (c_lo + c) * Q + 4 * warp + i);
                            odd[128] = 1;
                        }
                        m = fmaxf(m, fabsf(v));
                    }
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((lane & 15) == 0) atomicMax(m3 + half, __float_as_uint(m));
        };

        const float dskip = !STATE_ONLY && a.D ? __ldg(a.D + (q < 2 ? head0 : head1)) : 0.f;
        float log_hi = 0.f, log_lo = 0.f;   // sum of the segment's log-decays (state pass)
        // operand addresses of this thread: a row's 16-byte chunks k, k ^ 1, ... differ by an
        // exclusive or with the chunk's bits
        const uint32_t p_x = sT + Sm::OFF_X + half * 8192 + umma::sw128_offset(4 * warp, (lane & 15) >> 1) + 8 * (lane & 1);
        const uint32_t p_s = sT + Sm::OFF_S + (cg >> 1) * (N * 128) + umma::sw128_offset(srow, (cg & 1) * 4);
        const int hv = q >> 1, t = 32 * (q & 1) + lane;      // rows of y: half and token of this thread
        const int oc = 64 * hv + 16 * cg;                    // and its 16 columns
        const uint32_t p_o = sT + Sm::OFF_X + hv * 8192 + umma::sw128_offset(t, 2 * cg);

        if (chunks > 0) {
            fetch(0);
            convolve(0, mx);
        }
        auto state_max = [&](uint32_t *m3) {
            float ms = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) ms = amax2(ms, S[j]);
            uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(ms));
            if (mb >= kInf) {
                ms = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) ms = fmaxf(ms, fmaxf(finite_abs(S[j].x), finite_abs(S[j].y)));
                mb = __reduce_max_sync(0xffffffffu, __float_as_uint(ms));
            }
            if (lane == 0) atomicMax(m3 + 2 + (cg >> 1), mb);
        };
        if (!STATE_ONLY) state_max(mx);
        // y of this thread (token t of half hv, columns oc .. + 15) of chunk c through the gate:
        // a whole chunk into the tile that z came in, from where it leaves by TMA, a ragged one
        // straight out
        float2 y[8];
        auto gate = [&](int c) {
            const int t0 = begin + (c_lo + c) * Q, len = min(Q, end - t0);
            const uint32_t p_z = p_o + (Sm::OFF_Z - Sm::OFF_X) + (c & 1) * 16384;
            if (a.z) {
                wait(full_z + (c & 1), (uint32_t)(c >> 1) & 1u);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 zz = lds128(p_z ^ (16 * k));
                    const uint32_t zw[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[4 * k + e] = fmul2(y[4 * k + e], silu2(make_float2(bf16lo(zw[e]), bf16hi(zw[e]))));
                }
            }
            uint4 w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                w[k] = make_uint4(pack_bf16(y[4 * k]), pack_bf16(y[4 * k + 1]), pack_bf16(y[4 * k + 2]), pack_bf16(y[4 * k + 3]));
            if (len == Q) {
                sts128(p_z, w[0]);
                sts128(p_z ^ 16, w[1]);
                umma::fence_proxy_async_smem();
            } else if (t < len && (hv == 0 || live1)) {
                uint4 *o = reinterpret_cast<uint4 *>(a.out + (long long)(t0 + t) * (a.H * a.P) + xcol + oc);
                o[0] = w[0];
                o[1] = w[1];
            }
        };
        // operands of the x in xh, weighted by their records' R_W, in shared memory; the plain
        // one for y only
        auto store_x = [&](const float *w, float xs, uint32_t to) {
            const float4 wr4 = *reinterpret_cast<const float4 *>(w + R_W + 4 * warp);
            const float wr[4] = {wr4.x, wr4.y, wr4.z, wr4.w};
            const float2 xs2 = make_float2(xs, xs);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = (p_x ^ (16 * i)) + 128 * i;
                uint32_t x2[2], hi2[2], lo2[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 u = fmul2(xh[i][e], xs2), v = fmul2(u, make_float2(wr[i], wr[i]));
                    x2[e] = pack(u);
                    hi2[e] = pack(v);
                    const float2 h = half2_float2(hi2[e]);
                    lo2[e] = umma::pack_half2(v.x - h.x, v.y - h.y);
                }
                if (!STATE_ONLY) sts64(p, x2[0], x2[1]);
                sts64(p + to, hi2[0], hi2[1]);
                sts64(p + to + 16384, lo2[0], lo2[1]);
            }
        };
        if constexpr (STATE_ONLY) {
            // A chunk's products run under the next one's convolution and stores: the
            // operands (in z's place) and the sums (in y's) alternate between two buffers.
            float dec = 0.f, add = 0.f;   // of this thread's half, of the last chunk stored
            auto store = [&](int c) {
                const float *r = reinterpret_cast<const float *>(sm + Sm::OFF_REC) + (c & 1) * 2 * REC;
                wait(bar_m, (uint32_t)c & 1u);
                const uint2 m = *reinterpret_cast<const uint2 *>(mx + 4 * (c % 3));
                if (tid < 2) mx[4 * ((c + 2) % 3) + tid] = 0;   // chunk c - 1's, which all have read
                float xs0, xs1, i0, i1;
                scale_pow2(m.x, 13, xs0, i0);
                scale_pow2(m.y, 13, xs1, i1);
                wait(full + (c & 1), (uint32_t)(c >> 1) & 1u);
                store_x(half ? r + REC : r, half ? xs1 : xs0, (c & 1 ? Sm::OFF_Z : Sm::OFF_XH) - Sm::OFF_X);
                const float4 e = *reinterpret_cast<const float4 *>((cg < 2 ? r : r + REC) + R_END);
                carry += e.y;
                dec = ssm::next_decay(e.x, carry);
                add = e.w * (cg < 2 ? i0 : i1);
                const float sum = log_hi + e.z;   // two sums, since equal addends are rounded alike
                log_lo += e.z - (sum - log_hi);
                log_hi = sum;
                umma::fence_proxy_async_smem();
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(c & 1 ? bar_w : bar_x);
            };
            if (chunks > 0) {
                if (chunks > 1) fetch(1);
                arrive();
                store(0);
            }
            for (int c = 0; c < chunks; ++c) {
                const float2 dec2 = make_float2(dec, dec), add2 = make_float2(add, add);
                if (c + 1 < chunks) {
                    convolve(c + 1, mx + 4 * ((c + 1) % 3));
                    if (c + 2 < chunks) fetch(c + 2);
                    arrive();
                    store(c + 1);
                }
                wait(c & 1 ? bar_y : bar_u, (uint32_t)(c >> 1) & 1u);
                umma::tc_fence_after();
                uint32_t v[32];
                umma::tmem_ld32_nowait((c & 1 ? T_YW : T_U) + lane_off + sc0, v);
                umma::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) S[j] = ffma2(dec2, S[j], fmul2(add2, as_float2(v[2 * j], v[2 * j + 1])));
            }
        } else {
            // maxima of this chunk, of the next (written from its convolution on) and of the one
            // after (cleared now; its last readers, of the previous chunk, have met since)
            uint32_t *m_now = mx, *m_next = mx + 4, *m_after = mx + 8;
            arrive();
            for (int c = 0; c < chunks; ++c) {
                const int b = c & 1;
                const uint32_t ph = (uint32_t)c & 1u, ph_full = (uint32_t)(c >> 1) & 1u;
                const float *rec0 = reinterpret_cast<const float *>(sm + Sm::OFF_REC) + b * 2 * REC, *rec1 = rec0 + REC;
                const float *recv = hv ? rec1 : rec0;
                wait(bar_m, ph);
                if (tid < 4) m_after[tid] = 0;

                // ---- scales; operands into shared memory
                const uint4 mxv = *reinterpret_cast<const uint4 *>(m_now);
                float xs0, xs1, xinv0, xinv1;
                scale_pow2(mxv.x, 13, xs0, xinv0);
                scale_pow2(mxv.y, 13, xs1, xinv1);
                wait(full + b, ph_full);
                store_x(half ? rec1 : rec0, half ? xs1 : xs0, Sm::OFF_XH - Sm::OFF_X);
                float s0, s1, i0, i1;
                scale_pow2(mxv.z, 13, s0, i0);
                scale_pow2(mxv.w, 13, s1, i1);
                const float sinv = hv ? i1 : i0;     // of the rows of y of this thread
                const float ss = cg < 2 ? s0 : s1;
                const float2 ss2 = make_float2(ss, ss);
                if (srow < N) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(p_s ^ (16 * j), make_uint4(pack(fmul2(S[4 * j], ss2)), pack(fmul2(S[4 * j + 1], ss2)),
                                                          pack(fmul2(S[4 * j + 2], ss2)), pack(fmul2(S[4 * j + 3], ss2))));
                }
                umma::fence_proxy_async_smem();
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_x);
                // ---- under the products: the previous chunk's gate, this one's decayed scores,
                // the next one's x
                if (c + 1 < chunks) fetch(c + 1);
                if (c > 0) gate(c - 1);
                // decayed scores: 16 of them per thread, as the A operand in tensor memory.
                // Half 0 (lanes 0..63) writes columns 64 .. 95 and half 1 columns 0 .. 31, where
                // the other half's scores lie in lanes that nobody reads.
                wait(bar_sc, ph);
                umma::tc_fence_after();
                uint32_t p[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if ((q & 1) || cg < 2) {   // tokens 0 .. 31 see nothing of 32 .. 63
                    uint32_t sc[16];
                    umma::tmem_ld16_nowait(T_SC + lane_off + 64 * hv + 16 * cg, sc);
                    const float Lt = recv[R_LR + t];   // times the row's power of two
                    umma::tmem_ld_wait();
                    if ((q & 1) && cg < 2) {
                        // t > 31 >= s: e^{L_t - L_s} = e^{L_t - L_31} e^{L_31 - L_s}, both at most 1
                        const float et = ex2(Lt - recv[R_L + 31]);
                        const float2 et2 = make_float2(et, et);
#pragma unroll
                        for (int s4 = 0; s4 < 4; ++s4) {
                            const float4 u4 = *reinterpret_cast<const float4 *>(recv + R_UH + 16 * cg + 4 * s4);
                            p[2 * s4] = pack(fmul2(fmul2(make_float2(u4.x, u4.y), et2), as_float2(sc[4 * s4], sc[4 * s4 + 1])));
                            p[2 * s4 + 1] = pack(fmul2(fmul2(make_float2(u4.z, u4.w), et2), as_float2(sc[4 * s4 + 2], sc[4 * s4 + 3])));
                        }
                    } else {
#pragma unroll
                        for (int s4 = 0; s4 < 4; ++s4) {
                            const int s = 16 * cg + 4 * s4;
                            const float4 l4 = *reinterpret_cast<const float4 *>(recv + R_L + s);
                            const float4 u4 = *reinterpret_cast<const float4 *>(recv + R_U + s);
                            float2 w0 = fmul2(as_float2(sc[4 * s4], sc[4 * s4 + 1]), make_float2(u4.x, u4.y));
                            float2 w1 = fmul2(as_float2(sc[4 * s4 + 2], sc[4 * s4 + 3]), make_float2(u4.z, u4.w));
                            w0 = fmul2(w0, make_float2(ex2(Lt - l4.x), ex2(Lt - l4.y)));
                            w1 = fmul2(w1, make_float2(ex2(Lt - l4.z), ex2(Lt - l4.w)));
                            p[2 * s4] = pack(make_float2(s > t ? 0.f : w0.x, s + 1 > t ? 0.f : w0.y));
                            p[2 * s4 + 1] = pack(make_float2(s + 2 > t ? 0.f : w1.x, s + 3 > t ? 0.f : w1.y));
                        }
                    }
                }
                umma::tmem_st8(T_SC + lane_off + (hv ? 0 : 64) + 8 * cg, p);
                umma::tmem_st_wait();
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_w);
                if (c + 1 < chunks) convolve(c + 1, m_next);
                // ---- state
                wait(bar_u, ph);
                umma::tc_fence_after();
                {
                    const float *rs = (cg < 2 ? rec0 : rec1) + R_END;
                    const float dec = rs[0], add = rs[3] * (cg < 2 ? xinv0 : xinv1);
                    const float2 dec2 = make_float2(dec, dec), add2 = make_float2(add, add);
                    uint32_t v[32];
                    umma::tmem_ld32_nowait(T_U + lane_off + sc0, v);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[j] = ffma2(dec2, S[j], fmul2(add2, as_float2(v[2 * j], v[2 * j + 1])));
                }
                state_max(m_next);
                // ---- y before its gate
                const float fx = hv ? xinv1 : xinv0;
                const float fi = recv[R_YI + t] * sinv, fw = recv[R_YW + t] * fx, fd = dskip * fx;
                const float2 fi2 = make_float2(fi, fi), fw2 = make_float2(fw, fw), fd2 = make_float2(fd, fd);
                wait(bar_w, ph);   // x of the other warps
                const uint4 xa = lds128(p_o), xb = lds128(p_o ^ 16);
                const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
                if (c + 1 < chunks) arrive();   // y needs nothing that the others may overwrite
                wait(bar_y, ph);
                umma::tc_fence_after();
                uint32_t yi[16], yw[16];
                umma::tmem_ld16_nowait(T_YI + lane_off + oc, yi);
                umma::tmem_ld16_nowait(T_YW + lane_off + oc, yw);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmul2(half2_float2(xw[e]), fd2);
                umma::tmem_ld_wait();
                umma::tc_fence_before();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = ffma2(as_float2(yi[2 * e], yi[2 * e + 1]), fi2,
                                 ffma2(as_float2(yw[2 * e], yw[2 * e + 1]), fw2, y[e]));
                uint32_t *const done = m_now;
                m_now = m_next;
                m_next = m_after;
                m_after = done;
            }
            if (chunks > 0) {
                gate(chunks - 1);
                arrive();
            }
        }
        float *const to = !owner || *abort_flag                         ? nullptr
                          : STATE_ONLY || (seg == 0 && last_seg > 0)    ? seg_ptr(seg)
                          : seg == last_seg && a.S_final                ? a.S_final + sbase
                                                                        : nullptr;
        if (to) {
            if (odd[128]) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (odd[sc0 + 2 * j] < INT_MAX) S[j].x = kNan;
                    if (odd[sc0 + 2 * j + 1] < INT_MAX) S[j].y = kNan;
                }
            }
#pragma unroll
            for (int j = 0; j < 16; j += 2)
                *reinterpret_cast<float4 *>(to + 2 * j) = make_float4(S[j].x, S[j].y, S[j + 1].x, S[j + 1].y);
            if (STATE_ONLY && lane == 0 && q == 0 && (cg & 1) == 0)
                a.seg_decay[seg_at(seg) * 2 + (cg >> 1)] = log_hi + log_lo;
        }
    }
    umma::tc_fence_before();
    __syncthreads();
    if (!STATE_ONLY && odd[128]) {
        // from the first x of a column that is not finite on, its outputs are NaN
        const int col = tid & 127, from = odd[col], to = min(c_hi * Q, end - begin);   // from INT_MAX: none
        for (int u = from; u < to; ++u)
            if (u % (THREADS / 128) == tid >> 7)
                a.out[(long long)(begin + u) * (a.H * a.P) + xcol + col] = __float2bfloat16(kNan);
    }
    if (warp == MMA_WARP) umma::tmem_dealloc(tb, 512);
}

// FIRST: the mixer over segment 0 of every sequence, and behind them the states of the
// segments that follow.  Else the mixer over those; or, with no cuts, over every sequence.
template <int N, bool FIRST>
__global__ void __launch_bounds__(stc::THREADS, 1)
ssm_chain_kernel(const ChainArgs a, const __grid_constant__ ChainMaps maps) {
    const int y = blockIdx.y;
    if (FIRST && y < a.n_seq) {
        chain_segment<N, false>(a, maps, y, 0, __ldg(a.cuts + y));
        return;
    }
    int2 at = make_int2(y, 0), cut = make_int2(1, 0);
    if (FIRST || a.cap > 0) {
        const int4 row = __ldg(a.rows + (FIRST ? y - a.n_seq : y));
        if (row.x < 0) return;
        at = make_int2(row.x, row.y);
        cut = make_int2(row.z, row.w);
    }
    chain_segment<N, FIRST>(a, maps, at.x, at.y, cut);
}

namespace {

size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    int blocks_per_group, blocks, slots, cap, even;
    size_t tiles, rec, seg_state, seg_decay, cuts, rows, bytes;
};

// Segments: a chain (128 columns of a sequence) is sequential over its chunks, 4.6 us each
// however many chains there are, so long sequences are cut while SMs would be idle.  A
// first launch runs segment 0, half as long, of every sequence and beside it the states of
// the others, which take about 2 us a chunk; a second one the others, as many as there are SMs
// (cap rows of blocks).  The lengths are on the device, so ssm_prep shares the rows out.
// Cut and whole, us: one prompt of 32768 tokens, 32 heads of 128, N = 128: 768 and 2140
// (with segment 0 0.4 or 0.55 of the others: 784); 4000 tokens, 16 heads of 64: 88 and
// 279; 2 x 2048, 64 heads of 64: 130 and 162; 8 prompts of 0 to 4095, 64 heads of 64: 271
// and 332; 9000 + 100, 64 heads of 128: 411 and 609.  What a batch pays that is not cut in
// the end: 4 x 4096: 304 and 303, 8 x 1000, 32 heads: 97 and 94 (equal lengths that are
// given as such pay nothing).
// Pieces of 2, 3 or 4 chunks at least: 768 tokens, 32 heads of 64: 60, 62, 68 us; 400
// tokens, 16 heads: 50, 49, 49.
Plan plan_for(const SsmArgs &a, int sms) {
    Plan p;
    const int R = a.H / a.G;
    p.blocks_per_group = (R * a.P + 127) / 128;
    p.blocks = a.G * p.blocks_per_group;
    p.slots = a.n_tok / stc::Q + a.n_seq;
    p.even = (int)(((long long)p.slots * p.blocks + sms - 1) / sms);
    p.cap = sms / p.blocks;
    // no room, nothing long enough, or equal lengths whose part of the rows is too small
    const int known = a.cu_seqlens ? 1 : a.n_seq;
    if (p.cap / known < 2 || a.n_seq > stc::PREP_THREADS || a.n_tok / known < 3 * stc::MIN_SEG * stc::Q) p.cap = 0;
    p.tiles = round256((size_t)p.slots * a.G * (a.N / 64) * stc::KB);
    p.rec = round256((size_t)p.slots * a.H * stc::REC * 4);
    p.seg_state = round256((size_t)p.cap * p.blocks * a.N * 128 * 4);
    p.seg_decay = round256((size_t)p.cap * p.blocks * 2 * 4);
    p.cuts = p.cap > 0 ? round256((size_t)a.n_seq * 8) : 0;
    p.rows = round256((size_t)p.cap * 16);
    p.bytes = p.tiles + p.rec + p.seg_state + p.seg_decay + p.cuts + p.rows;
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
    char *w = ws + p.tiles + p.rec + p.seg_state + p.seg_decay;
    pa.cuts = reinterpret_cast<int2 *>(w);
    pa.rows = reinterpret_cast<int4 *>(w + p.cuts);
    pa.slots = p.slots;
    pa.cap = p.cap;
    pa.even = p.even;
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
    ca.n_seq = a.n_seq; ca.n_tok = a.n_tok; ca.H = a.H; ca.G = a.G; ca.P = a.P;
    ca.blocks_per_group = p.blocks_per_group;
    ca.cuts = pa.cuts;
    ca.rows = pa.rows;
    ca.cap = p.cap;
    cudaError_t e;
    if (a.n_tok > 0) {
        ssm_prep_kernel<N><<<dim3(p.slots + (p.cap > 0), a.G), stc::PREP_THREADS, 0, a.stream>>>(pa);
        if ((e = launched()) != cudaSuccess) return e;
    }
    constexpr int SMEM = stc::Smem<N>::SIZE;
    ChainMaps maps = {};
    if (a.n_tok > 0) {
        if ((e = make_tma_mat_bf16(reinterpret_cast<TmaMap *>(&maps.out), a.out, a.H * a.P, a.n_tok, a.H * a.P, 64,
                                   stc::Q)) != cudaSuccess)
            return e;
        if (a.z && (e = make_tma_mat_bf16(reinterpret_cast<TmaMap *>(&maps.z), a.z, a.H * a.P, a.n_tok, (int)a.ld_z,
                                          64, stc::Q)) != cudaSuccess)
            return e;
    }
    if ((e = cudaFuncSetAttribute(ssm_chain_kernel<N, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) !=
        cudaSuccess)
        return e;
    if (p.cap > 0) {
        if ((e = cudaFuncSetAttribute(ssm_chain_kernel<N, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) !=
            cudaSuccess)
            return e;
        ssm_chain_kernel<N, true><<<dim3(p.blocks, a.n_seq + p.cap), stc::THREADS, SMEM, a.stream>>>(ca, maps);
        if ((e = launched()) != cudaSuccess) return e;
    }
    ssm_chain_kernel<N, false><<<dim3(p.blocks, p.cap > 0 ? p.cap : a.n_seq), stc::THREADS, SMEM, a.stream>>>(ca, maps);
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
