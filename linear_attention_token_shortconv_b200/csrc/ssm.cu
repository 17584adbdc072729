// The selective state-space mixer on fp32 arithmetic: the prefill of fp32 tensors
// (and of bf16 tensors with an fp32 result), the single-token step, and the
// convolution history that joins the two.  Per head h of group g = h / (H / G):
//
//   xh = SiLU(conv4(x) + b),  Bh, Ch likewise        (causal depthwise, width 4)
//   D_t = softplus(dt_t + b_dt),  a_t = exp(-exp(A) D_t)
//   S_t = a_t S_{t-1} + D_t Bh_t xh_t^T              [N, P], fp32
//   y_t = S_t^T Ch_t + D xh_t,   out = y SiLU(z)
//
// The prefill is two kernels.  ssm_act writes the convolved channels and (D_t, a_t)
// of every token in fp32; ssm_scan runs the recurrence with the state in registers.
// A column p of the state depends on no other column, so a CTA takes 16 columns of
// one (sequence, head): 64 threads, each two columns of N / 8 rows, 8 lanes of a
// warp sharing the columns and adding their parts of y by shuffles, four tokens
// together.  What bounds it is the chain of tokens, at one or two warps a scheduler; few
// and long sequences are cut into segments, whose states a first pass finds.
// 1000 + 999 tokens, 16 heads of 64, N = 64: 76 us, of it 13 for ssm_act (129 uncut).
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "ssm.cuh"

namespace gdn {
using ssm::Raw;
using ssm::decay_pair;
using ssm::load4;
using ssm::next_decay;
using ssm::relative_rest;
using ssm::seq_range;

namespace {

template <typename T> Raw<T> raw_of(const SsmArgs &a) {
    return Raw<T>{static_cast<const T *>(a.x), static_cast<const T *>(a.B), static_cast<const T *>(a.C),
                  a.ld_x, a.ld_B, a.ld_C, a.H * a.P, a.G * a.N};
}

// What a decay's remainder is applied to: an infinity times it would be NaN, or the other
// infinity.
__device__ __forceinline__ float finite(float s) { return fminf(fmaxf(s, -FLT_MAX), FLT_MAX); }

constexpr int ACT_TOK = 16;   // consecutive tokens per thread of ssm_act

// act [N_tok, channels] = SiLU(conv + bias); step [N_tok, H] = (D_t, a_t, a_t's remainder
// relative to it, -log a_t).
// blockIdx.x: run of ACT_TOK packed tokens, blockIdx.y * 256 + threadIdx.x: four
// channels, then (past the channels) one head.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_act_kernel(const Raw<T> raw, const T *__restrict__ hist, const float *__restrict__ conv_w,
               const float *__restrict__ conv_b, const T *__restrict__ dt, long long ld_dt,
               const float *__restrict__ A, const float *__restrict__ b_dt, const int32_t *__restrict__ cu, int n_seq,
               int n_tok, int H, float *__restrict__ act, float4 *__restrict__ step) {
    const int chans = raw.hp + 2 * raw.gn;
    const int v = blockIdx.y * blockDim.x + threadIdx.x;
    const int t0 = blockIdx.x * ACT_TOK, t1 = min(t0 + ACT_TOK, n_tok);
    int n, begin, end;   // the sequence of t0
    auto locate = [&] {
        n = cu ? seq_of_token(cu, n_seq, t0) : t0 / (n_tok / n_seq);
        seq_range(cu, n_seq, n_tok, n, begin, end);
    };
    if (v >= chans / 4) {
        const int h = v - chans / 4;
        if (h >= H) return;
        const float rate = expf(__ldg(A + h)), bias = __ldg(b_dt + h);
        locate();
        for (int t = t0; t < t1; ++t) {
            while (t >= end && n + 1 < n_seq) seq_range(cu, n_seq, n_tok, ++n, begin, end);
            if (t < begin || t >= end) continue;   // behind the last sequence
            const float d = softplus_acc(to_f32(dt[t * ld_dt + h]) + bias);
            const float2 a = decay_pair(rate * d);
            // the log is bounded so that sums of it stay finite; e^-10000 is 0
            step[(size_t)t * H + h] = make_float4(d, a.x, relative_rest(a), fminf(rate * d, 1e4f));
        }
        return;
    }
    const int c = 4 * v;
    float4 w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __ldg(reinterpret_cast<const float4 *>(conv_w) + c + e);
    const float4 b4 = conv_b ? __ldg(reinterpret_cast<const float4 *>(conv_b) + v) : make_float4(0, 0, 0, 0);
    locate();
    float4 r[4];   // raw rows t - 3 .. t
    bool fresh = true;
    for (int t = t0; t < t1; ++t) {
        while (t >= end && n + 1 < n_seq) {
            seq_range(cu, n_seq, n_tok, ++n, begin, end);
            fresh = true;
        }
        if (t < begin || t >= end) { fresh = true; continue; }   // behind the last sequence
        if (fresh) {
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int u = t - 3 + j;
                if (u >= begin) r[j + 1] = load4(raw.at(u, c));
                else if (hist) r[j + 1] = load4(hist + ((size_t)n * 3 + (u - begin + 3)) * chans + c);
                else r[j + 1] = make_float4(0, 0, 0, 0);
            }
            fresh = false;
        }
        r[0] = r[1]; r[1] = r[2]; r[2] = r[3];
        r[3] = load4(raw.at(t, c));
        float4 o;
        o.x = ssm::silu(fmaf(w[0].w, r[3].x, fmaf(w[0].z, r[2].x, fmaf(w[0].y, r[1].x, fmaf(w[0].x, r[0].x, b4.x)))));
        o.y = ssm::silu(fmaf(w[1].w, r[3].y, fmaf(w[1].z, r[2].y, fmaf(w[1].y, r[1].y, fmaf(w[1].x, r[0].y, b4.y)))));
        o.z = ssm::silu(fmaf(w[2].w, r[3].z, fmaf(w[2].z, r[2].z, fmaf(w[2].y, r[1].z, fmaf(w[2].x, r[0].z, b4.z)))));
        o.w = ssm::silu(fmaf(w[3].w, r[3].w, fmaf(w[3].z, r[2].w, fmaf(w[3].y, r[1].w, fmaf(w[3].x, r[0].w, b4.w)))));
        *reinterpret_cast<float4 *>(act + (size_t)t * chans + c) = o;
    }
}

constexpr int SCAN_COLS = 16, SCAN_TOK = 16, SCAN_THREADS = 64;

// An asynchronous copy of 16 bytes to shared memory, zeros where `in` is false.
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool in) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Sequences of at least `from` tokens in segments of `len` (a multiple of SCAN_TOK).
// STATE_ONLY runs every segment but a sequence's last from zero, segment 0 from S0, and
// leaves the state and the sum of its log-decays; the main pass starts each segment from
// those before it, joined.
struct Segments {
    int from, len;           // from = INT_MAX: no sequence
    // segment 0 of sequence n has slot n, its segment k > 0 slot n_seq + begin / len + k - 1:
    // the blocks that all sequences have start first, and spread over the SMs
    int slots;
    float *state;            // [slot][H][N][P]
    float *decay;            // [slot][H]: -log
    float *s0_copy;          // S0 where the final state replaces it, else NULL
};

template <int N, typename T, typename Tout, bool STATE_ONLY>
__global__ void __launch_bounds__(SCAN_THREADS)
ssm_scan_kernel(const float *__restrict__ act, const float4 *__restrict__ step, const float *__restrict__ Dw,
                const T *__restrict__ z, long long ld_z, const float *S0, const int32_t *__restrict__ cu, int n_seq,
                int n_tok, int H, int G, int P, const Segments seg, Tout *__restrict__ out, float *S_final) {
    constexpr int R = N / 8;             // state rows of a thread
    struct Stage {
        float b[SCAN_TOK][N], c[SCAN_TOK][N], x[SCAN_TOK][SCAN_COLS];
        float4 d[SCAN_TOK];
    };
    __shared__ __align__(16) Stage stages[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = P / SCAN_COLS, slot = blockIdx.y, h = blockIdx.x / cols, p0 = blockIdx.x % cols * SCAN_COLS;
    const int slice = lane & 7, lcol = 8 * warp + 2 * (lane >> 3);   // rows 4 slice + 32 i + e, columns lcol, lcol + 1
    const int chans = H * P + 2 * G * N, g = h / (H / G);
    int n = slot, begin, end;
    if (slot >= n_seq) {   // the last sequence whose later segments start at or before this slot
        n = 0;
        for (int hi = n_seq; hi - n > 1;) {
            const int mid = (n + hi) >> 1;
            seq_range(cu, n_seq, n_tok, mid, begin, end);
            if (n_seq + begin / seg.len <= slot) n = mid; else hi = mid;
        }
    }
    seq_range(cu, n_seq, n_tok, n, begin, end);
    const int later = n_seq + begin / seg.len - 1;             // slot of segment k > 0: later + k
    const int k = slot < n_seq ? 0 : slot - later;
    if (slot >= n_seq && k < 1) return;
    const int last = end - begin >= seg.from ? (end - begin - 1) / seg.len : 0;
    if (STATE_ONLY ? k >= last : k > last) return;
    if (k < last) end = begin + (k + 1) * seg.len;
    begin += k * seg.len;
    auto load = [&](int t0, Stage &st) {
        const int len = end - t0;   // rows past the end are zeros
        const float *rows = act + (size_t)t0 * chans;
        for (int i = tid; i < SCAN_TOK * (N / 4); i += SCAN_THREADS) {
            const int r = i / (N / 4), q = i % (N / 4);
            const float *src = rows + (r < len ? (size_t)r * chans : 0) + H * P + g * N + 4 * q;
            copy_async(&st.b[r][4 * q], src, r < len);
            if (!STATE_ONLY) copy_async(&st.c[r][4 * q], src + G * N, r < len);
        }
        for (int i = tid; i < SCAN_TOK * (SCAN_COLS / 4); i += SCAN_THREADS) {
            const int r = i / (SCAN_COLS / 4), q = i % (SCAN_COLS / 4);
            copy_async(&st.x[r][4 * q], rows + (r < len ? (size_t)r * chans : 0) + h * P + p0 + 4 * q, r < len);
        }
        if (tid < SCAN_TOK) copy_async(&st.d[tid], step + (size_t)(t0 + (tid < len ? tid : 0)) * H + h, tid < len);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (begin < end) load(begin, stages[0]);
    // element of state row i of this thread in a [H][N][P] state
    auto at = [&](int i) { return ((size_t)h * N + 32 * (i / 4) + 4 * slice + (i & 3)) * P + p0 + lcol; };
    const size_t one = (size_t)H * N * P;
    float2 S[R];
    float carry = 0.f;   // relative remainder of the decays that S has not been given yet
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = make_float2(0.f, 0.f);
    if (STATE_ONLY || k == 0) {
        const float *from = k > 0 ? nullptr : !STATE_ONLY && last > 0 && seg.s0_copy ? seg.s0_copy : S0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (from) S[i] = *reinterpret_cast<const float2 *>(from + n * one + at(i));
            if (STATE_ONLY && from && seg.s0_copy) *reinterpret_cast<float2 *>(seg.s0_copy + n * one + at(i)) = S[i];
        }
    } else {
        for (int i0 = 0; i0 < k; ++i0) {   // S <- decay S + state
            const size_t j = i0 == 0 ? n : later + i0;
            float d = 0.f;
            if (i0 > 0) {
                const float2 a = decay_pair(seg.decay[j * H + h]);
                carry += relative_rest(a);
                d = next_decay(a.x, carry);
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                S[i] = ffma2(make_float2(d, d), S[i], *reinterpret_cast<const float2 *>(seg.state + j * one + at(i)));
        }
    }
    const float dw = Dw ? __ldg(Dw + h) : 0.f;
    float log_hi = 0.f, log_lo = 0.f;   // sum of the segment's log-decays
    for (int t0 = begin, b = 0; t0 < end; t0 += SCAN_TOK, b ^= 1) {
        const int len = min(SCAN_TOK, end - t0);
        const Stage &st = stages[b];
        if (t0 + SCAN_TOK < end) {
            load(t0 + SCAN_TOK, stages[b ^ 1]);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        // the stage's first decay takes the remainders before it: once a stage 3 % of the time,
        // at every token 14
        const float first = next_decay(st.d[0].y, carry);
        float logs = 0.f;
        // four tokens at a time: their recurrences follow one another, but their parts of y
        // (8 values) are added over the eight slices together, one value staying in each lane
        for (int r = 0; r < len; r += 4) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 da = st.d[r + u];
                const float a = r + u >= len ? 1.f : u == 0 && r == 0 ? first : da.y;
                carry += da.z;
                const float2 x = *reinterpret_cast<const float2 *>(&st.x[r + u][lcol]);
                const float2 dx = make_float2(da.x * x.x, da.x * x.y), aa = make_float2(a, a);
                if (STATE_ONLY) logs += da.w;
                float2 y = make_float2(0.f, 0.f);
#pragma unroll
                for (int i4 = 0; i4 < R / 4; ++i4) {
                    const float4 b = *reinterpret_cast<const float4 *>(&st.b[r + u][32 * i4 + 4 * slice]);
                    const float4 c = STATE_ONLY ? b : *reinterpret_cast<const float4 *>(&st.c[r + u][32 * i4 + 4 * slice]);
                    const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 &s = S[4 * i4 + e];
                        s = ffma2(aa, s, fmul2(make_float2(bb[e], bb[e]), dx));
                        if (!STATE_ONLY) y = ffma2(make_float2(cc[e], cc[e]), s, y);
                    }
                }
                v[2 * u] = y.x;
                v[2 * u + 1] = y.y;
            }
            if constexpr (!STATE_ONLY) {
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    const bool up = slice & o;
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                const int ru = r + (slice >> 1), cu1 = lcol + (slice & 1);   // this lane's token and column
                if (ru < len) {
                    const long long t = t0 + ru;
                    const int p = p0 + cu1;
                    float o = fmaf(dw, st.x[ru][cu1], v[0]);
                    if (z) o *= ssm::silu(to_f32(z[t * ld_z + (long long)h * P + p]));
                    out[(t * H + h) * P + p] = from_f32<Tout>(o);
                }
            }
        }
        if (STATE_ONLY) {
            // two sums, since equal addends are rounded alike
            const float sum = log_hi + logs;
            log_lo += logs - (sum - log_hi);
            log_hi = sum;
        }
        __syncthreads();   // before the stage is loaded again
    }
    // what is left of the remainders
#pragma unroll
    for (int i = 0; i < R; ++i) {
        S[i].x = fmaf(carry, finite(S[i].x), S[i].x);
        S[i].y = fmaf(carry, finite(S[i].y), S[i].y);
    }
    float *const to = STATE_ONLY ? seg.state + slot * one : k == last && S_final ? S_final + n * one : nullptr;
    if (to) {
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float2 *>(to + at(i)) = S[i];
    }
    if (STATE_ONLY && p0 == 0 && tid == 0) seg.decay[(size_t)slot * H + h] = log_hi + log_lo;
}

// tail [n, j] = the raw channels of token end - 3 + j of sequence n, or the row of
// the older history that lies as far back (zeros without one).  A thread reads its
// four channels' rows before it writes them, so tail may be the history itself.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_tail_kernel(const Raw<T> raw, const T *hist, const int32_t *__restrict__ cu, int n_seq, int n_tok, T *tail) {
    const int chans = raw.hp + 2 * raw.gn, c = 4 * (blockIdx.x * blockDim.x + threadIdx.x), n = blockIdx.y;
    if (c >= chans) return;
    typedef typename std::conditional<sizeof(T) == 2, uint2, uint4>::type V;   // four raw elements
    int begin, end;
    seq_range(cu, n_seq, n_tok, n, begin, end);
    V r[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int t = end - 3 + j;
        if (t >= begin) r[j] = *reinterpret_cast<const V *>(raw.at(t, c));
        else if (hist) r[j] = *reinterpret_cast<const V *>(hist + ((size_t)n * 3 + (t - begin + 3)) * chans + c);
        else r[j] = V{};
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) *reinterpret_cast<V *>(tail + ((size_t)n * 3 + j) * chans + c) = r[j];
}

template <typename T>
cudaError_t launch_tail(const SsmArgs &a) {
    const int chans = a.H * a.P + 2 * a.G * a.N;
    const dim3 grid((chans / 4 + 255) / 256, a.n_seq);
    ssm_tail_kernel<T><<<grid, 256, 0, a.stream>>>(raw_of<T>(a), static_cast<const T *>(a.hist), a.cu_seqlens, a.n_seq,
                                                   a.n_tok, static_cast<T *>(a.tail));
    return launched();
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace of the fp32 prefill, and its segments.  A block alone on an SM takes 129 ns a
// token, a full SM 58 per block (N = 128), and segments cost half as much again for their
// states.  So they are made where the sequences have no more blocks than there are SMs,
// SCAN_FULL of them an SM, of the sequences that are longer than an even share of the work
// (one of 8000 tokens, 16 heads of 64, N = 128: 1032 us whole, 479 with 3 to an SM, 343
// with 6, 359 with 10; 4 of 2000 with 32 heads, more blocks than SMs: 482 whole, 633 cut).
struct ScanPlan {
    int from, len, slots;
    size_t act, step, state, decay, s0_copy;
    size_t bytes() const { return act + step + state + decay + s0_copy; }
};
constexpr int SCAN_FULL = 6, SCAN_MIN = 64;

ScanPlan scan_plan(const SsmArgs &a, int sms) {
    ScanPlan p = {};
    const size_t chans = (size_t)a.H * a.P + 2 * (size_t)a.G * a.N, one = (size_t)a.H * a.N * a.P * 4;
    p.act = round256((size_t)a.n_tok * chans * 4);
    p.step = round256((size_t)a.n_tok * a.H * 16);
    p.slots = a.n_seq;
    p.from = INT_MAX;
    p.len = 1;
    const long long blocks = (long long)a.H * a.P / SCAN_COLS, all = a.n_seq * blocks;
    const long long len = all <= sms ? a.n_tok * blocks / (SCAN_FULL * sms - all) / SCAN_TOK * SCAN_TOK + SCAN_TOK : 0;
    const long long even = a.n_tok * blocks / sms;
    const int longest = a.cu_seqlens ? a.n_tok : a.n_tok / a.n_seq;
    if (all <= sms && longest >= 2 * SCAN_MIN) {
        p.len = len > SCAN_MIN ? (int)len : SCAN_MIN;
        p.from = even > 2 * p.len ? (int)even : 2 * p.len;
        p.slots += a.n_tok / p.len;
        p.state = round256(p.slots * one);
        p.decay = round256((size_t)p.slots * a.H * 4);
        p.s0_copy = round256(a.n_seq * one);
    }
    return p;
}

template <int N, typename T, typename Tout>
cudaError_t launch_scan(const SsmArgs &a, const float *act, const float4 *step, const ScanPlan &p, const Segments &seg) {
    const dim3 grid(a.H * (a.P / SCAN_COLS), p.slots);
    if (p.from < INT_MAX) {
        ssm_scan_kernel<N, T, Tout, true><<<grid, SCAN_THREADS, 0, a.stream>>>(
            act, step, a.D, static_cast<const T *>(a.z), a.ld_z, a.S0, a.cu_seqlens, a.n_seq, a.n_tok, a.H, a.G, a.P,
            seg, static_cast<Tout *>(a.out), a.S_final);
        const cudaError_t e = launched();
        if (e != cudaSuccess) return e;
    }
    ssm_scan_kernel<N, T, Tout, false><<<grid, SCAN_THREADS, 0, a.stream>>>(
        act, step, a.D, static_cast<const T *>(a.z), a.ld_z, a.S0, a.cu_seqlens, a.n_seq, a.n_tok, a.H, a.G, a.P, seg,
        static_cast<Tout *>(a.out), a.S_final);
    return launched();
}

template <typename T, typename Tout>
cudaError_t launch_fp32(const SsmArgs &a, char *ws, int sms) {
    const ScanPlan p = scan_plan(a, sms);
    const int chans = a.H * a.P + 2 * a.G * a.N;
    float *act = reinterpret_cast<float *>(ws);
    float4 *step = reinterpret_cast<float4 *>(ws + p.act);
    if (a.n_tok > 0) {
        const dim3 grid((a.n_tok + ACT_TOK - 1) / ACT_TOK, (chans / 4 + a.H + 255) / 256);
        ssm_act_kernel<T><<<grid, 256, 0, a.stream>>>(raw_of<T>(a), static_cast<const T *>(a.hist), a.conv_w, a.conv_b,
                                                      static_cast<const T *>(a.dt), a.ld_dt, a.A, a.b_dt,
                                                      a.cu_seqlens, a.n_seq, a.n_tok, a.H, act, step);
        const cudaError_t e = launched();
        if (e != cudaSuccess) return e;
    }
    char *const w = ws + p.act + p.step;
    const Segments seg = {p.from, p.len, p.slots, reinterpret_cast<float *>(w), reinterpret_cast<float *>(w + p.state),
                          p.s0_copy && a.S0 && a.S0 == a.S_final ? reinterpret_cast<float *>(w + p.state + p.decay) : nullptr};
    return a.N == 128 ? launch_scan<128, T, Tout>(a, act, step, p, seg) : launch_scan<64, T, Tout>(a, act, step, p, seg);
}

}  // namespace

size_t ssm_workspace_bytes(const SsmArgs &a, int sms) {
    if (ssm_tc_supported(a)) return ssm_tc_workspace_bytes(a, sms);
    return scan_plan(a, sms).bytes();
}

cudaError_t launch_ssm_prefill(const SsmArgs &a, void *ws, int sms) {
    cudaError_t e;
    if (ssm_tc_supported(a)) e = launch_ssm_tc(a, ws, sms);
    else if (a.in_bf16) e = launch_fp32<bf16, float>(a, static_cast<char *>(ws), sms);
    else {
        e = a.out_bf16 ? launch_fp32<float, bf16>(a, static_cast<char *>(ws), sms)
                       : launch_fp32<float, float>(a, static_cast<char *>(ws), sms);
    }
    if (e != cudaSuccess || !a.tail) return e;
    // last: every reader of the history has finished, so the tail may replace it
    return a.in_bf16 ? launch_tail<bf16>(a) : launch_tail<float>(a);
}

// ------------------------------------------------------------------ one token

namespace {

// One CTA per (head, sequence), 4 P threads of N / 16 float4 of state each: the state's
// loads are issued first, the convolution of the head's x channels and of its group's B
// and C runs while they are in flight, then every element is updated, written back and
// added into y.  The history of the x channels, which no other CTA reads, is shifted here;
// that of B and C, which all heads of a group read, by ssm_shift after this kernel.
// HBM-bound: 256 sequences x 32 heads of 128, N = 128, 1.09 GB: 170 us, 166 at the copy
// rate (200 with a head's state spread over CTAs of 32 columns, 186 with 64).  One
// sequence of 64 heads: 4.8 us, the launches and one trip to memory.
template <int N, int COLS, typename T, typename Tout>
__global__ void __launch_bounds__(4 * COLS)
ssm_decode_kernel(const Raw<T> raw, const T *__restrict__ dt, long long ld_dt, const float *__restrict__ conv_w,
                  const float *__restrict__ conv_b, T *hist, const float *__restrict__ A,
                  const float *__restrict__ b_dt, const float *__restrict__ Dw, const T *__restrict__ z,
                  long long ld_z, float *S, Tout *__restrict__ out, int H, int G) {
    constexpr int P = COLS, THREADS = 4 * COLS, F4 = COLS / 4, ROWS = 16, NV = N / ROWS;
    __shared__ __align__(16) float xs[COLS], bs[N], cs[N];
    __shared__ __align__(16) float part[ROWS][COLS];
    const int tid = threadIdx.x, h = blockIdx.x, col0 = h * COLS, b = blockIdx.y, g = h / (H / G);
    const int q = tid % F4, row0 = tid / F4;
    const int chans = raw.hp + 2 * raw.gn;
    float *Sh = S + (((size_t)b * H + h) * N + row0) * P + 4 * q;   // rows ROWS apart
    float4 s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = __ldcs(reinterpret_cast<const float4 *>(Sh + (size_t)i * ROWS * P));
    const float d = softplus_acc(to_f32(dt[b * ld_dt + h]) + __ldg(b_dt + h));
    const float2 a = decay_pair(expf(__ldg(A + h)) * d);
    for (int i = tid; i < COLS + 2 * N; i += THREADS) {
        const int c = i < COLS       ? col0 + i
                      : i < COLS + N ? raw.hp + g * N + (i - COLS)
                                     : raw.hp + raw.gn + g * N + (i - COLS - N);
        const float4 w = __ldg(reinterpret_cast<const float4 *>(conv_w) + c);
        T *hb = hist + (size_t)b * 3 * chans + c;
        const T r0 = hb[0], r1 = hb[chans], r2 = hb[2 * (size_t)chans], r3 = *raw.at(b, c);
        float v = conv_b ? __ldg(conv_b + c) : 0.f;
        v = fmaf(w.w, to_f32(r3), fmaf(w.z, to_f32(r2), fmaf(w.y, to_f32(r1), fmaf(w.x, to_f32(r0), v))));
        v = ssm::silu(v);
        if (i < COLS) {
            xs[i] = v;
            hb[0] = r1; hb[chans] = r2; hb[2 * (size_t)chans] = r3;
        } else if (i < COLS + N) bs[i - COLS] = d * v;
        else cs[i - COLS - N] = v;
    }
    __syncthreads();
    const float4 x = *reinterpret_cast<const float4 *>(&xs[4 * q]);
    float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = row0 + i * ROWS;
        const float bb = bs[row], cc = cs[row];
        s[i].x = fmaf(a.x, s[i].x, fmaf(a.y, finite(s[i].x), bb * x.x)); y.x = fmaf(cc, s[i].x, y.x);
        s[i].y = fmaf(a.x, s[i].y, fmaf(a.y, finite(s[i].y), bb * x.y)); y.y = fmaf(cc, s[i].y, y.y);
        s[i].z = fmaf(a.x, s[i].z, fmaf(a.y, finite(s[i].z), bb * x.z)); y.z = fmaf(cc, s[i].z, y.z);
        s[i].w = fmaf(a.x, s[i].w, fmaf(a.y, finite(s[i].w), bb * x.w)); y.w = fmaf(cc, s[i].w, y.w);
        __stcs(reinterpret_cast<float4 *>(Sh + (size_t)i * ROWS * P), s[i]);
    }
    *reinterpret_cast<float4 *>(&part[row0][4 * q]) = y;
    __syncthreads();
    if (tid < COLS) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v += part[r][tid];
        if (Dw) v = fmaf(__ldg(Dw + h), xs[tid], v);
        if (z) v *= ssm::silu(to_f32(z[b * ld_z + col0 + tid]));
        out[(size_t)b * H * P + col0 + tid] = from_f32<Tout>(v);
    }
}

// Shifts the history of the B and C channels by the current token, four channels a thread.
template <typename T>
__global__ void __launch_bounds__(128) ssm_shift_kernel(const Raw<T> raw, T *hist) {
    typedef typename std::conditional<sizeof(T) == 2, uint2, uint4>::type V;
    const int chans = raw.hp + 2 * raw.gn, c = raw.hp + 4 * (blockIdx.x * blockDim.x + threadIdx.x), b = blockIdx.y;
    if (c >= chans) return;
    T *hb = hist + (size_t)b * 3 * chans + c;
    const V r1 = *reinterpret_cast<V *>(hb + chans), r2 = *reinterpret_cast<V *>(hb + 2 * (size_t)chans);
    const V r3 = *reinterpret_cast<const V *>(raw.at(b, c));
    *reinterpret_cast<V *>(hb) = r1;
    *reinterpret_cast<V *>(hb + chans) = r2;
    *reinterpret_cast<V *>(hb + 2 * (size_t)chans) = r3;
}

template <int N, int P, typename T, typename Tout>
cudaError_t launch_decode_typed(const SsmArgs &a) {
    T *hist = static_cast<T *>(const_cast<void *>(a.hist));
    ssm_decode_kernel<N, P, T, Tout><<<dim3(a.H, a.n_seq), 4 * P, 0, a.stream>>>(
        raw_of<T>(a), static_cast<const T *>(a.dt), a.ld_dt, a.conv_w, a.conv_b, hist, a.A, a.b_dt, a.D,
        static_cast<const T *>(a.z), a.ld_z, a.S_final, static_cast<Tout *>(a.out), a.H, a.G);
    const cudaError_t e = launched();
    if (e != cudaSuccess) return e;
    ssm_shift_kernel<T><<<dim3((2 * a.G * a.N / 4 + 127) / 128, a.n_seq), 128, 0, a.stream>>>(raw_of<T>(a), hist);
    return launched();
}

template <int N, int P>
cudaError_t launch_decode_dims(const SsmArgs &a) {
    if (a.in_bf16)
        return a.out_bf16 ? launch_decode_typed<N, P, bf16, bf16>(a) : launch_decode_typed<N, P, bf16, float>(a);
    return a.out_bf16 ? launch_decode_typed<N, P, float, bf16>(a) : launch_decode_typed<N, P, float, float>(a);
}

}  // namespace

cudaError_t launch_ssm_decode(const SsmArgs &a) {
    if (a.N == 128) return a.P == 128 ? launch_decode_dims<128, 128>(a) : launch_decode_dims<128, 64>(a);
    return a.P == 128 ? launch_decode_dims<64, 128>(a) : launch_decode_dims<64, 64>(a);
}

}  // namespace gdn
