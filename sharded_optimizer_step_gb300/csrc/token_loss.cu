// Losses over a language model's logits, forward and backward: the clipped
// policy loss with a KL term and the preference loss of paired sequences.
//
// With x a token's logits, y its id: mx = max x, S = sum exp(x - mx),
// a = (x_y - mx) - log S.  The maximum is subtracted before the scaling to
// base 2, so rows of the type's lowest value and rows with -inf entries are
// right, and a is formed from differences, which keeps the digits that
// x_y - (mx + log S) would lose.  Both losses have d loss / d x =
// c (1[y] - softmax x) with one c per row, so a row is read for S, then again
// for its gradient.  Statistics, terms and coefficients are fp32, sums over
// tokens double; the gradient is rounded once, to the logits' type.
#include "common.cuh"

namespace shardstep {
namespace {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
// log2 e as the sum of two floats: the first alone is 1.3e-8 off, always to
// the same side, which a sum over a sequence's tokens would gather up.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = 1.9259629911e-8f;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int GT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (GT == kGradF32) return static_cast<const float*>(p)[i];
    if constexpr (GT == kGradF16) return f16_to_f32(static_cast<const uint16_t*>(p)[i]);
    return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
template <int GT>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
    if constexpr (GT == kGradF32)
        static_cast<float*>(p)[i] = x;
    else if constexpr (GT == kGradF16)
        static_cast<uint16_t*>(p)[i] = __half_as_ushort(__float2half_rn(x));
    else
        static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
}
template <int GT>
__device__ __forceinline__ const char* row_of(const void* x, int64_t i, int64_t stride) {
    return static_cast<const char*>(x) + i * stride * (GT == kGradF32 ? 4 : 2);
}

// A partial softmax sum: s = sum exp(x - m) over the elements seen, m their
// maximum.  An m of -inf (nothing seen but -inf) refers to 0 instead, so that
// no inf - inf arises; NaN elements reach s.
struct Soft {
    float m, s;
};
__device__ __forceinline__ float soft_ref(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float soft_exp(float x, float ref) {
    const float d = __fsub_rn(x, ref);
    return exp2_approx(__fmaf_rn(d, kLog2e, __fmul_rn(d, kLog2eLo)));
}
__device__ __forceinline__ Soft soft_join(Soft a, Soft b) {
    const float m = fmaxf(a.m, b.m);
    const float r = soft_ref(m);
    return Soft{m, __fadd_rn(__fmul_rn(a.s, soft_exp(a.m, r)), __fmul_rn(b.s, soft_exp(b.m, r)))};
}

// All threads get the block's join, formed in a fixed order.
__device__ __forceinline__ Soft block_soft(Soft a) {
    __shared__ Soft part[kRowWarps];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        a = soft_join(a, Soft{__shfl_xor_sync(kFull, a.m, d), __shfl_xor_sync(kFull, a.s, d)});
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = part[threadIdx.x & (kRowWarps - 1)];
#pragma unroll
    for (int d = kRowWarps / 2; d > 0; d >>= 1)
        a = soft_join(a, Soft{__shfl_xor_sync(kFull, a.m, d), __shfl_xor_sync(kFull, a.s, d)});
    return a;
}

// Thread 0 gets the block's sum in a fixed order.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kRowWarps];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_down_sync(kFull, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kRowWarps; ++w) s += part[w];
    return s;
}

// The row's id, or -1 where it lies outside the vocabulary: the token's log
// probability is then NaN, and so is the loss.
__device__ __forceinline__ int64_t token_id(const TokenArgs& a, int64_t i) {
    const int64_t y = a.ids64 ? static_cast<const int64_t*>(a.ids)[i]
                              : static_cast<const int32_t*>(a.ids)[i];
    return y >= 0 && y < a.v ? y : -1;
}

template <int GT>
__device__ __forceinline__ Soft row_soft(const char* x, int64_t v) {
    Soft a{-INFINITY, 0.0f};
    for (int64_t j = threadIdx.x; j < v; j += kRowThreads) {
        const float f = load1<GT>(x, j);
        const float m = fmaxf(a.m, f);
        const float r = soft_ref(m);
        a.s = __fadd_rn(__fmul_rn(a.s, soft_exp(a.m, r)), soft_exp(f, r));
        a.m = m;
    }
    return block_soft(a);
}

// grad = c (1[y] - exp(x - ref) inv), rounded once.
template <int GT>
__device__ __forceinline__ void row_grad(const char* x, char* g, int64_t v, int64_t y, float ref,
                                         float inv, float c) {
    const float f = -__fmul_rn(c, inv);
    for (int64_t j = threadIdx.x; j < v; j += kRowThreads) {
        float d = __fmul_rn(soft_exp(load1<GT>(x, j), ref), f);
        if (j == y) d = __fadd_rn(d, c);
        store1<GT>(g, j, d);
    }
}
template <int GT>
__device__ __forceinline__ void row_zero(char* g, int64_t v) {
    for (int64_t j = threadIdx.x; j < v; j += kRowThreads) store1<GT>(g, j, 0.0f);
}

// The blocks' sums (thread 0's t) added up by the block that arrives last, in
// block order; true there, with the sums in the workspace's total.
__device__ __forceinline__ bool join_blocks(LossWork* ws, const double* t, bool first) {
    __shared__ bool last;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 4; ++k) ws->partial[blockIdx.x][k] = t[k];
        __threadfence();
        last = atomicInc(&ws->arrived, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return false;
    __threadfence();
    if (threadIdx.x < 4) {
        double s = first ? 0.0 : ws->total[threadIdx.x];
        for (unsigned b = 0; b < gridDim.x; ++b) s += __ldcg(&ws->partial[b][threadIdx.x]);
        ws->total[threadIdx.x] = s;
    }
    __syncthreads();
    return true;
}

// One token's policy terms from its log probability:
//   u = exp(a - old); policy = -min(u A, clip(u) A); d = ref - a;
//   kl = expm1(d) - d; slope = d (policy + k kl) / d a.
struct PolicyTerms {
    float policy, kl, clipped, slope;
};
__device__ __forceinline__ PolicyTerms policy_terms(float lp, float old, float adv, float ref,
                                                    const PolicyArgs& p) {
    const float u = expf(__fsub_rn(lp, old));
    const float cu = u < p.lo ? p.lo : u > p.hi ? p.hi : u;
    const float one = __fmul_rn(u, adv), two = __fmul_rn(cu, adv);
    PolicyTerms t;
    t.clipped = one > two ? 1.0f : 0.0f;
    t.policy = one > two ? -two : -one;
    t.slope = one > two ? 0.0f : -one;
    t.kl = 0.0f;
    if (p.kl != 0.0f) {
        const float d = __fsub_rn(ref, lp);
        const float e = expm1f(d);
        t.kl = __fsub_rn(e, d);
        t.slope = __fsub_rn(t.slope, __fmul_rn(p.kl, e));
    }
    return t;
}

// The divisor of the means: given, or the sum of the weights, which every
// block adds up by itself in the same order.
__device__ __forceinline__ float weight_sum(const TokenArgs& a) {
    __shared__ float total;
    if (a.norm != 0.0f) return a.norm;
    if (a.w == nullptr) return static_cast<float>(a.n);
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < a.n; i += kRowThreads) s += static_cast<double>(a.w[i]);
    s = block_sum(s);
    if (threadIdx.x == 0) total = __double2float_rn(s);
    __syncthreads();
    return total;
}

template <int GT>
__global__ void __launch_bounds__(kRowThreads)
    policy_rows(const TokenArgs a, const PolicyArgs p) {
    pdl_enter();
    const float norm = weight_sum(a);
    const float out_scale =
        a.loss_scale != nullptr ? __fmul_rn(a.grad_scale, __ldg(a.loss_scale)) : a.grad_scale;
    double sums[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
        const char* x = row_of<GT>(a.x, i, a.x_stride);
        char* g = const_cast<char*>(row_of<GT>(a.grad, i, a.g_stride));
        const float w = a.w != nullptr ? a.w[i] : 1.0f;
        if (w == 0.0f) {   // not read at all: whatever it holds takes no part
            if (threadIdx.x == 0) a.logps[i] = 0.0f;
            if (a.grad != nullptr) row_zero<GT>(g, a.v);
            continue;
        }
        const int64_t y = token_id(a, i);
        const float xy = y >= 0 ? load1<GT>(x, y) : NAN;
        const Soft s = row_soft<GT>(x, a.v);
        const float lp = __fsub_rn(__fsub_rn(xy, s.m), logf(s.s));
        const PolicyTerms t =
            policy_terms(lp, p.old[i], p.adv[i], p.kl != 0.0f ? a.ref[i] : 0.0f, p);
        const float k = __fdiv_rn(w, norm);
        if (threadIdx.x == 0) {
            a.logps[i] = lp;
            const double kd = k;
            sums[0] += kd * __fadd_rn(t.policy, __fmul_rn(p.kl, t.kl));
            sums[1] += kd * t.policy;
            sums[2] += kd * t.kl;
            sums[3] += kd * t.clipped;
        }
        if (a.grad != nullptr)
            row_grad<GT>(x, g, a.v, y, soft_ref(s.m), __fdiv_rn(1.0f, s.s),
                         __fmul_rn(__fmul_rn(t.slope, k), out_scale));
    }
    if (join_blocks(a.ws, sums, true) && threadIdx.x < 4)
        a.stats[threadIdx.x] = __double2float_rn(a.ws->total[threadIdx.x]);
}

// The sequence that a row of the launch belongs to.
__device__ __forceinline__ int find_sequence(const PairTable& t, int row) {
    int lo = 0, hi = 2 * t.pairs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.start[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float softplus(float x) {
    return __fadd_rn(fmaxf(x, 0.0f), log1pf(expf(-fabsf(x))));
}
__device__ __forceinline__ float sigmoid(float x) {
    return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x)));
}

template <int GT>
__global__ void __launch_bounds__(kRowThreads)
    preference_forward(const TokenArgs a, const PreferenceArgs p,
                       const __grid_constant__ PairTable t) {
    pdl_enter();
    const int row0 = t.start[0], rows = t.start[2 * t.pairs] - row0;
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t i = row0 + r;
        const float w = a.w != nullptr ? a.w[i] : 1.0f;
        if (w == 0.0f) {
            if (threadIdx.x == 0) {
                a.logps[i] = 0.0f;
                p.term[i] = 0.0f;
            }
            continue;
        }
        const char* x = row_of<GT>(a.x, i, a.x_stride);
        const int64_t y = token_id(a, i);
        const float xy = y >= 0 ? load1<GT>(x, y) : NAN;
        const Soft s = row_soft<GT>(x, a.v);
        if (threadIdx.x == 0) {
            const float lp = __fsub_rn(__fsub_rn(xy, s.m), logf(s.s));
            a.logps[i] = lp;
            p.term[i] = __fmul_rn(w, __fsub_rn(lp, a.ref[i]));
            p.row_max[i] = soft_ref(s.m);
            p.row_inv[i] = __fdiv_rn(1.0f, s.s);
        }
    }
    // The last block: a warp per pair adds up its two sequences in a fixed
    // order and forms the pair's loss and slope.
    const double none[4] = {0.0, 0.0, 0.0, 0.0};
    if (!join_blocks(a.ws, none, p.first != 0)) return;
    const int lane = threadIdx.x & 31;
    const float norm = a.norm;
    double sums[3] = {0.0, 0.0, 0.0};
    for (int q = threadIdx.x >> 5; q < t.pairs; q += kRowWarps) {
        float r[2];
        for (int h = 0; h < 2; ++h) {
            double s = 0.0;
            for (int i = t.start[2 * q + h] + lane; i < t.start[2 * q + h + 1]; i += 32)
                s += static_cast<double>(__ldcg(p.term + i));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            r[h] = __double2float_rn(s);
        }
        const float h = __fmul_rn(p.beta, __fsub_rn(r[0], r[1]));
        const float ls = p.smoothing, us = __fsub_rn(1.0f, ls);
        if (lane == 0) {
            p.log_ratios[2 * q] = r[0];
            p.log_ratios[2 * q + 1] = r[1];
            const float dh = __fsub_rn(__fmul_rn(ls, sigmoid(h)), __fmul_rn(us, sigmoid(-h)));
            const float c = __fmul_rn(dh, __fdiv_rn(p.beta, norm));
            p.coef[2 * q] = c;
            p.coef[2 * q + 1] = -c;
            sums[0] += __fadd_rn(__fmul_rn(us, softplus(-h)), __fmul_rn(ls, softplus(h)));
            sums[1] += h;
            sums[2] += h > 0.0f ? 1.0 : 0.0;
        }
    }
    for (int k = 0; k < 3; ++k) {
        const double s = block_sum(lane == 0 ? sums[k] : 0.0);
        if (threadIdx.x == 0) {
            a.ws->total[k] += s;
            if (p.last)
                a.stats[k] = __double2float_rn(__ddiv_rn(a.ws->total[k], static_cast<double>(norm)));
        }
    }
}

template <int GT>
__global__ void __launch_bounds__(kRowThreads)
    preference_backward(const TokenArgs a, const PreferenceArgs p,
                        const __grid_constant__ PairTable t) {
    pdl_enter();
    const float out_scale =
        a.loss_scale != nullptr ? __fmul_rn(a.grad_scale, __ldg(a.loss_scale)) : a.grad_scale;
    const int row0 = t.start[0], rows = t.start[2 * t.pairs] - row0;
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t i = row0 + r;
        char* g = const_cast<char*>(row_of<GT>(a.grad, i, a.g_stride));
        const float w = a.w != nullptr ? a.w[i] : 1.0f;
        if (w == 0.0f) {
            row_zero<GT>(g, a.v);
            continue;
        }
        const float c = __fmul_rn(__fmul_rn(p.coef[find_sequence(t, static_cast<int>(i))], w),
                                  out_scale);
        row_grad<GT>(row_of<GT>(a.x, i, a.x_stride), g, a.v, token_id(a, i), p.row_max[i],
                     p.row_inv[i], c);
    }
}

int row_blocks(int64_t rows) {
    const int64_t most = 2 * static_cast<int64_t>(device_sms());
    const int64_t cap = most < kLossMaxBlocks ? most : kLossMaxBlocks;
    return static_cast<int>(rows < 1 ? 1 : rows < cap ? rows : cap);
}

template <int GT>
cudaError_t go_policy(const TokenArgs& a, const PolicyArgs& p, cudaStream_t s) {
    return launch_after(policy_rows<GT>, dim3(row_blocks(a.n)), dim3(kRowThreads), 0, s, a, p);
}
template <int GT>
cudaError_t go_pref(const TokenArgs& a, const PreferenceArgs& p, const PairTable& t, bool back,
                    cudaStream_t s) {
    const dim3 grid(row_blocks(t.start[2 * t.pairs] - t.start[0]));
    return back ? launch_after(preference_backward<GT>, grid, dim3(kRowThreads), 0, s, a, p, t)
                : launch_after(preference_forward<GT>, grid, dim3(kRowThreads), 0, s, a, p, t);
}
cudaError_t pref(const TokenArgs& a, const PreferenceArgs& p, const PairTable& t, int dtype,
                 bool back, cudaStream_t s) {
    const cudaError_t e = dtype == kGradF32   ? go_pref<kGradF32>(a, p, t, back, s)
                          : dtype == kGradF16 ? go_pref<kGradF16>(a, p, t, back, s)
                                              : go_pref<kGradBF16>(a, p, t, back, s);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_policy_loss(const TokenArgs& a, const PolicyArgs& p, int dtype,
                               cudaStream_t stream) {
    const cudaError_t e = dtype == kGradF32   ? go_policy<kGradF32>(a, p, stream)
                          : dtype == kGradF16 ? go_policy<kGradF16>(a, p, stream)
                                              : go_policy<kGradBF16>(a, p, stream);
    note_launch();
    return e;
}
cudaError_t launch_preference_forward(const TokenArgs& a, const PreferenceArgs& p,
                                      const PairTable& t, int dtype, cudaStream_t stream) {
    return pref(a, p, t, dtype, false, stream);
}
cudaError_t launch_preference_backward(const TokenArgs& a, const PreferenceArgs& p,
                                       const PairTable& t, int dtype, cudaStream_t stream) {
    return pref(a, p, t, dtype, true, stream);
}

}  // namespace shardstep
