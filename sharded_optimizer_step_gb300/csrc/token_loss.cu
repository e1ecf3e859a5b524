// Losses over a language model's logits, forward and backward: the clipped
// policy loss with a KL term and the preference loss of paired sequences.
//
// With x a token's logits and y its id, the row's exponentials refer to the
// id's own logit, rounded to a whole power of two: e_j = 2^(x_j log2 e - R),
// R = rint(x_y log2 e).  Their sum S is at least about 1 (the id's own term),
// no maximum has to be known before the first term, and the log probability
// a = ln 2 (x_y log2 e - R) - log S is formed from small numbers.  Where that
// range does not do (S past 2^120, x_y infinite or huge, a NaN) the row is
// summed again against its true maximum, which is subtracted before anything
// is scaled, so rows of the type's lowest value and rows with -inf are right.
// Both losses have d loss / d x = c (1[y] - softmax x) with one c per row.
// Statistics, terms and coefficients are fp32, sums over tokens two floats within a
// block and double from block to block; the gradient is rounded once, to the
// logits' type.
//
// Three kernels, all bound by the logits' and the gradient's traffic:
//   stream_forward  a forward pass: each logit is read once, nothing is kept.
//   staged_rows     policy: a row is brought into shared memory in 16 KB chunks by
//                   bulk copies, summed there, overwritten in place with the
//                   gradient and stored by bulk copies, while the next rows are on
//                   their way: each logit read once, each gradient written once.
//                   backward: the same ring without the sum, after a forward pass.
//   offset_backward  a backward pass where the gradient's rows lie at other offsets
//                   from 16-byte boundaries than the logits'.
// Which of them: the policy loss takes one pass of staged_rows where a row fits its
// 13 slots of shared memory (4096 rows of 32000 bf16 logits: 96 us against 137 in
// two passes), else stream_forward and a backward pass (2048 rows of 128256 bf16
// logits: 267 us; the same in one kernel that read a row again from L2 through
// registers: 1056).  The preference loss always takes two passes: a row's slope
// needs the sums of its whole pair.  A gradient at other offsets: 177 us for the
// policy loss of 4096 x 32000, against 96.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "pairs.cuh"
#include "tma.cuh"

namespace shardstep {
namespace {

constexpr int kRowThreads = 512;              // threads of a plain kernel's block
constexpr unsigned kFull = 0xFFFFFFFFu;
// log2 e; the same as a number of 12 bits and the rest.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eHead = 1.4423828125f;
constexpr float kLog2eTail = static_cast<float>(1.4426950408889634 - 1.4423828125);
constexpr float kLn2 = 0.6931471805599453f, kLn2Hi = 2839.0f / 4096.0f,
                kLn2Lo = static_cast<float>(0.6931471805599453 - 2839.0 / 4096.0);
constexpr float kFastLogit = 32768.0f;        // |x_y| below this: R and its products are fine
constexpr float kFastSum = 0x1p120f;
constexpr float kLargeSum = 0x1p16f;          // settle()
// Sums are weighted: see weight().
constexpr uint32_t kWeightBits = 0x3FB48362u; // 1.41025949
constexpr float kWeight = 1.410259485244751f;
constexpr float kUnweighted = 0x1.6b0dc2p-1f; // 1 / (kWeight (1 + 3.41e-8))

// Status of this device's staged loss launches (0 = no wait ran out).
__device__ unsigned int g_loss_status = 0;

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
constexpr __host__ __device__ int elem_bytes() {
    return GT == kGradF32 ? 4 : 2;
}
template <int GT>
__device__ __forceinline__ const char* row_of(const void* x, int64_t i, int64_t stride) {
    return static_cast<const char*>(x) + i * stride * elem_bytes<GT>();
}

// A sum held as two floats, each addition exact up to the low one's rounding
// (Knuth's two-sum): as good as a double here, without the double-precision
// units, of which an SM has so few that a block's worth of additions took a
// microsecond or two.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x);
        const float b = __fsub_rn(s, hi);
        const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
        lo = __fadd_rn(lo, e);
    }
    __device__ __forceinline__ void add(Sum2 x) {
        add(x.hi);
        lo = __fadd_rn(lo, x.lo);
    }
    // inf and NaN are the high part's
    __device__ __forceinline__ float value() const {
        return fabsf(hi) <= 0x1.fffffep127f ? __fadd_rn(hi, lo) : hi;
    }
    __device__ __forceinline__ double wide() const {
        return fabsf(hi) <= 0x1.fffffep127f
                   ? __dadd_rn(static_cast<double>(hi), static_cast<double>(lo))
                   : static_cast<double>(hi);
    }
};
// All lanes get the warp's sum, in a fixed order.
__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x.add(Sum2{__shfl_xor_sync(kFull, x.hi, d), __shfl_xor_sync(kFull, x.lo, d)});
    return x;
}

// The T threads that work on one row, with a named barrier of their own.
template <int T>
struct TeamShared {
    float part[2][T / 32];
    Sum2 wide[T / 32];
};
template <int T>
struct Team {
    int bar, tid;
    TeamShared<T>* sh;

    __device__ __forceinline__ void sync() const {
        if (T == 32)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(T) : "memory");
    }
    // The same, true for all where any thread passes true.
    __device__ __forceinline__ bool sync_or(bool any) const {
        if (T == 32) return __any_sync(kFull, any);
        int r;
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n"
            " selp.s32 %0, 1, 0, q;\n}\n"
            : "=r"(r)
            : "r"(static_cast<int>(any)), "r"(bar), "n"(T)
            : "memory");
        return r != 0;
    }
    // Sums and maxima over the team in a fixed order; every thread gets the
    // result.  *any: in, this thread's; out, of all threads.  `turn` alternates
    // between calls, so that one barrier per call is enough.
    __device__ __forceinline__ float sum(float x, bool* any, int turn) const {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, d));
        if (T == 32) {
            *any = __any_sync(kFull, *any);
            return x;
        }
        if ((tid & 31) == 0) sh->part[turn][tid >> 5] = x;
        *any = sync_or(*any);
        x = sh->part[turn][tid & (T / 32 - 1)];
#pragma unroll
        for (int d = T / 64; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, d));
        return x;
    }
    __device__ __forceinline__ float max(float x) const {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, d));
        sync();
        if ((tid & 31) == 0) sh->part[0][tid >> 5] = x;
        sync();
        for (int w = 0; w < T / 32; ++w) x = fmaxf(x, sh->part[0][w]);
        sync();
        return x;
    }
    __device__ __forceinline__ float sum(Sum2 x) const {
        x = warp_sum(x);
        sync();
        if ((tid & 31) == 0) sh->wide[tid >> 5] = x;
        sync();
        x = Sum2{0.0f, 0.0f};
        for (int w = 0; w < T / 32; ++w) x.add(sh->wide[w]);
        sync();
        return x.value();
    }
};

// --------------------------------------------------- a row's exponentials

// How a row's exponentials are formed: fast, 2^(x log2 e - ref); else
// 2^((x - ref) log2 e) with ref the row's maximum (0 for a row of -inf).
//
// Two errors of some 1e-8 would have one sign for all of a row's terms, so that a
// sequence's summed log ratio would gather them up (100 tokens: 2e-6, as much as a
// 32-bit log-softmax's random errors).  Neither is left, whatever the row looks like:
//   The float log2 e lacks 1.3e-8 of itself, and x (log2 e - float) is below half the
//     last place of most arguments, so it cannot be added to one.  An argument takes
//     log2 e as 12 bits and a tail: x times the 12 bits, less the reference, is
//     exact for 16-bit logits of a size that counts, and the tail's product is added
//     with one rounding.  (The tail is positive: -inf stays -inf.)
//   ex2.approx's mean relative error, measured over every float of each binade, is
//     +3.4e-8 from 1 on and -5.0e-8 below -1 (inside +0.8e-8 and -2.5e-8 at most): see
//     weight().
struct RowRef {
    float ref;
    bool fast;
};
__device__ __forceinline__ float row_arg(float x, RowRef r) {
    if (r.fast) return __fmaf_rn(x, kLog2eTail, __fmaf_rn(x, kLog2eHead, -r.ref));
    const float d = __fsub_rn(x, r.ref);
    return __fmaf_rn(d, kLog2eTail, __fmul_rn(d, kLog2eHead));
}
__device__ __forceinline__ float row_exp(float x, RowRef r) { return exp2_approx(row_arg(x, r)); }
// What the exponential of argument t counts in a row's sum: 1.41026, and one last
// place (8.45e-8 of it) more for t < 0, which levels the two mean errors.  The sum
// is 1.41026 (1 + 3.41e-8) times too large, which kUnweighted takes off the log
// probability's; the gradient's quotients carry kWeight instead.
__device__ __forceinline__ float weight(float t) {
    return __uint_as_float(kWeightBits + (__float_as_uint(t) >> 31));
}
__device__ __forceinline__ float row_term(float x, RowRef r) {
    const float t = row_arg(x, r);
    return __fmul_rn(exp2_approx(t), weight(t));
}
__device__ __forceinline__ RowRef fast_ref(float xy) {
    return RowRef{rintf(__fmul_rn(xy, kLog2e)), fabsf(xy) < kFastLogit};
}
// The id's log probability as the sum of two floats.  It is some 10 in size and
// what is wanted of it is mostly its small distance from another model's: rounded
// to one float (up to 5e-7 off), that distance summed over a short sequence was
// further from the exact one than a 32-bit log-softmax's.  log S = k log 2 + log m
// with S = 2^k m and m in [0.75, 1.5), so that the logarithm's own rounding is
// that of a number below 0.41; k times the upper 12 bits of log 2 is exact.
struct Logp {
    float hi, lo;
};
__device__ __forceinline__ Logp two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return Logp{s, fabsf(s) < INFINITY ? e : 0.0f};
}
__device__ __forceinline__ Logp row_logp(float xy, RowRef r, float sum) {
    sum = __fmul_rn(sum, kUnweighted);
    // sum is normal, or NaN, which the product keeps
    const int k = (__float_as_int(sum) - __float_as_int(0.75f)) >> 23;
    const float m = __fmul_rn(sum, __int_as_float((127 - k) << 23));
    const float minus_k = static_cast<float>(-k);
    const float big = __fmul_rn(minus_k, kLn2Hi);
    const float small = __fmaf_rn(minus_k, kLn2Lo, -logf(m));
    if (!r.fast) {
        const Logp d = two_sum(xy, -r.ref), e = two_sum(d.hi, big);
        return two_sum(e.hi, __fadd_rn(__fadd_rn(d.lo, e.lo), small));
    }
    return two_sum(big, __fmaf_rn(row_arg(xy, r), kLn2, small));
}
// lp - x.
__device__ __forceinline__ float logp_less(Logp lp, float x) {
    return __fadd_rn(__fsub_rn(lp.hi, x), lp.lo);
}

// A row's sum and what its exponentials refer to, for its gradient: a fast row's
// sum may be close to 2^120, and c / S would then lose its last bits or vanish for
// slopes that the gradient's type still holds (an id 80 below the largest logit,
// c = 1e-9: 5% off).  The exponent of a large sum moves into the reference; of a
// small one it stays, so that the id's own exponential has the bits that went into
// the sum, which own_grad takes it off.
struct RowScale {
    RowRef r;
    float sum;
};
__device__ __forceinline__ RowScale settle(RowRef r, float sum) {
    if (!r.fast || sum < kLargeSum) return RowScale{r, sum};
    const int k = (__float_as_int(sum) >> 23) - 127;
    return RowScale{RowRef{__fadd_rn(r.ref, static_cast<float>(k)), true},
                    __fmul_rn(sum, __int_as_float((127 - k) << 23))};
}

// The sum against the true maximum, from global memory: rows that the fast
// form does not cover.  The products of x - max stay in range whatever x is.
template <int GT, int T>
__device__ __forceinline__ RowScale slow_row(const char* x, int64_t v, const Team<T>& team) {
    float m = -INFINITY;
    for (int64_t j = team.tid; j < v; j += T) m = fmaxf(m, load1<GT>(x, j));
    m = team.max(m);
    const RowRef r{m == -INFINITY ? 0.0f : m, false};
    float s = 0.0f;
    for (int64_t j = team.tid; j < v; j += T) s = __fadd_rn(s, row_term(load1<GT>(x, j), r));
    bool none = false;
    team.sync();
    s = team.sum(s, &none, 0);
    team.sync();
    if (m == -INFINITY) s = NAN;   // nothing but -inf (or NaN): no distribution
    return RowScale{r, s};
}

// -------------------------------------------------------- terms of a token

// The row's id, or -1 where it lies outside the vocabulary: the token's log
// probability is then NaN, and so is the loss.
__device__ __forceinline__ int64_t token_id(const TokenArgs& a, int64_t i) {
    const int64_t y = a.ids64 ? static_cast<const int64_t*>(a.ids)[i]
                              : static_cast<const int32_t*>(a.ids)[i];
    return y >= 0 && y < a.v ? y : -1;
}
__device__ __forceinline__ float token_weight(const TokenArgs& a, int64_t i) {
    return a.w != nullptr ? a.w[i] : 1.0f;
}
__device__ __forceinline__ float out_scale(const TokenArgs& a) {
    return a.loss_scale != nullptr ? __fmul_rn(a.grad_scale, __ldg(a.loss_scale)) : a.grad_scale;
}

// One token's policy terms from its log probability:
//   u = exp(a - old); policy = -min(u A, clip(u) A); d = ref - a;
//   kl = expm1(d) - d; slope = d (policy + k kl) / d a.
struct PolicyTerms {
    float policy, kl, clipped, slope;
};
__device__ __forceinline__ PolicyTerms policy_terms(Logp lp, float old, float adv, float ref,
                                                    const PolicyArgs& p) {
    const float u = expf(logp_less(lp, old));
    const float cu = u < p.lo ? p.lo : u > p.hi ? p.hi : u;
    const float one = __fmul_rn(u, adv), two = __fmul_rn(cu, adv);
    PolicyTerms t;
    t.clipped = one > two ? 1.0f : 0.0f;
    t.policy = one > two ? -two : -one;
    t.slope = one > two ? 0.0f : -one;
    t.kl = 0.0f;
    if (p.kl != 0.0f) {
        const float d = -logp_less(lp, ref);
        const float e = expm1f(d);
        t.kl = __fsub_rn(e, d);
        t.slope = __fsub_rn(t.slope, __fmul_rn(p.kl, e));
    }
    return t;
}

// The divisor of the means: given, or the sum of the weights, which every
// team adds up by itself in the same order.
template <int T>
__device__ __forceinline__ float weight_sum(const TokenArgs& a, const Team<T>& team) {
    if (a.norm != 0.0f) return a.norm;
    if (a.w == nullptr) return static_cast<float>(a.n);
    Sum2 s{0.0f, 0.0f};
#pragma unroll 8
    for (int64_t i = team.tid; i < a.n; i += T) s.add(a.w[i]);
    return team.sum(s);
}
// The same where the block has gone over the launch's weights already: over all
// of them unless the call takes several launches.
template <int T>
__device__ __forceinline__ float weight_sum(const TokenArgs& a, const Team<T>& team, int64_t rows,
                                            float weight) {
    if (a.norm == 0.0f && a.w != nullptr && rows == a.n) return weight;
    return weight_sum(a, team);
}

// The blocks' sums (lane k's s is the block's k-th) added up by the block that
// arrives last, in a fixed order, and carried to the call's next launch or
// written as its statistics; by one warp.
__device__ __forceinline__ void join_sums(const TokenArgs& a, double s, bool first, bool last) {
    const int lane = threadIdx.x & 31;
    LossWork* ws = a.ws;
    if (lane < 4) ws->partial[blockIdx.x][lane] = s;
    __syncwarp();
    unsigned mine = 0;
    if (lane == 0) {
        __threadfence();
        mine = atomicInc(&ws->arrived, gridDim.x - 1) == gridDim.x - 1;
        __threadfence();
    }
    if (!__shfl_sync(kFull, mine, 0)) return;
    __syncwarp();
    double t[4] = {0.0, 0.0, 0.0, 0.0};
    for (unsigned b = lane; b < gridDim.x; b += 32)
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] += __ldcg(&ws->partial[b][k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t[k] += __shfl_xor_sync(kFull, t[k], d);
        if (lane == 0) {
            if (!first) t[k] += ws->total[k];
            ws->total[k] = t[k];
            if (last) a.stats[k] = __double2float_rn(t[k]);
        }
    }
}

__device__ __forceinline__ void add_policy(Sum2* sums, const PolicyTerms& t, const PolicyArgs& p,
                                           float k) {
    sums[0].add(__fmul_rn(k, __fadd_rn(t.policy, __fmul_rn(p.kl, t.kl))));
    sums[1].add(__fmul_rn(k, t.policy));
    sums[2].add(__fmul_rn(k, t.kl));
    sums[3].add(__fmul_rn(k, t.clipped));
}

// The sequence of the launch that row i belongs to.
template <class Table>
__device__ __forceinline__ int find_sequence(const Table& t, int64_t i) {
    int lo = 0, hi = 2 * t.pairs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.start[mid] <= i) lo = mid;
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

// A pair's loss and slope from its tokens' terms, added up in a fixed order by
// one warp.
template <class Table>
__device__ __forceinline__ void finish_pair(const TokenArgs& a, const PreferenceArgs& p,
                                            const Table& t, int q) {
    const int lane = threadIdx.x & 31;
    Sum2 r[2];
    for (int h = 0; h < 2; ++h) {
        Sum2 s{0.0f, 0.0f};
        const unsigned end = t.start[2 * q + h + 1];
        // unsigned: i may pass 2^31
        for (unsigned i = t.start[2 * q + h] + lane; i < end; i += 8 * 32) {
            float x[8];          // in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = i + 32 * k < end ? __ldcg(p.term + i + 32 * k) : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s.add(x[k]);
        }
        r[h] = warp_sum(s);
    }
    if (lane != 0) return;
    p.log_ratios[2 * q] = r[0].value();
    p.log_ratios[2 * q + 1] = r[1].value();
    r[0].add(Sum2{-r[1].hi, -r[1].lo});          // rounded after the difference
    const float h = __fmul_rn(p.beta, r[0].value());
    const float ls = p.smoothing, us = __fsub_rn(1.0f, ls);
    const float dh = __fsub_rn(__fmul_rn(ls, sigmoid(h)), __fmul_rn(us, sigmoid(-h)));
    const float c = __fmul_rn(dh, __fdiv_rn(p.beta, a.norm));
    p.coef[2 * q] = c;
    p.coef[2 * q + 1] = -c;
    a.ws->pair_loss[q][0] = __fadd_rn(__fmul_rn(us, softplus(-h)), __fmul_rn(ls, softplus(h)));
    a.ws->pair_loss[q][1] = h;
    a.ws->pair_loss[q][2] = h > 0.0f ? 1.0 : 0.0;
}

// The pairs that a block's rows completed, to be finished at its end by all of
// its warps: the last rows of a launch complete most pairs at once, and one warp
// would take them one after the other (16 pairs of 500 tokens: 40 us).
struct ReadyPairs {
    int n;
    int pair[kPairsPerLaunch];
};
// Each lane has written the words of one more row of its pair q (-1: none): the
// lane that brings a pair's count to its rows notes the pair.
template <class Table>
__device__ __forceinline__ void rows_done(const TokenArgs& a, const Table& t, int q,
                                          ReadyPairs* ready) {
    // lanes of one pair count as one, by the pair's lowest lane
    const unsigned same = __match_any_sync(kFull, q);
    const bool leads = q >= 0 && __ffs(same) - 1 == static_cast<int>(threadIdx.x & 31);
    __syncwarp();
    if (!leads) return;
    unsigned before;
    const unsigned rows = __popc(same);
    __threadfence();
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                 : "=r"(before)
                 : "l"(&a.ws->rows_done[q]), "r"(rows)
                 : "memory");
    if (before + rows == static_cast<unsigned>(t.start[2 * q + 2] - t.start[2 * q])) {
        a.ws->rows_done[q] = 0;
        ready->pair[atomicAdd(&ready->n, 1)] = q;
    }
}

// Pairs without a token, which no row finishes.
template <class Table>
__device__ __forceinline__ void empty_pairs(const TokenArgs& a, const PreferenceArgs& p,
                                            const Table& t) {
    for (int q = blockIdx.x; q < t.pairs; q += gridDim.x)
        if (t.start[2 * q + 2] == t.start[2 * q]) finish_pair(a, p, t, q);
}

// The pairs' losses, added up by the last block in pair order per lane.
// Every thread of the block calls it.
template <class Table>
__device__ __forceinline__ void preference_stats(const TokenArgs& a, const PreferenceArgs& p,
                                                 const Table& t) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicInc(&a.ws->arrived, gridDim.x - 1) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    for (int k = 0; k < 3; ++k) {
        double s = 0.0;
        for (int q = threadIdx.x; q < t.pairs; q += 32) s += __ldcg(&a.ws->pair_loss[q][k]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        if (threadIdx.x == 0) {
            s += p.first ? 0.0 : a.ws->total[k];
            a.ws->total[k] = s;
            if (p.last) a.stats[k] = __double2float_rn(__ddiv_rn(s, static_cast<double>(a.norm)));
        }
    }
}

// What a backward pass of its own needs of a row; a negative sum marks the slow
// form.
__device__ __forceinline__ void save_row(const PreferenceArgs& p, int64_t i, RowRef r, float sum) {
    const RowScale s = settle(r, sum);
    p.row_ref[i] = s.r.ref;
    p.row_sum[i] = r.fast ? s.sum : -s.sum;
}
// c: the slope of the row's sequence times its weight, or what the policy loss's
// forward pass has left.
__device__ __forceinline__ float row_coef(const PreferenceArgs& p, int64_t i, float w,
                                          float scale) {
    const float c = p.coef != nullptr ? __fmul_rn(p.coef[p.seq[i]], w) : p.term[i];
    return __fmul_rn(c, scale);
}

// The id's own gradient, c (1 - e_y / S), as (c / S) (S - e_y) with its weighted
// term of the sum: the difference is that of the other tokens' terms, and exactly 0
// where there are none.  Of another token with exponential e: -(e kWeight) c / S.
__device__ __forceinline__ float own_grad(float x, RowRef r, float sum, float cs) {
    return __fmul_rn(__fsub_rn(sum, row_term(x, r)), cs);
}

// ------------------------------------------------------- shares of the rows

// The rows of a launch are dealt out to `units` (blocks, or teams of warps): the
// live rows in turn, and the rows of weight 0, which cost less or nothing, in
// turn after them.  Dealt out by their index alone, the 30% masked rows of 4096
// left some blocks with a quarter more live rows than others.  Every block finds
// its own share by going over all weights in the same order; the host keeps a
// launch below kShareRows rows per SM so that the shares fit shared memory.
struct Share {
    const uint32_t* live;     // row - begin; null (no weights): first + j * units
    const uint32_t* dead;
    int n_live, n_dead;
    int64_t begin, first, units;
    bool backwards;           // the live rows from the last to the first

    __device__ __forceinline__ int64_t row(int j) const {
        if (backwards) j = n_live - 1 - j;
        return live != nullptr ? begin + live[j] : first + j * units;
    }
    __device__ __forceinline__ int64_t dead_row(int j) const { return begin + dead[j]; }
};
// How many of n things dealt out in turn unit u gets.
__device__ __forceinline__ int dealt(int64_t n, int64_t u, int64_t units) {
    return static_cast<int>(n > u ? (n - u + units - 1) / units : 0);
}
// What a block finds on its way over the weights.
struct Dealt {
    int n_live, n_dead;       // of the launch
    float weight;             // the sum of the launch's weights
};
// Of the things of one kind that a thread has found, the set bits of `rows` with
// ranks from `rank` on, those dealt to block b go to its list: a rank goes to the
// blocks in turn, then to each block's teams in turn, so that a row's block is the
// same whatever the number of teams.  The block's rank is looked for, not each
// row's block: one division per thread.
__device__ __forceinline__ void take_share(unsigned rows, unsigned rank, unsigned row0, unsigned b,
                                           unsigned teams, uint32_t* list) {
    const unsigned end = rank + __popc(rows);
    unsigned q = rank > b ? (rank - b + gridDim.x - 1) / gridDim.x : 0;
    for (unsigned mine = b + q * gridDim.x; mine < end; mine += gridDim.x, ++q) {
        unsigned left = rows;
        for (unsigned k = rank; k < mine; ++k) left &= left - 1;
        list[q % teams * (kShareRows / teams) + q / teams] = row0 + __ffs(left) - 1;
    }
}
// Fills the lists of the block's teams, each of up to kShareRows / teams rows;
// every thread of the block calls it.  A warp takes 8 times 32 consecutive rows
// at a time, and its lanes 0-7 and 8-15 look among these for the block's live and
// masked ones; the next weights are on their way meanwhile.
template <int THREADS>
__device__ __forceinline__ Dealt deal_rows(const TokenArgs& a, int64_t begin, int64_t end,
                                           unsigned teams, uint32_t* live, uint32_t* dead) {
    constexpr int kWarps = THREADS / 32, kGroups = 8, kStep = THREADS * kGroups;
    __shared__ unsigned counts[2][kWarps];
    __shared__ Sum2 sums[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane % kGroups;
    const unsigned n = static_cast<unsigned>(end - begin);
    unsigned live_before = 0;
    Sum2 weight{0.0f, 0.0f};
    float w[kGroups];
    const auto fetch = [&](unsigned base) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const unsigned r = base + 32 * (kGroups * warp + k) + lane;
            w[k] = r < n ? a.w[begin + r] : 0.0f;
        }
    };
    fetch(0);
    int turn = 0;
    for (unsigned base = 0; base < n; base += kStep, turn ^= 1) {
        unsigned alive = 0, before = 0, own = 0;   // this lane's group; live rows of the warp
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const unsigned m = __ballot_sync(kFull, w[k] != 0.0f);
            if (k == group) {
                alive = m;
                before = own;
            }
            own += __popc(m);
            weight.add(w[k]);
        }
        fetch(base + kStep);
        if (lane == 0) counts[turn][warp] = own;
        __syncthreads();
        const unsigned c = lane < kWarps ? counts[turn][lane] : 0;
        const unsigned below = __reduce_add_sync(kFull, lane < warp ? c : 0);
        const unsigned total = __reduce_add_sync(kFull, c);
        const unsigned row0 = base + 32 * (kGroups * warp + group);
        const unsigned here = row0 < n ? n - row0 : 0;
        const unsigned rank = live_before + below + before;
        if (lane < kGroups)
            take_share(alive, rank, row0, blockIdx.x, teams, live);
        else if (lane < 2 * kGroups)
            take_share(~alive & (here < 32 ? (1u << here) - 1 : kFull), row0 - rank, row0,
                       gridDim.x - 1 - blockIdx.x, teams, dead);
        live_before += total;
    }
    weight = warp_sum(weight);
    if (lane == 0) sums[warp] = weight;
    __syncthreads();
    weight = lane < kWarps ? sums[lane] : Sum2{0.0f, 0.0f};
    return Dealt{static_cast<int>(live_before),
                 static_cast<int>(end - begin) - static_cast<int>(live_before),
                 warp_sum(weight).value()};
}
// The share of the block's team `team` of `teams`.  The rows of weight 0 are
// dealt out from the last block down, so that the blocks with a live row more get
// one of them less.
__device__ __forceinline__ Share share_of(const TokenArgs& a, int64_t begin, int64_t end, int team,
                                          int teams, const Dealt& found, const uint32_t* live,
                                          const uint32_t* dead) {
    const int64_t blocks = gridDim.x, units = blocks * teams;
    const int64_t u = team * blocks + blockIdx.x, down = team * blocks + blocks - 1 - blockIdx.x;
    if (a.w == nullptr)
        return Share{nullptr, nullptr, dealt(end - begin, u, units), 0, begin, begin + u, units,
                     false};
    return Share{live,  dead,  dealt(found.n_live, u, units), dealt(found.n_dead, down, units),
                 begin, begin, units, false};
}

// ------------------------------------------------------ the staged kernels

constexpr int kChunk = 16384;                 // bytes of a chunk, of a slot
constexpr int kSlots = 13;                    // slots of the ring: 208 KB
constexpr int kZeroBytes = 4096;
constexpr size_t kStagedSmem =
    static_cast<size_t>(kSlots) * kChunk + kZeroBytes + 8 * kShareRows;

enum class Pass { kPolicy, kBackward };

// A row's bytes: `head` elements up to the first 16-byte boundary, `body` bytes
// in whole 16-byte vectors from there, `tail` elements after them (a row
// without a whole vector is all head).
struct RowBytes {
    const char* body_at;
    uint32_t body;
    int head, tail;
};
template <int GT>
__device__ __forceinline__ RowBytes row_bytes(const char* row, int64_t v) {
    constexpr int es = elem_bytes<GT>();
    const uintptr_t a = reinterpret_cast<uintptr_t>(row), b = a + v * es;
    const uintptr_t a16 = (a + 15) & ~uintptr_t{15}, b16 = b & ~uintptr_t{15};
    if (b16 <= a16) return RowBytes{row, 0, static_cast<int>(v), 0};
    return RowBytes{row + (a16 - a), static_cast<uint32_t>(b16 - a16),
                    static_cast<int>((a16 - a) / es), static_cast<int>((b - b16) / es)};
}

__device__ __forceinline__ Pair exp2_pair(Pair t) {
    const float2 f = floats(t);
    return make_pair(exp2_approx(f.x), exp2_approx(f.y));
}

// The k-th pair of a 16-byte vector as floats, and back.
template <int GT>
constexpr __host__ __device__ int vec_pairs() {
    return 16 / elem_bytes<GT>() / 2;
}
template <int GT>
__device__ __forceinline__ Pair pair_of(const uint4& u, int k) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (GT == kGradF32) {
        return make_pair(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    } else if constexpr (GT == kGradF16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        return make_pair(f.x, f.y);
    } else {
        return make_pair(bf16_lo(w[k]), bf16_hi(w[k]));
    }
}
template <int GT>
__device__ __forceinline__ uint32_t pack_pair(Pair p) {
    const float2 x = floats(p);
    if constexpr (GT == kGradF16) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(x.x, x.y);
}

// The constants of a row's fast exponentials, both halves alike.
struct FastRow {
    Pair head, tail, neg_ref;
};
__device__ __forceinline__ FastRow fast_row(RowRef r) {
    return FastRow{make_pair(kLog2eHead, kLog2eHead), make_pair(kLog2eTail, kLog2eTail),
                   make_pair(-r.ref, -r.ref)};
}
__device__ __forceinline__ Pair fast_args(Pair x, const FastRow& r) {
    return fma2(x, r.tail, fma2(x, r.head, r.neg_ref));
}
// A row's fast sum, in two chains.
struct RowSum {
    Pair acc[2];
};
template <int GT>
__device__ __forceinline__ void sum_vector(const uint4& u, const FastRow& r, RowSum* s) {
#pragma unroll
    for (int k = 0; k < vec_pairs<GT>(); ++k) {
        const Pair t = fast_args(pair_of<GT>(u, k), r);
        const float2 f = floats(t);
        s->acc[k & 1] = fma2(exp2_pair(t), make_pair(weight(f.x), weight(f.y)), s->acc[k & 1]);
    }
}
__device__ __forceinline__ float row_total(const RowSum& s) {
    const float2 a = floats(add2(s.acc[0], s.acc[1]));
    return __fadd_rn(a.x, a.y);
}
// A vector's gradient without the id's own term, e f.
template <int GT>
__device__ __forceinline__ uint4 pack_vector(const Pair* o) {
    if constexpr (GT == kGradF32) {
        const float2 a = floats(o[0]), b = floats(o[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                          __float_as_uint(b.y));
    } else {
        return make_uint4(pack_pair<GT>(o[0]), pack_pair<GT>(o[1]), pack_pair<GT>(o[2]),
                          pack_pair<GT>(o[3]));
    }
}
template <int GT>
__device__ __forceinline__ uint4 grad_vector(const uint4& u, const FastRow& r, Pair f) {
    Pair o[vec_pairs<GT>()];
#pragma unroll
    for (int k = 0; k < vec_pairs<GT>(); ++k) {
        o[k] = mul2(exp2_pair(fast_args(pair_of<GT>(u, k), r)), f);
    }
    return pack_vector<GT>(o);
}
template <int GT>
__device__ __forceinline__ uint4 grad_vector_slow(const uint4& u, RowRef r, Pair f) {
    Pair o[vec_pairs<GT>()];
#pragma unroll
    for (int k = 0; k < vec_pairs<GT>(); ++k) {
        const float2 x = floats(pair_of<GT>(u, k));
        o[k] = mul2(make_pair(row_exp(x.x, r), row_exp(x.y, r)), f);
    }
    return pack_vector<GT>(o);
}

// ------------------------------------- the backward pass at other offsets

// The 16 bytes that begin `shift` elements into lo, of lo and hi in turn.
template <int GT>
__device__ __forceinline__ uint4 join_vectors(const uint4& lo, const uint4& hi, int shift) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int words = GT == kGradF32 ? shift : shift >> 1;
    if (words & 2)
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    if (words & 1)
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    if (GT != kGradF32 && (shift & 1))
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Elements [from, to) of a vector, one by one.
template <int GT>
__device__ __forceinline__ void store_some(char* at, const uint4& o, int from, int to) {
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int e = 0; e < 16 / elem_bytes<GT>(); ++e) {
        if (e < from || e >= to) continue;
        if constexpr (GT == kGradF32)
            reinterpret_cast<uint32_t*>(at)[e] = w[e];
        else
            reinterpret_cast<uint16_t*>(at)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2)));
    }
}
// Element e of a vector replaced by x.
template <int GT>
__device__ __forceinline__ uint4 with_element(const uint4& o, int e, float x) {
    uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (GT == kGradF32) {
            if (e == k) w[k] = __float_as_uint(x);
        } else {
            const uint32_t bits = pack_pair<GT>(make_pair(x, 0.0f)) & 0xFFFFu;
            if (e == 2 * k) w[k] = (w[k] & 0xFFFF0000u) | bits;
            if (e == 2 * k + 1) w[k] = (w[k] & 0xFFFFu) | bits << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The gradient, c (1[y] - e / S), of rows whose forward pass has left S, where
// gradient and logits lie at different offsets from 16-byte boundaries, so that a
// staged row's bytes cannot be stored back in bulk.  A lane forms the gradient of
// a whole vector of logits; with the next lane's it holds the 16 bytes between two
// boundaries of the gradient's row.  What a warp's 32 vectors do not fill goes out
// one element at a time.  Bound by memory and the loads' latency: 4096 rows of 32000
// bf16 logits in 127 us, 4.1 TB/s (206 us with every element loaded and stored by
// itself).
template <int GT>
__global__ void __launch_bounds__(kRowThreads, 2)
    offset_backward(const TokenArgs a, const PreferenceArgs p, int64_t begin, int64_t end) {
    constexpr int es = elem_bytes<GT>(), kElems = 16 / es, kStep = kRowThreads, U = 4;
    pdl_enter();
    const float scale = out_scale(a);
    const int lane = threadIdx.x & 31;
    for (int64_t i = begin + blockIdx.x; i < end; i += gridDim.x) {
        char* g = const_cast<char*>(row_of<GT>(a.grad, i, a.g_stride));
        const float w = token_weight(a, i);
        if (w == 0.0f) {
            const RowBytes b = row_bytes<GT>(g, a.v);
            char* body = const_cast<char*>(b.body_at);
            if (threadIdx.x < b.head) store1<GT>(g, threadIdx.x, 0.0f);
            if (threadIdx.x < b.tail) store1<GT>(body + b.body, threadIdx.x, 0.0f);
            for (uint32_t at = 16 * threadIdx.x; at < b.body; at += 16 * kStep)
                __stcs(reinterpret_cast<uint4*>(body + at), make_uint4(0, 0, 0, 0));
            continue;
        }
        const char* x = row_of<GT>(a.x, i, a.x_stride);
        const RowBytes b = row_bytes<GT>(x, a.v);
        const int64_t y = token_id(a, i);
        const float sum = p.row_sum[i], s = fabsf(sum);
        const RowRef r{p.row_ref[i], !(sum < 0.0f)};
        const float cs = __fdiv_rn(row_coef(p, i, w, scale), s), other = -__fmul_rn(cs, kWeight);
        const FastRow fr = fast_row(r);
        const Pair f = make_pair(other, other);
        if (threadIdx.x < 32) {           // the elements outside whole vectors
            int64_t edge = -1;
            if (lane < 16 && lane < b.head) edge = lane;
            if (lane >= 16 && lane - 16 < b.tail) edge = a.v - b.tail + lane - 16;
            if (edge >= 0) {
                const float xe = load1<GT>(x, edge);
                store1<GT>(g, edge, edge == y ? own_grad(xe, r, s, cs)
                                              : __fmul_rn(row_exp(xe, r), other));
            }
        }
        char* to = g + b.head * es;       // the first whole vector's gradient
        const int shift =
            static_cast<int>((16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15) / es;
        const int n = static_cast<int>(b.body / 16);
        const int64_t yv = y >= b.head ? (y - b.head) / kElems : -1;
        for (int v0 = threadIdx.x - lane; v0 < n; v0 += U * kStep) {
            uint4 u[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = v0 + k * kStep + lane;
                u[k] = at < n ? ldcs16(reinterpret_cast<const uint4*>(b.body_at) + at)
                              : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = v0 + k * kStep + lane;
                if (at - lane >= n) break;
                uint4 o = r.fast ? grad_vector<GT>(u[k], fr, f) : grad_vector_slow<GT>(u[k], r, f);
                if (at == yv)
                    o = with_element<GT>(o, static_cast<int>((y - b.head) % kElems),
                                         own_grad(load1<GT>(x, y), r, s, cs));
                const uint4 next{__shfl_down_sync(kFull, o.x, 1), __shfl_down_sync(kFull, o.y, 1),
                                 __shfl_down_sync(kFull, o.z, 1), __shfl_down_sync(kFull, o.w, 1)};
                char* dst = to + static_cast<int64_t>(at) * 16;
                if (shift == 0 ? at < n : lane < 31 && at + 1 < n)
                    __stcs(reinterpret_cast<uint4*>(dst + shift * es),
                           join_vectors<GT>(o, next, shift));
                else if (at < n)
                    store_some<GT>(dst, o, shift, kElems);
                if (lane == 0) store_some<GT>(dst, o, 0, shift);
            }
        }
    }
}

__device__ __forceinline__ void st_release(unsigned* p, unsigned x) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_addr(p)), "r"(x) : "memory");
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned x;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(smem_addr(p)) : "memory");
    return x;
}

// The ring's position: the slot of the next chunk, its barriers' parity and the
// chunk's number since the start.
struct Ring {
    int slot;
    uint32_t parity;
    unsigned chunk;
    __device__ __forceinline__ void next() {
        ++chunk;
        if (++slot == kSlots) {
            slot = 0;
            parity ^= 1u;
        }
    }
    // any number: a row of the backward pass may be longer than the ring
    __device__ __forceinline__ void skip(uint32_t chunks) {
        chunk += chunks;
        slot = static_cast<int>(chunk % kSlots);
        parity = chunk / kSlots & 1u;
    }
};

// What the computing warps need of a row besides its logits.
struct RowParam {
    float w;        // 0: the row takes no part
    int32_t y;      // the id, -1 outside the vocabulary
    float xy;       // its logit (policy)
    float f[3];     // policy: old, advantage, ref;
                    // backward: c, the reference and the sum of the exponentials
};
constexpr int kBatch = 32;            // rows whose parameters are fetched at once

// The parameters of live row i; the caller's lanes take a row each, so the
// dependent loads of 32 rows overlap.
template <int GT>
__device__ __forceinline__ RowParam policy_param(const TokenArgs& a, const PolicyArgs& pol,
                                                 int64_t i) {
    const int64_t y = token_id(a, i);
    RowParam q{token_weight(a, i), static_cast<int32_t>(y), NAN, {pol.old[i], pol.adv[i], 0.0f}};
    if (pol.kl != 0.0f) q.f[2] = a.ref[i];
    if (y >= 0) q.xy = load1<GT>(row_of<GT>(a.x, i, a.x_stride), y);
    return q;
}

// Until chunk r.chunk has landed.  A team skips the other team's rows, so it may
// ask for a slot whose earlier copy is still on its way: a parity alone would
// then say yes to the copy before that.  It first waits for its own chunk to be
// issued, which the slot's earlier use has to be over for; from there on the
// parity is that of its chunk.  `seen`: the issued count this thread last read.
__device__ __forceinline__ bool wait_chunk(uint64_t* full, const unsigned* issued, unsigned* seen,
                                           const Ring& r, unsigned long long limit_ns) {
    if (static_cast<int>(*seen - r.chunk) <= 0) {
        *seen = ld_acquire(issued);
        if (static_cast<int>(*seen - r.chunk) <= 0) {
            const unsigned long long t0 = now_ns();
            do {
                if (now_ns() - t0 > limit_ns) return false;
                *seen = ld_acquire(issued);
            } while (static_cast<int>(*seen - r.chunk) <= 0);
        }
    }
    return mbar_wait(&full[r.slot], r.parity, limit_ns);
}

// A row of weight 0 of the gradient, by one warp, from `zeros`.
template <int GT>
__device__ __forceinline__ void zero_row(const TokenArgs& a, int64_t i, const uint8_t* zeros) {
    const int lane = threadIdx.x & 31;
    char* g = const_cast<char*>(row_of<GT>(a.grad, i, a.g_stride));
    const RowBytes b = row_bytes<GT>(g, a.v);
    char* dst = const_cast<char*>(b.body_at);
    if (lane < b.head) store1<GT>(g, lane, 0.0f);
    if (lane < b.tail) store1<GT>(dst + b.body, lane, 0.0f);
    if (lane == 0) {
        const uint64_t once = evict_first();
        for (uint32_t o = 0; o < b.body; o += kZeroBytes)
            bulk_store(dst + o, zeros, b.body - o < kZeroBytes ? b.body - o : kZeroBytes, once);
        bulk_commit();
        bulk_wait_read<1>();
    }
}

// One block per SM takes its share of the launch's rows.
//   2 teams of 8 computing warps, live rows in turn: sum a row's chunks as they
//     land, join, form the row's terms, then overwrite the chunks with the
//     gradient; the up to 15 + 7 elements outside whole vectors stay in the
//     registers of the team's first warp.  While one team joins its sum and
//     forms its terms the other has the arithmetic units;
//   loading warp: per live row, its body's chunks into free slots;
//   storing warp: stores each finished chunk and frees its slot;
//   zero warp: the rows of weight 0, from a zeroed piece of shared memory;
//   parameter warp: the rows' weights, ids, logits of the ids and so on, 32
//     rows ahead at a time; at the end it joins the blocks' sums, while the last
//     rows are still being stored.
// Every wait is bounded: one that runs out sets a status bit, the block leaves at
// the end of the row, and its copies in flight are waited for first.
// Bound by the logits' read and the gradient's write.  Policy, with gradient: 4096
// rows of 32000 bf16 logits, 30% masked, 81.4 us, 5.5 TB/s; 8192 rows of 50257, 25%
// masked, 233 us, 6.2 TB/s.  Backward: 8111 rows of 32000, 30% masked, 149 us, 5.9
// TB/s.
// Loads and stores are evict-first, chosen on the kernel's own time (4096 x 32000: 83
// us against 86).  The gradient's next reader loses little by it if it is a matrix
// product (with 1024 columns after 152 to 2048 rows of 32000: the two take 26.9 to
// 135.1 us, with plain stores 26.8 to 134.8), more if it is bound by memory (a sum
// after 1024 rows: 57.6 against 49.5).
constexpr int kTeams = 2;
constexpr int kTeamThreads = 256, kTeamWarps = kTeamThreads / 32;
constexpr int kWorkWarps = kTeams * kTeamWarps;
constexpr int kLoadWarp = kWorkWarps, kStoreWarp = kWorkWarps + 1, kParamWarp = kWorkWarps + 2,
              kZeroWarp = kWorkWarps + 3;
constexpr int kStagedThreads = 32 * (kWorkWarps + 4);

template <int GT, Pass M>
__global__ void __launch_bounds__(kStagedThreads, 1)
    staged_rows(const TokenArgs a, const PolicyArgs pol, const PreferenceArgs p,
                int64_t begin, int64_t end, bool first_launch, bool last_launch,
                unsigned long long wait_ns) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ TeamShared<kTeamThreads> sh[kTeams];
    __shared__ double team_sums[kTeams][4];
    __shared__ uint64_t full[kSlots], done[kSlots], empty[kSlots];
    __shared__ unsigned issued_chunks;    // by the loading warp so far
    __shared__ unsigned stored_rows;      // by the storing warp so far
    __shared__ uint64_t param_full[2], param_empty[2], sums_full;
    __shared__ RowParam params[2][kBatch];
    uint8_t* zeros = smem + static_cast<size_t>(kSlots) * kChunk;
    uint32_t* live_list = reinterpret_cast<uint32_t*>(zeros + kZeroBytes);
    uint32_t* dead_list = live_list + kShareRows;
    constexpr int es = elem_bytes<GT>();
    constexpr bool kPolicy = M == Pass::kPolicy;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        issued_chunks = 0;
        stored_rows = 0;
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], kTeamWarps);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&param_full[s], 1);
            mbar_init(&param_empty[s], kWorkWarps);
        }
        mbar_init(&sums_full, kTeams);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int k = tid; k < kZeroBytes / 4; k += kStagedThreads)
        reinterpret_cast<uint32_t*>(zeros)[k] = 0;
    fence_async();
    __syncthreads();
    pdl_enter();
    Dealt found{0, 0, 0.0f};
    if (a.w != nullptr)
        found = deal_rows<kStagedThreads>(a, begin, end, 1, live_list, dead_list);
    Share share = share_of(a, begin, end, 0, 1, found, live_list, dead_list);
    // the backward pass after a forward pass over the same rows: those read last
    // are the ones that L2 still holds
    share.backwards = !kPolicy;
    const int rows = share.n_live;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            const uint64_t once = evict_first();
            Ring r{0, 0, 0};
            int64_t issued = 0;
            bool ok = true;
            for (int j = 0; j < rows && ok; ++j) {
                const RowBytes b = row_bytes<GT>(row_of<GT>(a.x, share.row(j), a.x_stride), a.v);
                for (uint32_t o = 0; o < b.body; o += kChunk) {
                    if (issued >= kSlots && !mbar_wait(&empty[r.slot], r.parity ^ 1u, wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t n = b.body - o < kChunk ? b.body - o : kChunk;
                    mbar_expect_tx(&full[r.slot], n);
                    bulk_load_once(smem + static_cast<size_t>(r.slot) * kChunk, b.body_at + o, n,
                                   &full[r.slot], once);
                    r.next();
                    ++issued;
                    st_release(&issued_chunks, static_cast<unsigned>(issued));
                }
            }
            if (!ok) atomicOr(&g_loss_status, kStatusProducerTimeout);
            // the last (at most kSlots) chunks land before the block may exit
            const int64_t skip = issued > kSlots ? issued - kSlots : 0;
            Ring d{static_cast<int>(skip % kSlots), static_cast<uint32_t>(skip / kSlots) & 1u, 0};
            bool drained = true;
            for (int64_t k = skip; k < issued; ++k) {
                drained = mbar_wait(&full[d.slot], d.parity, kDrainNs) && drained;
                d.next();
            }
            if (!drained) atomicOr(&g_loss_status, kStatusDrainTimeout);
        }
    } else if (warp == kStoreWarp) {
        const uint64_t once = evict_first();
        Ring r{0, 0, 0};
        bool ok = true;
        for (int j = 0; j < rows && ok; ++j) {
            char* g = const_cast<char*>(row_of<GT>(a.grad, share.row(j), a.g_stride));
            const RowBytes b = row_bytes<GT>(g, a.v);
            char* dst = const_cast<char*>(b.body_at);
            int held = -1;            // the slot of the newest store group, or none
            for (uint32_t o = 0; o < b.body; o += kChunk) {
                ok = __all_sync(kFull, mbar_wait(&done[r.slot], r.parity, wait_ns));
                if (!ok) break;
                if (lane == 0) {
                    bulk_store(dst + o, smem + static_cast<size_t>(r.slot) * kChunk,
                               b.body - o < kChunk ? b.body - o : kChunk, once);
                    bulk_commit();
                    if (held >= 0) {          // the store before this one has been read
                        bulk_wait_read<1>();
                        mbar_arrive(&empty[held]);
                    }
                }
                held = r.slot;
                r.next();
            }
            // the loading warp may want the row's last slot at once
            if (lane == 0 && held >= 0) {
                bulk_wait_read<0>();
                mbar_arrive(&empty[held]);
            }
            if (lane == 0) st_release(&stored_rows, static_cast<unsigned>(j + 1));
        }
        if (!ok && lane == 0) atomicOr(&g_loss_status, kStatusProducerTimeout);
        if (lane == 0) bulk_wait_read<0>();
    } else if (warp == kZeroWarp) {
        // spread over the live rows: written all at once at the start, they took the
        // memory from the live rows' loads, which could not catch up later (4096
        // rows of 32000, 30% masked: 92.6 us)
        const unsigned long long t0 = now_ns();
        for (int j = 0; j < share.n_dead; ++j) {
            const unsigned after =
                static_cast<unsigned>(static_cast<int64_t>(j) * rows / share.n_dead);
            while (ld_acquire(&stored_rows) < after && now_ns() - t0 < wait_ns) __nanosleep(200);
            zero_row<GT>(a, share.dead_row(j), zeros);
        }
        if (lane == 0) bulk_wait_read<0>();
    } else if (warp == kParamWarp) {
        const float scale = kPolicy ? 0.0f : out_scale(a);
        bool ok = true;
        for (int j = 0, n = 0; j < rows && ok; j += kBatch, ++n) {
            const int buf = n & 1;
            RowParam q{0.0f, -1, 0.0f, {0.0f, 0.0f, 0.0f}};
            if (j + lane < rows) {
                const int64_t i = share.row(j + lane);
                if (kPolicy) {
                    q = policy_param<GT>(a, pol, i);
                } else {
                    q.w = token_weight(a, i);
                    q.y = static_cast<int32_t>(token_id(a, i));
                    q.f[0] = row_coef(p, i, q.w, scale);
                    q.f[1] = p.row_ref[i];
                    q.f[2] = p.row_sum[i];
                }
            }
            if (n >= 2)
                ok = __all_sync(kFull, mbar_wait(&param_empty[buf],
                                                 static_cast<uint32_t>((n >> 1) - 1) & 1u,
                                                 wait_ns));
            if (!ok) break;
            params[buf][lane] = q;
            __syncwarp();
            if (lane == 0) mbar_arrive(&param_full[buf]);
        }
        if (!ok && lane == 0) atomicOr(&g_loss_status, kStatusProducerTimeout);
        if (kPolicy) {
            // the block's sums, while the last rows are still being stored
            for (int j = lane; j < share.n_dead; j += 32) a.logps[share.dead_row(j)] = 0.0f;
            const bool in = __all_sync(kFull, mbar_wait(&sums_full, 0, 4 * wait_ns));
            double s = 0.0;
            if (lane < 4)
                for (int w = 0; w < kTeams; ++w) s += team_sums[w][lane];
            if (!in && lane == 0) atomicOr(&g_loss_status, kStatusConsumerTimeout);
            join_sums(a, s, first_launch, last_launch);   // in any case: it counts the blocks
        }
    } else if (warp < kWorkWarps) {
        const int which = warp / kTeamWarps;
        const Team<kTeamThreads> team{1 + which, tid - which * kTeamThreads, &sh[which]};
        const float norm = kPolicy ? weight_sum(a, team, end - begin, found.weight) : 1.0f;
        const float scale = kPolicy ? out_scale(a) : 0.0f;
        Sum2 sums[4] = {};
        Ring ring{0, 0, 0};
        unsigned seen = 0;
        // a wait that ran out, made the same for the whole team at a barrier before
        // any of it leaves
        bool bad = false;
        int turn = 0;
        for (int j = 0; j < rows && !bad; ++j) {
            const int buf = (j / kBatch) & 1;
            if (j % kBatch == 0) {
                bad = !mbar_wait(&param_full[buf], static_cast<uint32_t>(j / (2 * kBatch)) & 1u,
                                 wait_ns);
                bad = team.sync_or(bad);
                if (bad) break;
            }
            const RowParam q = params[buf][j % kBatch];
            if (j % kBatch == kBatch - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&param_empty[buf]);
            }
            const int64_t i = share.row(j);
            const char* x = row_of<GT>(a.x, i, a.x_stride);
            const RowBytes b = row_bytes<GT>(x, a.v);
            if (j % kTeams != which) {        // the other team's
                ring.skip((b.body + kChunk - 1) / kChunk);
                continue;
            }
            // this lane's element outside the whole vectors, if any
            int64_t edge = -1;
            if (team.tid < 32) {
                if (lane < 16 && lane < b.head) edge = lane;
                if (lane >= 16 && lane - 16 < b.tail) edge = a.v - b.tail + lane - 16;
            }
            const float xe = edge >= 0 ? load1<GT>(x, edge) : 0.0f;
            RowRef r;
            float s, c;
            if (kPolicy) {
                r = fast_ref(q.xy);
                const FastRow fr = fast_row(r);
                RowSum acc{};
                Ring at_ring = ring;
                for (uint32_t o = 0; o < b.body; o += kChunk) {
                    bad = bad || !wait_chunk(full, &issued_chunks, &seen, at_ring, wait_ns);
                    const uint32_t n = b.body - o < kChunk ? b.body - o : kChunk;
                    const uint8_t* in = smem + static_cast<size_t>(at_ring.slot) * kChunk;
                    if (r.fast && !bad) {
#pragma unroll
                        for (int k = 0; k < kChunk / (16 * kTeamThreads); ++k) {
                            const uint32_t at = 16 * (k * kTeamThreads + team.tid);
                            if (at < n)
                                sum_vector<GT>(*reinterpret_cast<const uint4*>(in + at), fr, &acc);
                        }
                    }
                    at_ring.next();
                }
                s = row_total(acc);
                if (edge >= 0 && r.fast) s = __fadd_rn(s, row_term(xe, r));
                s = team.sum(s, &bad, turn);
                turn ^= 1;
                if (bad) break;
                if (!r.fast || !(s < kFastSum)) {
                    const RowScale sr = slow_row<GT>(x, a.v, team);
                    r = sr.r;
                    s = sr.sum;
                }
                const Logp lp = row_logp(q.xy, r, s);
                const PolicyTerms pt = policy_terms(lp, q.f[0], q.f[1], q.f[2], pol);
                const float k = __fdiv_rn(q.w, norm);
                c = __fmul_rn(__fmul_rn(pt.slope, k), scale);
                if (team.tid == 0) {
                    a.logps[i] = lp.hi;
                    add_policy(sums, pt, pol, k);
                }
                const RowScale settled = settle(r, s);
                r = settled.r;
                s = settled.sum;
            } else {
                c = q.f[0];
                s = fabsf(q.f[2]);
                r = RowRef{q.f[1], !(q.f[2] < 0.0f)};
            }
            const float cs = __fdiv_rn(c, s), other = -__fmul_rn(cs, kWeight);
            char* g = const_cast<char*>(row_of<GT>(a.grad, i, a.g_stride));
            // the id's place among the vectors of the body, in bytes
            const int64_t yb = q.y < b.head ? -1 : static_cast<int64_t>(q.y - b.head) * es;
            const FastRow fr = fast_row(r);
            const Pair f = make_pair(other, other);
            for (uint32_t o = 0; o < b.body; o += kChunk) {
                if (!kPolicy)
                    bad = bad || !wait_chunk(full, &issued_chunks, &seen, ring, wait_ns);
                const uint32_t n = b.body - o < kChunk ? b.body - o : kChunk;
                uint8_t* io = smem + static_cast<size_t>(ring.slot) * kChunk;
                // the id's element, if it is in this chunk: its vector's thread
                // takes the logit before and writes the gradient after the vector
                const int64_t in = yb - o;
                const bool own = in >= 0 && in < n && in / 16 % kTeamThreads == team.tid;
                const float xv = own && !bad ? load1<GT>(io, in / es) : 0.0f;
                if (r.fast && !bad) {
#pragma unroll
                    for (int k = 0; k < kChunk / (16 * kTeamThreads); ++k) {
                        const uint32_t at = 16 * (k * kTeamThreads + team.tid);
                        uint4* v4 = reinterpret_cast<uint4*>(io + at);
                        if (at < n) *v4 = grad_vector<GT>(*v4, fr, f);
                    }
                } else if (!bad) {
                    for (uint32_t at = 16 * team.tid; at < n; at += 16 * kTeamThreads) {
                        uint4* v4 = reinterpret_cast<uint4*>(io + at);
                        *v4 = grad_vector_slow<GT>(*v4, r, f);
                    }
                }
                if (own && !bad) store1<GT>(io, in / es, own_grad(xv, r, s, cs));
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&done[ring.slot]);
                ring.next();
            }
            if (edge >= 0)
                store1<GT>(g, edge, edge == q.y ? own_grad(xe, r, s, cs)
                                                : __fmul_rn(row_exp(xe, r), other));
            if (!kPolicy) bad = team.sync_or(bad);
        }
        if (bad && team.tid == 0) atomicOr(&g_loss_status, kStatusConsumerTimeout);
        if (kPolicy && team.tid == 0) {
            for (int k = 0; k < 4; ++k) team_sums[which][k] = sums[k].wide();
            mbar_arrive(&sums_full);
        }
    }
}

// ------------------------------------------------ the streaming forward pass

// A forward pass needs a row's sum alone, so no row has to stay: each of a
// block's 16 warps streams its own part of its team's row through three 4 KB
// slots of its own, lane 0 starting the next copy as soon as a slot has been
// summed.  Nothing is shared on the way; a team of W warps joins its sums once a
// row, and what follows from a row's sum is formed for 32 rows at once, a row
// per lane.  W = 16 where rows are few, so that a row's copies spread over the
// SM's warps, else 4.  Bound by the one read of the logits: 8192 rows of 50257 bf16
// logits, 25% masked, 102 us, 6.1 TB/s; 2048 rows of 32000 fp16, 10% masked, 31 us,
// 3.8 TB/s, of which some 21 us stream and the rest starts and joins.
constexpr int kStreamWarps = 16, kStreamThreads = 32 * kStreamWarps;
constexpr int kStreamSlots = 3, kStreamChunk = 4096;
constexpr size_t kStreamSmem =
    static_cast<size_t>(kStreamWarps) * kStreamSlots * kStreamChunk + 8 * kShareRows;

// The chunks of a warp's parts of its team's live rows, in order.
struct Parts {
    const char* at;      // the current row's part
    uint32_t len, off;   // its bytes; those already taken
    int row;             // the next row of the share
};

// The policy loss's stand-in for a table of pairs.
struct NoTable {
    int32_t pairs;
};
template <int GT, int W, class Table>
__global__ void __launch_bounds__(kStreamThreads, 1)
    stream_forward(const TokenArgs a, const PolicyArgs pol, const PreferenceArgs p,
                   const __grid_constant__ Table t, int64_t begin, int64_t end, bool first_launch,
                   bool last_launch, unsigned long long wait_ns) {
    constexpr bool PREF = !std::is_same<Table, NoTable>::value;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kRowTeams = kStreamWarps / W;
    __shared__ TeamShared<32 * W> sh[kRowTeams];
    __shared__ TeamShared<kStreamThreads> block_sh;
    __shared__ double team_sums[kRowTeams][4];
    __shared__ uint64_t full[kStreamWarps][kStreamSlots];
    __shared__ ReadyPairs ready;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int which = warp / W, part = warp % W;
    const Team<32 * W> team{1 + which, tid - which * 32 * W, &sh[which]};
    uint8_t* slots = smem + static_cast<size_t>(warp) * kStreamSlots * kStreamChunk;
    uint32_t* live_list = reinterpret_cast<uint32_t*>(
        smem + static_cast<size_t>(kStreamWarps) * kStreamSlots * kStreamChunk);
    uint32_t* dead_list = live_list + kShareRows;
    if (tid == 0) ready.n = 0;
    if (lane == 0) {
        for (int s = 0; s < kStreamSlots; ++s) mbar_init(&full[warp][s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_enter();
    Dealt found{0, 0, 0.0f};
    if (a.w != nullptr)
        found = deal_rows<kStreamThreads>(a, begin, end, kRowTeams, live_list, dead_list);
    const Share share = share_of(a, begin, end, which, kRowTeams, found,
                                 live_list + which * (kShareRows / kRowTeams),
                                 dead_list + which * (kShareRows / kRowTeams));
    const int rows = share.n_live;
    // this warp's part of a row's body: whole vectors, contiguous
    const auto part_of = [&](const RowBytes& b, const char** at) {
        const uint32_t each = (b.body / 16 + W - 1) / W * 16;
        const uint32_t lo = part * each < b.body ? part * each : b.body;
        *at = b.body_at + lo;
        return b.body - lo < each ? b.body - lo : each;
    };

    Parts c{nullptr, 0, 0, 0};
    int issued = 0;
    // Starts the copy of the next chunk, if there is one, into slot s.
    const auto start_next = [&](int s) {
        while (c.off >= c.len) {
            if (c.row >= rows) return;
            const char* x = row_of<GT>(a.x, share.row(c.row++), a.x_stride);
            c.len = part_of(row_bytes<GT>(x, a.v), &c.at);
            c.off = 0;
        }
        const uint32_t n = c.len - c.off < kStreamChunk ? c.len - c.off : kStreamChunk;
        if (lane == 0) {
            mbar_expect_tx(&full[warp][s], n);
            bulk_load(slots + s * kStreamChunk, c.at + c.off, n, &full[warp][s]);
        }
        c.off += n;
        ++issued;
    };
    for (int s = 0; s < kStreamSlots; ++s) start_next(s);

    float norm = 1.0f;
    if (!PREF) norm = weight_sum(a, Team<kStreamThreads>{0, tid, &block_sh}, end - begin, found.weight);
    if constexpr (PREF) {
        if (warp == 0 && begin == t.start[0]) empty_pairs(a, p, t);
    }
    Sum2 sums[4] = {};
    int slot = 0, taken = 0, turn = 0;
    uint32_t parity = 0;
    bool bad = false;
    const auto param = [&](int j) {
        RowParam q{0.0f, -1, 0.0f, {0.0f, 0.0f, 0.0f}};
        if (j + lane >= rows) return q;
        const int64_t i = share.row(j + lane);
        if (!PREF) return policy_param<GT>(a, pol, i);
        q.w = token_weight(a, i);
        q.f[0] = a.ref[i];
        const int64_t y = token_id(a, i);
        q.xy = y >= 0 ? load1<GT>(row_of<GT>(a.x, i, a.x_stride), y) : NAN;
        return q;
    };
    RowParam mine = param(0), after = param(32);
    for (int j0 = 0; j0 < rows && !bad; j0 += 32) {
        RowRef my_ref{0.0f, true};
        float my_sum = 1.0f;
        for (int l = 0; l < 32 && j0 + l < rows && !bad; ++l) {
            const float xy = __shfl_sync(kFull, mine.xy, l);
            const char* x = row_of<GT>(a.x, share.row(j0 + l), a.x_stride);
            const RowBytes b = row_bytes<GT>(x, a.v);
            const char* unused;
            const uint32_t len = part_of(b, &unused);
            // this lane's element outside the whole vectors, if any
            int64_t edge = -1;
            if (part == 0) {
                if (lane < 16 && lane < b.head) edge = lane;
                if (lane >= 16 && lane - 16 < b.tail) edge = a.v - b.tail + lane - 16;
            }
            const float xe = edge >= 0 ? load1<GT>(x, edge) : 0.0f;
            RowRef r = fast_ref(xy);
            const FastRow fr = fast_row(r);
            RowSum acc{};
            for (uint32_t o = 0; o < len && !bad; o += kStreamChunk) {
                bad = !__all_sync(kFull, mbar_wait(&full[warp][slot], parity, wait_ns));
                if (bad) break;
                const uint32_t n = len - o < kStreamChunk ? len - o : kStreamChunk;
                const uint8_t* in = slots + slot * kStreamChunk;
                if (r.fast) {
                    if (n == kStreamChunk) {
#pragma unroll
                        for (int k = 0; k < kStreamChunk / 512; ++k)
                            sum_vector<GT>(*reinterpret_cast<const uint4*>(in + 16 * (32 * k + lane)),
                                           fr, &acc);
                    } else {
                        for (uint32_t at = 16 * lane; at < n; at += 512)
                            sum_vector<GT>(*reinterpret_cast<const uint4*>(in + at), fr, &acc);
                    }
                }
                __syncwarp();                     // every lane has read the slot
                ++taken;
                start_next(slot);
                if (++slot == kStreamSlots) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
            float s = row_total(acc);
            if (edge >= 0 && r.fast) s = __fadd_rn(s, row_term(xe, r));
            s = team.sum(s, &bad, turn);
            turn ^= 1;
            if (bad) break;
            if (!r.fast || !(s < kFastSum)) {
                const RowScale sr = slow_row<GT>(x, a.v, team);
                r = sr.r;
                s = sr.sum;
            }
            if (lane == l) {
                my_ref = r;
                my_sum = s;
            }
        }
        if (bad) break;
        // the batch's terms, a row per lane
        if (part == 0) {
            int q = -1;
            if (j0 + lane < rows) {
                const int64_t i = share.row(j0 + lane);
                const Logp lp = row_logp(mine.xy, my_ref, my_sum);
                a.logps[i] = lp.hi;
                if constexpr (PREF) {
                    const int seq = find_sequence(t, i);
                    q = seq >> 1;
                    p.term[i] = __fmul_rn(mine.w, logp_less(lp, mine.f[0]));
                    p.seq[i] = seq;
                    save_row(p, i, my_ref, my_sum);
                } else {
                    const PolicyTerms pt = policy_terms(lp, mine.f[0], mine.f[1], mine.f[2], pol);
                    const float k = __fdiv_rn(mine.w, norm);
                    add_policy(sums, pt, pol, k);
                    if (p.term != nullptr) {      // for a backward pass of its own
                        p.term[i] = __fmul_rn(pt.slope, k);
                        save_row(p, i, my_ref, my_sum);
                    }
                }
            }
            if constexpr (PREF) rows_done(a, t, q, &ready);
        }
        mine = after;
        after = param(j0 + 64);
    }
    if (bad) {
        // copies in flight land before the block may exit
        bool drained = true;
        for (; taken < issued; ++taken) {
            drained = mbar_wait(&full[warp][slot], parity, kDrainNs) && drained;
            if (++slot == kStreamSlots) {
                slot = 0;
                parity ^= 1u;
            }
        }
        if (lane == 0)
            atomicOr(&g_loss_status,
                     kStatusConsumerTimeout | (drained ? 0u : kStatusDrainTimeout));
    }
    // the rows of weight 0
    if (part == 0 && !bad) {
        for (int j0 = 0; j0 < share.n_dead; j0 += 32) {
            int q = -1;
            if (j0 + lane < share.n_dead) {
                const int64_t i = share.dead_row(j0 + lane);
                a.logps[i] = 0.0f;
                if constexpr (PREF) {
                    const int seq = find_sequence(t, i);
                    q = seq >> 1;
                    p.term[i] = 0.0f;
                    p.seq[i] = seq;
                }
            }
            if constexpr (PREF) rows_done(a, t, q, &ready);
        }
    }
    if constexpr (PREF) {
        // the pairs that this block's rows completed, a warp each
        __syncthreads();
        for (int k = warp; k < ready.n; k += kStreamWarps) finish_pair(a, p, t, ready.pair[k]);
        if (end == t.start[2 * t.pairs]) preference_stats(a, p, t);
    } else {
        if (part == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Sum2 s = warp_sum(sums[k]);
                if (lane == 0) team_sums[which][k] = s.wide();
            }
        }
        __syncthreads();
        if (warp == 0) {
            double s = 0.0;
            if (lane < 4)
                for (int w = 0; w < kRowTeams; ++w) s += team_sums[w][lane];
            join_sums(a, s, first_launch, last_launch);
        }
    }
}

int row_blocks(int64_t rows, int per_sm) {
    const int64_t most = per_sm * static_cast<int64_t>(device_sms());
    const int64_t cap = most < kLossMaxBlocks ? most : kLossMaxBlocks;
    return static_cast<int>(rows < 1 ? 1 : rows < cap ? rows : cap);
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <class K>
cudaError_t opt_in(K kernel, size_t bytes, std::atomic<int>* applied) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 256;
    if (known && applied[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
    if (e == cudaSuccess && known) applied[dev].store(1, std::memory_order_relaxed);
    return e;
}

template <int GT, Pass M>
cudaError_t go_staged(const TokenArgs& a, const PolicyArgs& pol, const PreferenceArgs& p,
                      int64_t begin, int64_t end, cudaStream_t s) {
    static std::atomic<int> applied[256];
    const cudaError_t e = opt_in(staged_rows<GT, M>, kStagedSmem, applied);
    if (e != cudaSuccess) return e;
    return launch_after(staged_rows<GT, M>, dim3(row_blocks(end - begin, 1)),
                        dim3(kStagedThreads), kStagedSmem, s, a, pol, p, begin, end, begin == 0,
                        end == a.n, tma_wait_limit());
}
template <int GT, int W, class Table>
cudaError_t go_stream_w(const TokenArgs& a, const PolicyArgs& pol, const PreferenceArgs& p,
                        const Table& t, int64_t begin, int64_t end, cudaStream_t s) {
    static std::atomic<int> applied[256];
    const cudaError_t e = opt_in(stream_forward<GT, W, Table>, kStreamSmem, applied);
    if (e != cudaSuccess) return e;
    constexpr int teams = kStreamWarps / W;
    return launch_after(stream_forward<GT, W, Table>,
                        dim3(row_blocks((end - begin + teams - 1) / teams, 1)),
                        dim3(kStreamThreads), kStreamSmem, s, a, pol, p, t, begin, end,
                        begin == 0, end == a.n, tma_wait_limit());
}
// Warps per row: 4 from 8 rows per SM on (1216 rows of 32000 bf16 logits: 22.3 us
// against 26.9 with 16; 2000 rows: 30.2 against 37.5), 16 below (152 rows: 10.7 us
// against 13.6; at 760 rows 4 are ahead already, 19.8 against 21.4: the two meet
// between 1 and 5 rows per SM).  One warp per row was 6% slower at 3800 rows.
template <int GT, class Table>
cudaError_t go_stream(const TokenArgs& a, const PolicyArgs& pol, const PreferenceArgs& p,
                      const Table& t, int64_t begin, int64_t end, cudaStream_t s) {
    if (end - begin >= 8 * static_cast<int64_t>(device_sms()))
        return go_stream_w<GT, 4>(a, pol, p, t, begin, end, s);
    return go_stream_w<GT, 16>(a, pol, p, t, begin, end, s);
}
template <int GT>
cudaError_t go_forward(const TokenArgs& a, const PreferenceArgs& p, const PairTableLarge& t,
                       int64_t begin, int64_t end, cudaStream_t s) {
    if (t.pairs > kPairsSmall) return go_stream<GT>(a, PolicyArgs{}, p, t, begin, end, s);
    PairTable<kPairsSmall> small;
    std::copy(t.start, t.start + 2 * t.pairs + 1, small.start);
    small.pairs = t.pairs;
    return go_stream<GT>(a, PolicyArgs{}, p, small, begin, end, s);
}

template <int GT>
cudaError_t go_backward(const TokenArgs& a, const PreferenceArgs& p, int64_t begin, int64_t end,
                        bool staged, cudaStream_t s) {
    if (staged) return go_staged<GT, Pass::kBackward>(a, PolicyArgs{}, p, begin, end, s);
    return launch_after(offset_backward<GT>, dim3(row_blocks(end - begin, 2)), dim3(kRowThreads),
                        0, s, a, p, begin, end);
}

}  // namespace

bool loss_row_fits(int64_t v, int dtype) {
    return v * (dtype == kGradF32 ? 4 : 2) <= static_cast<int64_t>(kSlots) * kChunk;
}

cudaError_t read_loss_status(unsigned int* status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_loss_status, sizeof(unsigned int));
    if (e != cudaSuccess || !clear) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_loss_status, &zero, sizeof(unsigned int));
}

int64_t loss_rows_per_launch() { return static_cast<int64_t>(kShareRows) * device_sms(); }

cudaError_t launch_policy_staged(const TokenArgs& a, const PolicyArgs& pol, int64_t begin,
                                 int64_t end, int dtype, cudaStream_t s) {
    const PreferenceArgs none{};
    const cudaError_t e =
        dtype == kGradF32   ? go_staged<kGradF32, Pass::kPolicy>(a, pol, none, begin, end, s)
        : dtype == kGradF16 ? go_staged<kGradF16, Pass::kPolicy>(a, pol, none, begin, end, s)
                            : go_staged<kGradBF16, Pass::kPolicy>(a, pol, none, begin, end, s);
    note_launch();
    return e;
}
cudaError_t launch_policy_forward(const TokenArgs& a, const PolicyArgs& pol,
                                  const PreferenceArgs& p, int64_t begin, int64_t end, int dtype,
                                  cudaStream_t s) {
    const NoTable t{0};
    const cudaError_t e = dtype == kGradF32   ? go_stream<kGradF32>(a, pol, p, t, begin, end, s)
                          : dtype == kGradF16 ? go_stream<kGradF16>(a, pol, p, t, begin, end, s)
                                              : go_stream<kGradBF16>(a, pol, p, t, begin, end, s);
    note_launch();
    return e;
}
cudaError_t launch_preference_forward(const TokenArgs& a, const PreferenceArgs& p,
                                      const PairTableLarge& t, int64_t begin, int64_t end,
                                      int dtype, cudaStream_t s) {
    const cudaError_t e = dtype == kGradF32   ? go_forward<kGradF32>(a, p, t, begin, end, s)
                          : dtype == kGradF16 ? go_forward<kGradF16>(a, p, t, begin, end, s)
                                              : go_forward<kGradBF16>(a, p, t, begin, end, s);
    note_launch();
    return e;
}
cudaError_t launch_loss_backward(const TokenArgs& a, const PreferenceArgs& p, int64_t begin,
                                 int64_t end, int dtype, bool staged, cudaStream_t stream) {
    const cudaError_t e =
        dtype == kGradF32   ? go_backward<kGradF32>(a, p, begin, end, staged, stream)
        : dtype == kGradF16 ? go_backward<kGradF16>(a, p, begin, end, staged, stream)
                            : go_backward<kGradBF16>(a, p, begin, end, staged, stream);
    note_launch();
    return e;
}

}  // namespace shardstep
