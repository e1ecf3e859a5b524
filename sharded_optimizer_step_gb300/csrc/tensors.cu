// Work over a list of separately allocated tensors: the AdamW step with its
// moments in 32 or in 8 bits, and the global gradient norm with its clipping
// factor.  The list travels as a kernel parameter (a table of pointers and
// block ranges), so a call keeps nothing on the device and copies nothing to
// it; a block finds its tensor by a search of the table.
//
// 8-bit moments.  A tensor's elements are taken in blocks of 256; each block
// keeps max|m| / 448 and max sqrt(v) / 1.9375 in fp32.  m is an e4m3 float of
// that scale (round to nearest even).  Of v its root is kept, r = sqrt(v), as
// an unsigned float of 4 exponent and 4 mantissa bits without subnormals:
// code c > 0 stands for (1 + (c & 15) / 16) 2^((c >> 4) - 15), 0 for zero.
// The root halves v's range in octaves, the missing sign pays for the fourth
// mantissa bit (at most 1/32 off instead of 1/16), and r is what the update
// divides by.  Rounding is to nearest, ties up: one integer add.  A non-zero
// root keeps at least code 1, so that a denominator is never taken for zero
// while its m survives.  Every block's largest element is its scale, so a
// uniform decay of a block is followed exactly, whatever the codes' spacing.
// Nearest has a limit: a root changes by at most (1 - b2) / 2 of itself per step
// downwards, so with b2 = 0.999 no code is ever left that way, and an element keeps
// its share of its block's largest (0.85 to 1.31 of the 32-bit roots for steady
// gradients); with b2 <= 0.95 codes follow.
#include <cuda_fp8.h>

#include "common.cuh"
#include "pairs.cuh"

namespace shardstep {
namespace {

constexpr int kListThreads = 256;

template <int GT>
__device__ __forceinline__ float cvt16(uint32_t h) {
    if constexpr (GT == kGradF16) return f16_to_f32(static_cast<uint16_t>(h));
    return bf16_to_f32(static_cast<uint16_t>(h));
}
template <int GT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (GT == kGradF32) return static_cast<const float*>(p)[i];
    return cvt16<GT>(static_cast<const uint16_t*>(p)[i]);
}
// W = 4 or 8 consecutive elements, i a multiple of W (16-byte aligned base).
template <int GT, int W>
__device__ __forceinline__ void loadw(const void* p, int64_t i, float* f) {
    if constexpr (GT == kGradF32) {
#pragma unroll
        for (int k = 0; k < W; k += 4)
            unpack4f(ldcs16(static_cast<const float*>(p) + i + k), f + k);
    } else {
        uint32_t w[W / 2];
        if constexpr (W == 8) {
            const uint4 r = ldcs16(static_cast<const uint16_t*>(p) + i);
            w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
        } else {
            const uint2 r = ldcs8(static_cast<const uint16_t*>(p) + i);
            w[0] = r.x; w[1] = r.y;
        }
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            f[2 * k] = cvt16<GT>(w[k] & 0xFFFFu);
            f[2 * k + 1] = cvt16<GT>(w[k] >> 16);
        }
    }
}

// fp32 -> the parameters' 16-bit type, round to nearest even.
template <int PT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (PT == kGradF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(a, b);
}
template <int PT>
__device__ __forceinline__ uint16_t pack1(float a) {
    return static_cast<uint16_t>(pack2<PT>(a, 0.0f) & 0xFFFFu);
}

// The tensor among lo .. hi that block b of the launch belongs to.
template <class Table>
__device__ __forceinline__ int find_tensor(const Table& t, uint32_t b, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.b0[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// (A search of all of 148 tensors took a tenth of the 8-bit step's instructions.)
template <int CAP>
__device__ __forceinline__ int find_tensor(const TensorTable<CAP>& t, uint32_t b) {
    const uint32_t k = b >> t.near_shift;
    return find_tensor(t, b, t.near[k], t.near[k + 1]);
}

// The 32-bit step: the fused step's update (adamw_elem, so the bits are those
// of the flat step at N_d = 1) over one block's chunk of a tensor.  Bound by
// memory: (gradient + 24 + 2) bytes per element.  A chunk's loads are all issued
// before its arithmetic.  124M elements in 148 tensors, bf16 gradients: 492 us,
// 7.08 TB/s; 400M: 1563 us, 7.16 TB/s.
template <int CAP, int GT, int PT>
__global__ void __launch_bounds__(kListThreads)
    tensors_adamw32(const __grid_constant__ TensorTable<CAP> t,
                    const __grid_constant__ GroupScalars gs, const float* coef,
                    const unsigned int* skip) {
    pdl_enter();
    if (skip_step(skip)) return;
    const int s = find_tensor(t, blockIdx.x);
    const AdamScalars c = resolve_adam(gs.c[t.group[s]]);
    const float k = coef != nullptr ? __ldg(coef) : 1.0f;
    const int64_t n = t.n[s];
    const int64_t base = static_cast<int64_t>(blockIdx.x - t.b0[s]) * kListChunk32;
    const void* G = t.grad[s];
    float* P = t.master[s];
    float* M = static_cast<float*>(t.m[s]);
    float* V = static_cast<float*>(t.v[s]);
    uint16_t* O = static_cast<uint16_t*>(t.param[s]);
    if (t.vec[s] && base + kListChunk32 <= n) {
        constexpr int U = kListChunk32 / (4 * kListThreads);
        float g[U][4];
        uint4 p4[U], m4[U], v4[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + 4 * (u * kListThreads + threadIdx.x);
            loadw<GT, 4>(G, i, g[u]);
            p4[u] = ldcs16(P + i);
            m4[u] = ldcs16(M + i);
            v4[u] = ldcs16(V + i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + 4 * (u * kListThreads + threadIdx.x);
            float pp[4], mm[4], vv[4];
            unpack4f(p4[u], pp);
            unpack4f(m4[u], mm);
            unpack4f(v4[u], vv);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                adamw_elem(coef != nullptr ? __fmul_rn(g[u][e], k) : g[u][e], pp[e], mm[e],
                           vv[e], c);
            stcs16(P + i, pack4f(pp));
            stcs16(M + i, pack4f(mm));
            stcs16(V + i, pack4f(vv));
            if (O != nullptr)
                stcs8(O + i, make_uint2(pack2<PT>(pp[0], pp[1]), pack2<PT>(pp[2], pp[3])));
        }
        return;
    }
    const int64_t end = base + kListChunk32 < n ? base + kListChunk32 : n;
    for (int64_t i = base + threadIdx.x; i < end; i += kListThreads) {
        float g = load1<GT>(G, i);
        if (coef != nullptr) g = __fmul_rn(g, k);
        float pp = P[i], mm = M[i], vv = V[i];
        adamw_elem(g, pp, mm, vv, c);
        P[i] = pp;
        M[i] = mm;
        V[i] = vv;
        if (O != nullptr) O[i] = pack1<PT>(pp);
    }
}

// ------------------------------------------------------- 8-bit moments

constexpr float kE4m3Max = 448.0f;
constexpr float kRootMax = 1.9375f;
constexpr float kTinyBlock = 0x1p-100f;

// Two e4m3 codes (low byte first) as floats.
__device__ __forceinline__ Pair e4m3x2_to_f32(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return make_pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(Pair p) {
    return __nv_cvt_float2_to_fp8x2(floats(p), __NV_SATFINITE, __NV_E4M3);
}
// The root's code: 1792 = (127 - 15) * 16 moves the exponent's bias.
__device__ __forceinline__ float root_to_f32(uint32_t c) {
    return c != 0 ? __uint_as_float((c << 19) + (1792u << 19)) : 0.0f;
}
// y in [0, 1.9375 (1 + 2^-22)]: the codes' end needs no clamp from above, the
// unsigned minimum of the bits and 1 is 0 for y = 0 alone.
__device__ __forceinline__ uint32_t f32_to_root(float y) {
    const int c = static_cast<int>(__float_as_uint(y) + 0x40000u - (1792u << 19)) >> 19;
    return static_cast<uint32_t>(max(c, static_cast<int>(min(__float_as_uint(y), 1u))));
}

// The scales of a block from the largest magnitudes' bit patterns (as
// unsigned integers these order like the magnitudes, NaN above infinity, so
// a non-finite element makes its block's scale non-finite and is not lost),
// and the factors that bring the largest values to the codes' ends.  The four
// divisions run side by side in four lanes.  Blocks below 2^-100 are stored
// as zeros: the factors would leave fp32's range.
struct BlockScales {
    float m_scale, m_up, r_scale, r_up;
};
__device__ __forceinline__ BlockScales block_scales(uint32_t m_big, uint32_t r_big) {
    const int lane = threadIdx.x & 31;
    const float big = __uint_as_float(lane & 2 ? r_big : m_big);
    const float top = lane & 2 ? kRootMax : kE4m3Max;
    float q = lane & 1 ? __fdiv_rn(top, big) : __fdiv_rn(big, top);
    if (big < kTinyBlock) q = 0.0f;
    BlockScales b;
    b.m_scale = __shfl_sync(0xFFFFFFFFu, q, 0);
    b.m_up = __shfl_sync(0xFFFFFFFFu, q, 1);
    b.r_scale = __shfl_sync(0xFFFFFFFFu, q, 2);
    b.r_up = __shfl_sync(0xFFFFFFFFu, q, 3);
    return b;
}

// 4 consecutive elements of a lane, as two pairs: codes <-> values.
__device__ __forceinline__ void decode4(uint32_t mc, uint32_t vc, float ms, float vs, Pair* m,
                                        Pair* r) {
    const Pair ms2 = make_pair(ms, ms), vs2 = make_pair(vs, vs);
    m[0] = mul2(e4m3x2_to_f32(mc & 0xFFFFu), ms2);
    m[1] = mul2(e4m3x2_to_f32(mc >> 16), ms2);
    r[0] = mul2(make_pair(root_to_f32(vc & 0xFFu), root_to_f32((vc >> 8) & 0xFFu)), vs2);
    r[1] = mul2(make_pair(root_to_f32((vc >> 16) & 0xFFu), root_to_f32(vc >> 24)), vs2);
}
// The roots come negated, as the step has them.
__device__ __forceinline__ void encode4(const Pair* m, const Pair* r_neg, const BlockScales& b,
                                        uint32_t* mc, uint32_t* vc) {
    const Pair mu = make_pair(b.m_up, b.m_up), ru = make_pair(-b.r_up, -b.r_up);
    *mc = f32_to_e4m3x2(mul2(m[0], mu)) | (f32_to_e4m3x2(mul2(m[1], mu)) << 16);
    const float2 y0 = floats(mul2(r_neg[0], ru)), y1 = floats(mul2(r_neg[1], ru));
    *vc = f32_to_root(y0.x) + (f32_to_root(y0.y) << 8) + (f32_to_root(y1.x) << 16) +
          (f32_to_root(y1.y) << 24);
}
// max(|a|, |b|, |c|), NaN where one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The scales of a warp's block from each lane's 2 x 4 elements.
__device__ __forceinline__ uint32_t lane_max(const Pair (*x)[2]) {
    float big = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 f = floats(x[h][k]);
            big = max3_abs(big, f.x, f.y);
        }
    return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big));
}

// min(|a|, |b|, |c|), NaN where one is.
__device__ __forceinline__ float min3_abs(float a, float b, float c) {
    float d;
    asm("min.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Roots and quotients two elements to an instruction, correctly rounded, by
// Markstein's corrections ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): an approximation, one Newton step, and the
// residual, which fma gives exactly, times the reciprocal.  They hold where no
// residual leaves the normal range: see kFastLeast.  Signs are chosen so that no
// operand has to be negated on the way.
constexpr float kFastLeast = 0x1p-80f;

// -sqrt(v) from -v.  Equal to the IEEE root for all 2^24 fractions of [1, 4).
__device__ __forceinline__ Pair neg_sqrt2(Pair v_neg) {
    const float2 v = floats(v_neg);
    float a, b;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(-v.x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(-v.y));
    const Pair y = make_pair(a, b), half = make_pair(0.5f, 0.5f);
    Pair s = mul2(v_neg, y), h = mul2(y, half);      // s: the negative root
    const Pair e = fma2(s, h, half);
    s = fma2(s, e, s);
    h = fma2(h, e, h);
    return fma2(fma2(s, s, v_neg), h, s);
}
// 1 / d from -d.  Equal to the IEEE quotient for all 2^23 fractions of d.
__device__ __forceinline__ Pair reciprocal2(Pair d_neg) {
    const float2 d = floats(d_neg);
    float a, b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(-d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(-d.y));
    const Pair y = make_pair(a, b);
    return fma2(y, fma2(d_neg, y, make_pair(1.0f, 1.0f)), y);
}
// n / d from -d and y = RN(1 / d): twice the correction, so that the quotient is
// within an ulp before the step that rounds it whatever the fractions are.
__device__ __forceinline__ Pair divide2(Pair n, Pair d_neg, Pair y) {
    Pair q = mul2(n, y);
    q = fma2(fma2(q, d_neg, n), y, q);
    return fma2(fma2(q, d_neg, n), y, q);
}

// The 8-bit step: a warp per block of 256 elements, 4 + 4 per lane (128 apart,
// so that every access of a warp is one contiguous run), so a block's maxima
// are two warp reductions and nothing leaves the registers between the load and
// the store of a code.  Per element, one IEEE rounding per operation as in
// adamw_elem, with the root of v in and out:
//   p -= lr wd p;  m = b1 m + (1 - b1) g;  r = sqrt(b2 r^2 + (1 - b2) g g);
//   p -= (lr / bc1) m / (r / sqrt(bc2) + eps), with m and r before rounding
// to their codes.  Bound by memory in the limit, (gradient + 8 + 4 + 2) bytes
// per element, if the issue slots keep up: all arithmetic goes two elements to
// an instruction, roots and quotients too where the block's values allow it (124M
// elements in 326 us, 6.1 TB/s, with issue slots 64% busy; 16 us more with the IEEE
// operations alone).  One block per warp: a warp that took 4 in turn needed 450 us
// with the next block's loads in flight, for want of warps to hide a block's chain
// of dependent operations behind.
template <int CAP, int GT, int PT>
__global__ void __launch_bounds__(kListThreads)
    tensors_adamw8(const __grid_constant__ TensorTable<CAP> t,
                   const __grid_constant__ GroupScalars gs, const float* coef,
                   const unsigned int* skip) {
    pdl_enter();
    if (skip_step(skip)) return;
    const int s = find_tensor(t, blockIdx.x);
    const AdamScalars c = resolve_adam(gs.c[t.group[s]]);
    const float inv_root =
        c.dev != nullptr ? __fdiv_rn(1.0f, c.sqrt_bc2) : gs.inv_sqrt_bc2[t.group[s]];
    const float k = coef != nullptr ? __ldg(coef) : 1.0f;
    const int64_t n = t.n[s];
    const void* G = t.grad[s];
    float* P = t.master[s];
    uint8_t* M = static_cast<uint8_t*>(t.m[s]);
    uint8_t* V = static_cast<uint8_t*>(t.v[s]);
    uint16_t* O = static_cast<uint16_t*>(t.param[s]);
    const bool vec = t.vec[s] != 0;
    const Pair lr_wd = make_pair(-c.lr_wd, -c.lr_wd), b1 = make_pair(c.beta1, c.beta1),
               o1 = make_pair(c.omb1, c.omb1), b2_neg = make_pair(-c.beta2, -c.beta2),
               o2_neg = make_pair(-c.omb2, -c.omb2), kk = make_pair(k, k);
    // Products that are added to are formed as a b + (-0), the same value: of a
    // plain product and a sum of pairs the assembler makes one fma (one rounding
    // instead of two) whatever their rounding modifiers, which it cannot do here
    // as long as it does not know the -0.
    const Pair nz = make_pair(gs.neg_zero, gs.neg_zero);
    const Pair root_neg = make_pair(-c.sqrt_bc2, -c.sqrt_bc2), inv = make_pair(inv_root, inv_root),
               eps_neg = make_pair(-c.eps, -c.eps), size = make_pair(c.step_size, c.step_size);
    const int64_t blk = static_cast<int64_t>(blockIdx.x - t.b0[s]) * (kListChunk8 / kMomentBlock) +
                        (threadIdx.x >> 5);
    const int64_t base = blk * kMomentBlock;
    if (base >= n) return;
    const int64_t i = base + 4 * (threadIdx.x & 31);
    float* MS = t.m_scale[s] + blk;
    float* VS = t.v_scale[s] + blk;
    const bool whole = vec && base + kMomentBlock <= n;
    float g[2][4];
    Pair p[2][2], m[2][2], r[2][2];     // r: the old root, -v, then the new root negated
    uint32_t mc[2], vc[2];
    const float ms = *MS, vs = *VS;
    if (whole) {
        uint4 p4[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            loadw<GT, 4>(G, i + 128 * h, g[h]);
            mc[h] = __ldcs(reinterpret_cast<const uint32_t*>(M + i + 128 * h));
            vc[h] = __ldcs(reinterpret_cast<const uint32_t*>(V + i + 128 * h));
            p4[h] = ldcs16(P + i + 128 * h);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
            unpack4f(p4[h], f);
            p[h][0] = make_pair(f[0], f[1]);
            p[h][1] = make_pair(f[2], f[3]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
            mc[h] = vc[h] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t j = i + 128 * h + e;
                g[h][e] = f[e] = 0.0f;
                if (j < n) {
                    g[h][e] = load1<GT>(G, j);
                    f[e] = P[j];
                    mc[h] |= static_cast<uint32_t>(M[j]) << (8 * e);
                    vc[h] |= static_cast<uint32_t>(V[j]) << (8 * e);
                }
            }
            p[h][0] = make_pair(f[0], f[1]);
            p[h][1] = make_pair(f[2], f[3]);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        decode4(mc[h], vc[h], ms, vs, m[h], r[h]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            Pair gg = make_pair(g[h][2 * e], g[h][2 * e + 1]);
            if (coef != nullptr) gg = mul2(gg, kk);
            p[h][e] = add2(p[h][e], fma2(lr_wd, p[h][e], nz));
            m[h][e] = add2(fma2(b1, m[h][e], nz), fma2(o1, gg, nz));
            r[h][e] = add2(fma2(b2_neg, mul2(r[h][e], r[h][e]), nz),
                           fma2(mul2(o2_neg, gg), gg, nz));
        }
    }
    if (!whole) {   // places past the tensor's end take no part in the maxima
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t j = i + 128 * h + 2 * e;
                const float2 a = floats(m[h][e]), b = floats(r[h][e]);
                m[h][e] = make_pair(j < n ? a.x : 0.0f, j + 1 < n ? a.y : 0.0f);
                r[h][e] = make_pair(j < n ? b.x : 0.0f, j + 1 < n ? b.y : 0.0f);
            }
    }
    // the root of the largest v is the largest root
    const uint32_t m_big = lane_max(m), v_big = lane_max(r);
    const uint32_t r_big = __float_as_uint(__fsqrt_rn(__uint_as_float(v_big)));
    const BlockScales b = block_scales(m_big, r_big);
    if ((threadIdx.x & 31) == 0) {
        *MS = b.m_scale;
        *VS = b.r_scale;
    }
    Pair num[2][2];
    float least = INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            num[h][e] = mul2(size, m[h][e]);
            const float2 a = floats(num[h][e]), v = floats(r[h][e]);
            least = min3_abs(least, a.x, a.y);
            least = min3_abs(least, v.x, v.y);
        }
    // Every v and every numerator at least 2^-80 (a zero is not: its sign would be
    // lost), v below 2^30, sqrt(bc2) from 2^-8 to 1, eps below 1: denominators lie
    // between 2^-40 and 2^23 + 1, quotients between 2^-104 and 2^100, residuals
    // above 2^-130.
    const bool fast = __all_sync(0xFFFFFFFFu, least >= kFastLeast) &&
                      __uint_as_float(v_big) < 0x1p30f &&
                      fabsf(__fmul_rn(c.step_size, __uint_as_float(m_big))) < 0x1p60f &&
                      c.sqrt_bc2 > 0x1p-8f && c.sqrt_bc2 <= 1.0f && c.eps >= 0.0f &&
                      c.eps < 1.0f;
    if (fast) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                r[h][e] = neg_sqrt2(r[h][e]);
                const Pair den_neg = add2(divide2(r[h][e], root_neg, inv), eps_neg);
                num[h][e] = divide2(num[h][e], den_neg, reciprocal2(den_neg));
            }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 v = floats(r[h][e]), a = floats(num[h][e]);
                const float x = __fsqrt_rn(-v.x), y = __fsqrt_rn(-v.y);
                r[h][e] = make_pair(-x, -y);
                num[h][e] = make_pair(
                    __fdiv_rn(a.x, __fadd_rn(__fdiv_rn(x, c.sqrt_bc2), c.eps)),
                    __fdiv_rn(a.y, __fadd_rn(__fdiv_rn(y, c.sqrt_bc2), c.eps)));
            }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        encode4(m[h], r[h], b, &mc[h], &vc[h]);
        float f[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 x = floats(p[h][e]), q = floats(num[h][e]);
            f[2 * e] = __fsub_rn(x.x, q.x);
            f[2 * e + 1] = __fsub_rn(x.y, q.y);
        }
        if (whole) {
            stcs16(P + i + 128 * h, pack4f(f));
            __stcs(reinterpret_cast<uint32_t*>(M + i + 128 * h), mc[h]);
            __stcs(reinterpret_cast<uint32_t*>(V + i + 128 * h), vc[h]);
            if (O != nullptr)
                stcs8(O + i + 128 * h, make_uint2(pack2<PT>(f[0], f[1]), pack2<PT>(f[2], f[3])));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t j = i + 128 * h + e;
                if (j < n) {
                    P[j] = f[e];
                    M[j] = static_cast<uint8_t>(mc[h] >> (8 * e));
                    V[j] = static_cast<uint8_t>(vc[h] >> (8 * e));
                    if (O != nullptr) O[j] = pack1<PT>(f[e]);
                }
            }
        }
    }
}

// Codes -> fp32 moments: m = code * scale, v = (code * scale)^2.  A thread takes
// 4 consecutive elements at 2 places 1024 apart.  Bound by memory: 124M elements
// in 182 us, 6.85 TB/s.
constexpr int kDecodeChunk = 2 * 4 * kListThreads;
__global__ void __launch_bounds__(kListThreads)
    moments_decode(const uint8_t* __restrict__ M, const float* __restrict__ MS,
                   const uint8_t* __restrict__ V, const float* __restrict__ VS, int64_t n,
                   float* __restrict__ Mo, float* __restrict__ Vo, bool vec) {
    pdl_enter();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kDecodeChunk;
    if (vec && base + kDecodeChunk <= n) {
        uint32_t mc[2], vc[2];
        float ms[2], vs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = base + 4 * (h * kListThreads + threadIdx.x);
            mc[h] = __ldcs(reinterpret_cast<const uint32_t*>(M + i));
            vc[h] = __ldcs(reinterpret_cast<const uint32_t*>(V + i));
            ms[h] = __ldg(MS + i / kMomentBlock);
            vs[h] = __ldg(VS + i / kMomentBlock);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = base + 4 * (h * kListThreads + threadIdx.x);
            Pair m[2], r[2];
            decode4(mc[h], vc[h], ms[h], vs[h], m, r);
            const float2 a = floats(m[0]), b = floats(m[1]);
            const float2 x = floats(mul2(r[0], r[0])), y = floats(mul2(r[1], r[1]));
            const float f[4] = {a.x, a.y, b.x, b.y}, g[4] = {x.x, x.y, y.x, y.y};
            stcs16(Mo + i, pack4f(f));
            stcs16(Vo + i, pack4f(g));
        }
        return;
    }
    const int64_t end = base + kDecodeChunk < n ? base + kDecodeChunk : n;
    for (int64_t i = base + threadIdx.x; i < end; i += kListThreads) {
        Mo[i] = __fmul_rn(floats(e4m3x2_to_f32(M[i])).x, MS[i / kMomentBlock]);
        const float x = __fmul_rn(root_to_f32(V[i]), VS[i / kMomentBlock]);
        Vo[i] = __fmul_rn(x, x);
    }
}

// fp32 moments -> codes and scales, a warp per block, laid out as in the step.
// For setting a state once; its loads are single elements.
__global__ void __launch_bounds__(kListThreads)
    moments_encode(const float* __restrict__ Mi, const float* __restrict__ Vi, int64_t n,
                   uint8_t* __restrict__ M, float* __restrict__ MS, uint8_t* __restrict__ V,
                   float* __restrict__ VS, bool vec) {
    pdl_enter();
    const int64_t blk =
        static_cast<int64_t>(blockIdx.x) * (kListThreads / 32) + (threadIdx.x >> 5);
    const int64_t base = blk * kMomentBlock;
    if (base >= n) return;
    const int64_t i = base + 4 * (threadIdx.x & 31);
    const bool whole = vec && base + kMomentBlock <= n;
    Pair m[2][2], r[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t j = i + 128 * h + e;
            a[e] = j < n ? Mi[j] : 0.0f;
            b[e] = j < n ? Vi[j] : 0.0f;
        }
        m[h][0] = make_pair(a[0], a[1]);
        m[h][1] = make_pair(a[2], a[3]);
        r[h][0] = make_pair(-__fsqrt_rn(b[0]), -__fsqrt_rn(b[1]));
        r[h][1] = make_pair(-__fsqrt_rn(b[2]), -__fsqrt_rn(b[3]));
    }
    const uint32_t m_big = lane_max(m), r_big = lane_max(r);
    const BlockScales b = block_scales(m_big, r_big);
    if ((threadIdx.x & 31) == 0) {
        MS[blk] = b.m_scale;
        VS[blk] = b.r_scale;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t mc, vc;
        encode4(m[h], r[h], b, &mc, &vc);
        if (whole) {
            __stcs(reinterpret_cast<uint32_t*>(M + i + 128 * h), mc);
            __stcs(reinterpret_cast<uint32_t*>(V + i + 128 * h), vc);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t j = i + 128 * h + e;
                if (j < n) {
                    M[j] = static_cast<uint8_t>(mc >> (8 * e));
                    V[j] = static_cast<uint8_t>(vc >> (8 * e));
                }
            }
        }
    }
}

// ------------------------------------------------------------- the norm

// Sum of the first lanes' doubles of a block's warps in a fixed order; the
// result in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kListThreads / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kListThreads / 32; ++w) s += part[w];
    __syncthreads();
    return s;
}

// acc += the squares of the elements of 16 bytes.
template <int GT>
__device__ __forceinline__ void add_squares(const uint4& raw, Pair* acc) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (GT == kGradF32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Pair x = make_pair(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
            acc[k] = fma2(x, x, acc[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const Pair x = make_pair(cvt16<GT>(w[k] & 0xFFFFu), cvt16<GT>(w[k] >> 16));
            acc[k] = fma2(x, x, acc[k]);
        }
    }
}

// Squares are formed and summed in fp32, in 8 sums per thread over the chunks
// a block takes in turn (b, b + gridDim, ...); the threads' sums are joined in
// double in a fixed order, the blocks' likewise by the block that arrives
// last, so the result does not depend on the order in which blocks run.
// Bound by the one read of the gradients: 124M bf16 elements in 148 tensors take
// 41.6 us, 6.0 TB/s; 400M 119 us, 6.7 TB/s.
template <int CAP, int GT>
__global__ void __launch_bounds__(kListThreads, 4)
    tensors_norm(const __grid_constant__ NormTable<CAP> t, const NormArgs a) {
    pdl_enter();
    Pair acc[4] = {0, 0, 0, 0};
    const uint32_t chunks = t.b0[t.count];
    int s = blockIdx.x < chunks ? find_tensor(t, blockIdx.x, 0, t.count - 1) : 0;
    for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
        while (b >= t.b0[s + 1]) ++s;
        const int64_t n = t.n[s];
        const int64_t base = static_cast<int64_t>(b - t.b0[s]) * kNormChunk;
        const void* G = t.p[s];
        if (t.vec[s] && base + kNormChunk <= n) {
            // all of the chunk's loads in flight before any arithmetic
            constexpr int es = GT == kGradF32 ? 4 : 2;
            constexpr int U = kNormChunk * es / (16 * kListThreads);
            const char* at = static_cast<const char*>(G) + base * es + 16 * threadIdx.x;
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = ld_once(at + 16 * kListThreads * u);
#pragma unroll
            for (int u = 0; u < U; ++u) add_squares<GT>(raw[u], acc);
        } else {
            const int64_t end = base + kNormChunk < n ? base + kNormChunk : n;
            for (int64_t i = base + threadIdx.x; i < end; i += kListThreads) {
                const float x = load1<GT>(G, i);
                const Pair x2 = make_pair(x, 0.0f);
                acc[0] = fma2(x2, x2, acc[0]);
            }
        }
    }
    // the 8 sums and the warp's in fp32, pairwise; double from there on (an SM has
    // few units for it)
    const float2 f = floats(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
    float own = __fadd_rn(f.x, f.y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) own = __fadd_rn(own, __shfl_xor_sync(0xFFFFFFFFu, own, d));
    double sum = block_sum((threadIdx.x & 31) == 0 ? static_cast<double>(own) : 0.0);
    __shared__ bool last;
    if (threadIdx.x == 0) {
        double* slot = a.ws->partial + blockIdx.x;
        *slot = a.first ? sum : __dadd_rn(*slot, sum);
        __threadfence();
        // wraps to 0 with the last arrival: the workspace is ready for the next call
        last = atomicInc(&a.ws->arrived, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last || !a.last) return;
    __threadfence();
    double total = 0.0;
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kListThreads)
        total += __ldcg(a.ws->partial + b);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    total = block_sum(total);
    if (threadIdx.x == 0) {
        const float scale = a.scale != nullptr ? __ldg(a.scale) : 1.0f;
        const float norm =
            __double2float_rn(__ddiv_rn(__dsqrt_rn(total), static_cast<double>(scale)));
        float f = __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f));
        if (f > 1.0f) f = 1.0f;
        a.out[0] = norm;
        a.out[1] = __fdiv_rn(f, scale);
        if (a.found != nullptr && !(fabsf(norm) <= 0x1.fffffep127f)) *a.found = 1u;
    }
}

template <int CAP, int GT, int PT>
cudaError_t go_adamw(const TensorTable<CAP>& t, int bits, const GroupScalars& gs,
                     const float* coef, const unsigned int* skip, cudaStream_t s) {
    const dim3 grid(t.b0[t.count]), block(kListThreads);
    const cudaError_t e =
        bits == 8 ? launch_after(tensors_adamw8<CAP, GT, PT>, grid, block, 0, s, t, gs, coef, skip)
                  : launch_after(tensors_adamw32<CAP, GT, PT>, grid, block, 0, s, t, gs, coef,
                                 skip);
    note_launch();
    return e;
}
template <int CAP, int GT>
cudaError_t go_adamw_p(const TensorTable<CAP>& t, int param_type, int bits,
                       const GroupScalars& gs, const float* coef, const unsigned int* skip,
                       cudaStream_t s) {
    return param_type == kGradF16 ? go_adamw<CAP, GT, kGradF16>(t, bits, gs, coef, skip, s)
                                  : go_adamw<CAP, GT, kGradBF16>(t, bits, gs, coef, skip, s);
}

}  // namespace

template <int CAP>
cudaError_t launch_tensors_adamw(const TensorTable<CAP>& t, int grad_type, int param_type,
                                 int bits, const GroupScalars& gs, const float* coef,
                                 const unsigned int* skip, cudaStream_t s) {
    switch (grad_type) {
        case kGradF32: return go_adamw_p<CAP, kGradF32>(t, param_type, bits, gs, coef, skip, s);
        case kGradF16: return go_adamw_p<CAP, kGradF16>(t, param_type, bits, gs, coef, skip, s);
        default: return go_adamw_p<CAP, kGradBF16>(t, param_type, bits, gs, coef, skip, s);
    }
}
template cudaError_t launch_tensors_adamw<kTensorsSmall>(const TensorTable<kTensorsSmall>&, int,
                                                         int, int, const GroupScalars&,
                                                         const float*, const unsigned int*,
                                                         cudaStream_t);
template cudaError_t launch_tensors_adamw<kTensorsLarge>(const TensorTable<kTensorsLarge>&, int,
                                                         int, int, const GroupScalars&,
                                                         const float*, const unsigned int*,
                                                         cudaStream_t);

cudaError_t launch_moments_decode(const uint8_t* m, const float* m_scale, const uint8_t* v,
                                  const float* v_scale, int64_t n, float* m_out, float* v_out,
                                  bool vec, cudaStream_t stream) {
    const int64_t blocks = (n + kDecodeChunk - 1) / kDecodeChunk;
    const cudaError_t e = launch_after(moments_decode, dim3(static_cast<unsigned>(blocks)),
                                       dim3(kListThreads), 0, stream, m, m_scale, v, v_scale, n,
                                       m_out, v_out, vec);
    note_launch();
    return e;
}

cudaError_t launch_moments_encode(const float* m_in, const float* v_in, int64_t n, uint8_t* m,
                                  float* m_scale, uint8_t* v, float* v_scale, bool vec,
                                  cudaStream_t stream) {
    const int64_t blocks = (n + kListChunk8 - 1) / kListChunk8;
    const cudaError_t e = launch_after(moments_encode, dim3(static_cast<unsigned>(blocks)),
                                       dim3(kListThreads), 0, stream, m_in, v_in, n, m, m_scale,
                                       v, v_scale, vec);
    note_launch();
    return e;
}

template <int CAP>
cudaError_t launch_tensors_norm(const NormTable<CAP>& t, int type, const NormArgs& a, int blocks,
                                cudaStream_t stream) {
    const dim3 grid(blocks), block(kListThreads);
    cudaError_t e;
    switch (type) {
        case kGradF32:
            e = launch_after(tensors_norm<CAP, kGradF32>, grid, block, 0, stream, t, a);
            break;
        case kGradF16:
            e = launch_after(tensors_norm<CAP, kGradF16>, grid, block, 0, stream, t, a);
            break;
        default:
            e = launch_after(tensors_norm<CAP, kGradBF16>, grid, block, 0, stream, t, a);
            break;
    }
    note_launch();
    return e;
}
template cudaError_t launch_tensors_norm<kNormSmall>(const NormTable<kNormSmall>&, int,
                                                     const NormArgs&, int, cudaStream_t);
template cudaError_t launch_tensors_norm<kNormLarge>(const NormTable<kNormLarge>&, int,
                                                     const NormArgs&, int, cudaStream_t);

}  // namespace shardstep
