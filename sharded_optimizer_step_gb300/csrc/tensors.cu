// Work over a list of separately allocated tensors: the AdamW step with its
// moments in 32 or in 8 bits, and the global gradient norm with its clipping
// factor.  The list travels as a kernel parameter (a table of pointers and
// block ranges), so a call keeps nothing on the device and copies nothing to
// it; a block finds its tensor by a binary search of the table.
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
#include <cuda_fp8.h>

#include "common.cuh"

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

// The tensor that block b of the launch belongs to.
template <class Table>
__device__ __forceinline__ int find_tensor(const Table& t, uint32_t b) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.b0[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The 32-bit step: the fused step's update (adamw_elem, so the bits are those
// of the flat step at N_d = 1) over one block's chunk of a tensor.  Bound by
// memory: (gradient + 24 + 2) bytes per element.
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
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// The root's code: 1792 = (127 - 15) * 16 moves the exponent's bias.
__device__ __forceinline__ float root_to_f32(uint32_t c) {
    return c != 0 ? __uint_as_float((c + 1792u) << 19) : 0.0f;
}
__device__ __forceinline__ uint32_t f32_to_root(float y) {
    int c = static_cast<int>((__float_as_uint(y) + 0x40000u) >> 19) - 1792;
    c = c < 1 ? 1 : c > 255 ? 255 : c;
    return y > 0.0f ? static_cast<uint32_t>(c) : 0u;
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

// 8 consecutive elements of a lane: codes <-> values.
__device__ __forceinline__ void decode8(uint2 mc, uint2 vc, float ms, float vs, float* m,
                                        float* r) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? mc.x : mc.y;
        const float2 f = e4m3x2_to_f32((w >> (16 * (k & 1))) & 0xFFFFu);
        m[2 * k] = __fmul_rn(f.x, ms);
        m[2 * k + 1] = __fmul_rn(f.y, ms);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t w = k < 4 ? vc.x : vc.y;
        r[k] = __fmul_rn(root_to_f32((w >> (8 * (k & 3))) & 0xFFu), vs);
    }
}
__device__ __forceinline__ void encode8(const float* m, const float* r, const BlockScales& b,
                                        uint2* mc, uint2* vc) {
    uint32_t h[4], q[8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = f32_to_e4m3x2(__fmul_rn(m[2 * k], b.m_up), __fmul_rn(m[2 * k + 1], b.m_up));
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = f32_to_root(__fmul_rn(r[k], b.r_up));
    *mc = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    *vc = make_uint2(q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                     q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24));
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ BlockScales scales_of(const float* m, const float* r) {
    uint32_t mb = 0, rb = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        mb = max(mb, abs_bits(m[k]));
        rb = max(rb, abs_bits(r[k]));
    }
    return block_scales(__reduce_max_sync(0xFFFFFFFFu, mb), __reduce_max_sync(0xFFFFFFFFu, rb));
}

// One element with the root of v in and out:
//   p -= lr wd p;  m = b1 m + (1 - b1) g;  r = sqrt(b2 r^2 + (1 - b2) g g);
//   p -= (lr / bc1) m / (r / sqrt(bc2) + eps), with m and r before rounding
// to their codes.  One IEEE rounding per operation, as in adamw_elem.
__device__ __forceinline__ void adamw_root_elem(float g, float& p, float& m, float& r,
                                                const AdamScalars& c) {
    p = __fsub_rn(p, __fmul_rn(c.lr_wd, p));
    m = __fadd_rn(__fmul_rn(c.beta1, m), __fmul_rn(c.omb1, g));
    r = __fsqrt_rn(__fadd_rn(__fmul_rn(c.beta2, __fmul_rn(r, r)),
                             __fmul_rn(__fmul_rn(c.omb2, g), g)));
    const float den = __fadd_rn(__fdiv_rn(r, c.sqrt_bc2), c.eps);
    p = __fsub_rn(p, __fdiv_rn(__fmul_rn(c.step_size, m), den));
}

// The 8-bit step: a warp per block of 256 elements, 8 consecutive ones per
// lane, so a block's maxima are two warp reductions and nothing leaves the
// registers between the load and the store of a code.  Bound by memory in the
// limit, (gradient + 8 + 4 + 2) bytes per element; about 70 instructions per
// element keep the issue slots close behind.
template <int CAP, int GT, int PT>
__global__ void __launch_bounds__(kListThreads)
    tensors_adamw8(const __grid_constant__ TensorTable<CAP> t,
                   const __grid_constant__ GroupScalars gs, const float* coef,
                   const unsigned int* skip) {
    pdl_enter();
    if (skip_step(skip)) return;
    const int s = find_tensor(t, blockIdx.x);
    const AdamScalars c = resolve_adam(gs.c[t.group[s]]);
    const float k = coef != nullptr ? __ldg(coef) : 1.0f;
    const int64_t n = t.n[s];
    const int64_t blk = static_cast<int64_t>(blockIdx.x - t.b0[s]) * (kListChunk8 / kMomentBlock) +
                        (threadIdx.x >> 5);
    const int64_t base = blk * kMomentBlock;
    if (base >= n) return;
    const int64_t i = base + 8 * (threadIdx.x & 31);
    const void* G = t.grad[s];
    float* P = t.master[s];
    uint8_t* M = static_cast<uint8_t*>(t.m[s]);
    uint8_t* V = static_cast<uint8_t*>(t.v[s]);
    uint16_t* O = static_cast<uint16_t*>(t.param[s]);
    float* MS = t.m_scale[s] + blk;
    float* VS = t.v_scale[s] + blk;
    const bool whole = t.vec[s] && base + kMomentBlock <= n;
    float g[8], p[8], m[8], r[8];
    uint2 mc = make_uint2(0, 0), vc = make_uint2(0, 0);
    const float ms = *MS, vs = *VS;
    if (whole) {
        loadw<GT, 8>(G, i, g);
        mc = ldcs8(M + i);
        vc = ldcs8(V + i);
        unpack4f(ldcs16(P + i), p);
        unpack4f(ldcs16(P + i + 4), p + 4);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] = p[e] = 0.0f;
            if (i + e < n) {
                g[e] = load1<GT>(G, i + e);
                p[e] = P[i + e];
                const uint32_t a = M[i + e], b = V[i + e];
                if (e < 4) {
                    mc.x |= a << (8 * e);
                    vc.x |= b << (8 * e);
                } else {
                    mc.y |= a << (8 * (e - 4));
                    vc.y |= b << (8 * (e - 4));
                }
            }
        }
    }
    decode8(mc, vc, ms, vs, m, r);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        adamw_root_elem(coef != nullptr ? __fmul_rn(g[e], k) : g[e], p[e], m[e], r[e], c);
    if (!whole) {   // places past the tensor's end take no part in the maxima
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e >= n) m[e] = r[e] = 0.0f;
    }
    const BlockScales b = scales_of(m, r);
    encode8(m, r, b, &mc, &vc);
    if ((threadIdx.x & 31) == 0) {
        *MS = b.m_scale;
        *VS = b.r_scale;
    }
    if (whole) {
        stcs16(P + i, pack4f(p));
        stcs16(P + i + 4, pack4f(p + 4));
        stcs8(M + i, mc);
        stcs8(V + i, vc);
        if (O != nullptr)
            stcs16(O + i, make_uint4(pack2<PT>(p[0], p[1]), pack2<PT>(p[2], p[3]),
                                     pack2<PT>(p[4], p[5]), pack2<PT>(p[6], p[7])));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i + e < n) {
                P[i + e] = p[e];
                M[i + e] = static_cast<uint8_t>((e < 4 ? mc.x : mc.y) >> (8 * (e & 3)));
                V[i + e] = static_cast<uint8_t>((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)));
                if (O != nullptr) O[i + e] = pack1<PT>(p[e]);
            }
        }
    }
}

// Codes -> fp32 moments: m = code * scale, v = (code * scale)^2.
__global__ void __launch_bounds__(kListThreads)
    moments_decode(const uint8_t* __restrict__ M, const float* __restrict__ MS,
                   const uint8_t* __restrict__ V, const float* __restrict__ VS, int64_t n,
                   float* __restrict__ Mo, float* __restrict__ Vo, bool vec) {
    pdl_enter();
    const int64_t i = 8 * (static_cast<int64_t>(blockIdx.x) * kListThreads + threadIdx.x);
    if (i >= n) return;
    const int64_t blk = i / kMomentBlock;
    const float ms = __ldg(MS + blk), vs = __ldg(VS + blk);
    float m[8], r[8];
    if (vec && i + 8 <= n) {
        decode8(ldcs8(M + i), ldcs8(V + i), ms, vs, m, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = __fmul_rn(r[e], r[e]);
        stcs16(Mo + i, pack4f(m));
        stcs16(Mo + i + 4, pack4f(m + 4));
        stcs16(Vo + i, pack4f(r));
        stcs16(Vo + i + 4, pack4f(r + 4));
        return;
    }
    for (int e = 0; e < 8 && i + e < n; ++e) {
        Mo[i + e] = __fmul_rn(e4m3x2_to_f32(M[i + e]).x, ms);
        const float x = __fmul_rn(root_to_f32(V[i + e]), vs);
        Vo[i + e] = __fmul_rn(x, x);
    }
}

// fp32 moments -> codes and scales, a warp per block.
__global__ void __launch_bounds__(kListThreads)
    moments_encode(const float* __restrict__ Mi, const float* __restrict__ Vi, int64_t n,
                   uint8_t* __restrict__ M, float* __restrict__ MS, uint8_t* __restrict__ V,
                   float* __restrict__ VS, bool vec) {
    pdl_enter();
    const int64_t blk =
        static_cast<int64_t>(blockIdx.x) * (kListThreads / 32) + (threadIdx.x >> 5);
    const int64_t base = blk * kMomentBlock;
    if (base >= n) return;
    const int64_t i = base + 8 * (threadIdx.x & 31);
    float m[8], r[8];
    const bool whole = vec && base + kMomentBlock <= n;
    if (whole) {
        loadw<kGradF32, 8>(Mi, i, m);
        loadw<kGradF32, 8>(Vi, i, r);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[e] = i + e < n ? Mi[i + e] : 0.0f;
            r[e] = i + e < n ? Vi[i + e] : 0.0f;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = __fsqrt_rn(r[e]);
    const BlockScales b = scales_of(m, r);
    uint2 mc, vc;
    encode8(m, r, b, &mc, &vc);
    if ((threadIdx.x & 31) == 0) {
        MS[blk] = b.m_scale;
        VS[blk] = b.r_scale;
    }
    if (whole) {
        stcs8(M + i, mc);
        stcs8(V + i, vc);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i + e < n) {
                M[i + e] = static_cast<uint8_t>((e < 4 ? mc.x : mc.y) >> (8 * (e & 3)));
                V[i + e] = static_cast<uint8_t>((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)));
            }
        }
    }
}

// ------------------------------------------------------------- the norm

// Sum of a block's doubles in a fixed tree order; the result in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kListThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_down_sync(0xFFFFFFFFu, x, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kListThreads / 32; ++w) s += part[w];
    __syncthreads();
    return s;
}

// Squares are formed and summed in fp32, in 8 sums per thread over the chunks
// a block takes in turn (b, b + gridDim, ...); the threads' sums are joined in
// double in a fixed order, the blocks' likewise by the block that arrives
// last, so the result does not depend on the order in which blocks run.
// Bound by the one read of the gradients.
template <int CAP, int GT>
__global__ void __launch_bounds__(kListThreads)
    tensors_norm(const __grid_constant__ NormTable<CAP> t, const NormArgs a) {
    pdl_enter();
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t chunks = t.b0[t.count];
    int s = blockIdx.x < chunks ? find_tensor(t, blockIdx.x) : 0;
    for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
        while (b >= t.b0[s + 1]) ++s;
        const int64_t n = t.n[s];
        const int64_t base = static_cast<int64_t>(b - t.b0[s]) * kNormChunk;
        const void* G = t.p[s];
        if (t.vec[s] && base + kNormChunk <= n) {
            constexpr int U = kNormChunk / (8 * kListThreads);
            float f[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u)
                loadw<GT, 8>(G, base + 8 * (u * kListThreads + threadIdx.x), f[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = __fmaf_rn(f[u][e], f[u][e], acc[e]);
        } else {
            const int64_t end = base + kNormChunk < n ? base + kNormChunk : n;
            for (int64_t i = base + threadIdx.x; i < end; i += kListThreads) {
                const float x = load1<GT>(G, i);
                acc[0] = __fmaf_rn(x, x, acc[0]);
            }
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += static_cast<double>(acc[e]);
    sum = block_sum(sum);
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
    const int64_t blocks = (n + 8 * kListThreads - 1) / (8 * kListThreads);
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
