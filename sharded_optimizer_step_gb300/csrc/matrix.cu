// Orthogonalised updates of matrices: the Newton-Schulz quintic iteration
//
//   X = u / (|u| + eps)            (transposed where u is taller than wide)
//   A = X X^T,  B = b A + c A A,   X = a X + B X     `rounds` times
//
// over a list of matrices, as such or as an optimizer's step.  Three grouped
// products a round, one launch each for all matrices of a group; A and B are
// symmetric, so the first two compute the tiles on and above the diagonal and
// write each off-diagonal one to both places.
//
// The tensor cores multiply halves; to keep single precision each value v is
// held as two, hi = half(s v) and lo = half(s v - hi) with s a power of two: 22
// bits, of which three products hi hi + hi lo + lo hi make a product good to
// about 2^-21 (one product of single halves loses 2e-3 to 2e-2 of the result
// over five rounds, these three 1e-6).  s is 2^15 for X and A, whose elements
// stay below sqrt(2) and 2, and 2^14 for B, below 4 (the host checks the
// coefficients for it): nothing overflows, and an element of rms 1 / sqrt(m n),
// the smallest that occurs throughout, still has its 22 bits at m n = 2^30.
//
// Layout.  All operands live in the workspace as the images of what shared
// memory holds: blocks of 128 rows x 64 columns, 16 KB of hi then 16 KB of lo,
// rows of 128 bytes in the tensor cores' 128-byte swizzle.  A tile's operands
// are then whole contiguous pieces, copied by bulk copies without a tensor map,
// and one block serves both as rows of k (X and A times their transposes) and
// as k rows (X behind B).  Both sides are padded to 128 with zeros, which the
// products keep zero.
#include "elem.cuh"
#include "tcgen05.cuh"

namespace shardstep {
namespace {

__device__ unsigned int g_matrix_status;

constexpr int kTile = 128;                    // of the results, both ways
constexpr int kBlockBytes = 32768;            // 128 x 64 halves, hi and lo
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kBlockBytes;
constexpr int kMatrixThreads = 192;           // producer, products, four warps of results
constexpr int kTmemColumns = 256;             // two accumulators of 128
// The tensor cores cut sums off at fp32's last bit instead of rounding them, so a
// long sum of positive terms (a row's square) falls behind by K / 16 times half a
// bit.  A sum over k therefore goes in pieces of this many, which the result warps
// add up in their registers (rounding to nearest).
constexpr int kPiece = 512;
constexpr float kScaleX = 32768.0f, kScaleB = 16384.0f;

enum class Step { kGram, kPoly, kApply, kLast };

struct Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t done[2], taken[2];               // an accumulator is complete / has been read
    uint64_t drain;
    uint32_t tmem;
};

// Byte offset of element (row, col) within an image block's hi half.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t col) {
    return row * 128 + (((col / 8) ^ (row % 8)) * 16) + (col % 8) * 2;
}
// The image block that holds (row, col); `width` columns, padded.
__device__ __forceinline__ char* block_at(void* image, int row, int col, int width) {
    return static_cast<char*>(image) +
           (static_cast<int64_t>(row / 128) * (width / 64) + col / 64) * kBlockBytes;
}
__device__ __forceinline__ const char* block_at(const void* image, int row, int col, int width) {
    return block_at(const_cast<void*>(image), row, col, width);
}

struct Halves {
    uint16_t hi, lo;
};
__device__ __forceinline__ Halves split(float v) {
    const __half h = __float2half_rn(v);
    return Halves{__half_as_ushort(h), __half_as_ushort(__float2half_rn(v - __half2float(h)))};
}
__device__ __forceinline__ void split_pair(float a, float b, uint32_t* hi, uint32_t* lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
}

// The matrix of a tile, by the first tiles of the list.
__device__ __forceinline__ int find(const uint32_t* first, int count, uint32_t tile) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct Tile {
    int matrix, row, col;    // of the result, in elements
    int k;                   // length of the sum
};
template <Step STEP>
__device__ __forceinline__ Tile tile_at(const MatrixTable& t, uint32_t index) {
    constexpr bool sym = STEP == Step::kGram || STEP == Step::kPoly;
    const uint32_t* first = sym ? t.sym0 : t.full0;
    Tile out;
    out.matrix = find(first, t.count, index);
    const MatrixItem& x = t.item[out.matrix];
    int i = static_cast<int>(index - first[out.matrix]);
    const int side = x.mp / kTile;
    if constexpr (sym) {
        int r = 0;
        while (i >= side - r) i -= side - r++;
        out.row = r * kTile;
        out.col = (r + i) * kTile;
    } else {          // the rows of a column first: they share X's columns
        out.row = i % side * kTile;
        out.col = i / side * kTile;
    }
    out.k = STEP == Step::kGram ? x.np : x.mp;
    return out;
}

// ------------------------------------------------------------------ results

// 32 columns of a thread's row, as halves of s v, to an image.
__device__ __forceinline__ void store_row(void* image, int row, int col, int width,
                                          const float* v) {
    char* block = block_at(image, row, col, width);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint4 hi, lo;
        split_pair(v[8 * k], v[8 * k + 1], &hi.x, &lo.x);
        split_pair(v[8 * k + 2], v[8 * k + 3], &hi.y, &lo.y);
        split_pair(v[8 * k + 4], v[8 * k + 5], &hi.z, &lo.z);
        split_pair(v[8 * k + 6], v[8 * k + 7], &hi.w, &lo.w);
        char* p = block + swizzled(row % 128, col % 64 + 8 * k);
        *reinterpret_cast<uint4*>(p) = hi;
        *reinterpret_cast<uint4*>(p + kBlockBytes / 2) = lo;
    }
}
// The same values to the mirrored place: lanes are consecutive columns there.
__device__ __forceinline__ void store_mirrored(void* image, int row, int col, int width,
                                               const float* v) {
    char* block = block_at(image, col, row, width);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const Halves h = split(v[k]);
        char* p = block + swizzled(col % 128 + k, row % 64);
        *reinterpret_cast<uint16_t*>(p) = h.hi;
        *reinterpret_cast<uint16_t*>(p + kBlockBytes / 2) = h.lo;
    }
}
// s v of 32 columns of a row.
__device__ __forceinline__ void load_row(const void* image, int row, int col, int width,
                                         float* v) {
    const char* block = block_at(image, row, col, width);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const char* p = block + swizzled(row % 128, col % 64 + 8 * k);
        float hi[8], lo[8];
        unpack16<kGradF16>(*reinterpret_cast<const uint4*>(p), hi);
        unpack16<kGradF16>(*reinterpret_cast<const uint4*>(p + kBlockBytes / 2), lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * k + j] = hi[j] + lo[j];
    }
}

// The last round's results: an output, or the step of the weights.
__device__ __forceinline__ void finish(const MatrixItem& x, const MatrixCall& c, int row, int col,
                                       const float* v) {
    const MatrixGroup& g = c.group[x.group];
    if (row >= x.m) return;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        if (col + k >= x.n) continue;
        const int64_t at = x.tall ? static_cast<int64_t>(col + k) * x.m + row
                                  : static_cast<int64_t>(row) * x.n + col + k;
        if (x.master != nullptr) {
            float p = x.master[at];
            p -= g.lr_wd * p;
            p -= x.step * v[k];
            x.master[at] = p;
            if (x.out == nullptr) continue;
            if (c.out_type == kGradF16) static_cast<uint16_t*>(x.out)[at] = elem_from_f32<kGradF16>(p);
            else static_cast<uint16_t*>(x.out)[at] = f32_to_bf16(p);
        } else if (c.out_type == kGradF32) {
            static_cast<float*>(x.out)[at] = v[k];
        } else {
            static_cast<uint16_t*>(x.out)[at] =
                c.out_type == kGradF16 ? elem_from_f32<kGradF16>(v[k]) : f32_to_bf16(v[k]);
        }
    }
}

// ----------------------------------------------------------------- products

// One block per SM walks the tiles.  Warp 0 copies operands into a ring of
// stages, warp 1 issues the products into one of two accumulators, warps 2 to 5
// turn the other into results.  Every wait has a limit: past it the block sets
// the status word, lets its copies and products in flight end, frees its tensor
// memory and returns.
template <Step STEP>
__global__ void __launch_bounds__(kMatrixThreads, 1)
    matrix_product(const __grid_constant__ MatrixTable t,
                   const __grid_constant__ MatrixCall call, int from,
                   unsigned long long limit_ns) {
    extern __shared__ char raw[];
    __shared__ Shared sh;
    char* ring = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    constexpr bool sym = STEP == Step::kGram || STEP == Step::kPoly;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t tiles = sym ? t.sym0[t.count] : t.full0[t.count];
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&sh.done[k], 1);
            mbar_init(&sh.taken[k], 4);
        }
        mbar_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<kTmemColumns>(&sh.tmem);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_enter();
    const bool skip = skip_step(call.skip);

    if (!skip && warp == 0) {
        if (lane == 0) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            uint32_t issued = 0;
            bool ok = true;
            for (uint32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
                const Tile at = tile_at<STEP>(t, i);
                const MatrixItem& x = t.item[at.matrix];
                const void* left = STEP == Step::kGram   ? x.x[from]
                                   : STEP == Step::kPoly ? x.gram
                                                         : x.poly;
                for (int k = 0; k < at.k; k += 64, ++issued) {
                    const uint32_t s = issued % kStages;
                    if (issued >= kStages &&
                        !mbar_wait(&sh.empty[s], (issued / kStages - 1) & 1, limit_ns)) {
                        ok = false;
                        break;
                    }
                    char* to = ring + s * kStageBytes;
                    mbar_expect_tx(&sh.full[s], kStageBytes);
                    bulk_load(to, block_at(left, at.row, k, at.k), kBlockBytes, &sh.full[s]);
                    to += kBlockBytes;
                    if constexpr (sym) {
                        bulk_load(to, block_at(left, at.col, k, at.k), kBlockBytes, &sh.full[s]);
                    } else {
                        // 64 rows of each of two blocks: hi of both, then lo of both
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            bulk_load(to + j * 8192,
                                      block_at(x.x[from], k, at.col + j % 2 * 64, x.np) +
                                          j / 2 * (kBlockBytes / 2) + k % 128 * 128,
                                      8192, &sh.full[s]);
                    }
                }
            }
            if (!ok) atomicOr(&g_matrix_status, kStatusProducerTimeout);
            // the last copies of every stage land before the block's memory goes
            for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                if (!mbar_wait(&sh.full[j % kStages], (j / kStages) & 1, kDrainNs))
                    atomicOr(&g_matrix_status, kStatusDrainTimeout);
        }
    } else if (!skip && warp == 1) {
        if (lane == 0) {
            constexpr uint32_t form = half_product(kTile, kTile, !sym);
            uint32_t used = 0, n = 0;                     // stages, pieces
            bool ok = true;
            for (uint32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
                const Tile at = tile_at<STEP>(t, i);
                for (int k0 = 0; ok && k0 < at.k; k0 += kPiece, ++n) {
                    const uint32_t d = tmem + n % 2 * kTile;
                    if (n >= 2 && !mbar_wait(&sh.taken[n % 2], (n / 2 - 1) & 1, limit_ns)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const int end = at.k - k0 < kPiece ? at.k : k0 + kPiece;
                    for (int k = k0; k < end; k += 64, ++used) {
                        const uint32_t s = used % kStages;
                        if (!mbar_wait(&sh.full[s], (used / kStages) & 1, limit_ns)) {
                            ok = false;
                            break;
                        }
                        tmem_fence_after();
                        const uint32_t a = smem_addr(ring + s * kStageBytes);
                        const uint32_t b = a + kBlockBytes;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {      // 16 of k each
                            const uint64_t ah = k_major(a + q * 32);
                            const uint64_t al = k_major(a + kBlockBytes / 2 + q * 32);
                            const uint64_t bh =
                                sym ? k_major(b + q * 32) : mn_major(b + q * 2048, 8192);
                            const uint64_t bl =
                                sym ? k_major(b + kBlockBytes / 2 + q * 32)
                                    : mn_major(b + kBlockBytes / 2 + q * 2048, 8192);
                            mma_half(d, ah, bh, form, k > k0 || q > 0);
                            mma_half(d, ah, bl, form, true);
                            mma_half(d, al, bh, form, true);
                        }
                        mma_commit(&sh.empty[s]);
                    }
                    if (ok) mma_commit(&sh.done[n % 2]);
                }
            }
            if (!ok) atomicOr(&g_matrix_status, kStatusConsumerTimeout);
            mma_commit(&sh.drain);          // the products in flight end before their memory goes
            if (!mbar_wait(&sh.drain, 0, kDrainNs))
                atomicOr(&g_matrix_status, kStatusDrainTimeout);
        }
    } else if (!skip) {
        const int quarter = warp % 4;                    // the lanes this warp may read
        uint32_t n = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
            const Tile at = tile_at<STEP>(t, i);
            const MatrixItem& x = t.item[at.matrix];
            float sum[kTile / 32][32] = {};
            for (int k0 = 0; k0 < at.k; k0 += kPiece, ++n) {
                // every lane waits, so that all of them see the products
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.done[n % 2], (n / 2) & 1, limit_ns));
                if (!ok) break;
                tmem_fence_after();
#pragma unroll
                for (int c = 0; c < kTile / 32; ++c) {
                    uint32_t acc[32];
                    tmem_load32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                    n % 2 * kTile + c * 32,
                                acc);
#pragma unroll
                    for (int k = 0; k < 32; ++k) sum[c][k] += __uint_as_float(acc[k]);
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.taken[n % 2]);   // the next products may come
            }
            if (!ok) {
                atomicOr(&g_matrix_status, kStatusConsumerTimeout);
                break;
            }
            const int row = at.row + quarter * 32 + lane;
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c) {
                float* v = sum[c];
                const int col = at.col + c * 32;
                if constexpr (STEP == Step::kGram) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= 1.0f / kScaleX;
                    store_row(x.gram, row, col, x.mp, v);
                    if (at.row != at.col) store_mirrored(x.gram, row, col, x.mp, v);
                } else if constexpr (STEP == Step::kPoly) {
                    float g[32];
                    load_row(x.gram, row, col, x.mp, g);
                    const float b = call.b * (kScaleB / kScaleX);
                    const float c2 = call.c * (kScaleB / kScaleX / kScaleX);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = fmaf(c2, v[k], b * g[k]);
                    store_row(x.poly, row, col, x.mp, v);
                    if (at.row != at.col) store_mirrored(x.poly, row, col, x.mp, v);
                } else {
                    float y[32];
                    load_row(x.x[from], row, col, x.np, y);
                    constexpr float out = STEP == Step::kLast ? 1.0f / kScaleX : 1.0f;
                    const float a = call.a * out, p = out / kScaleB;
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = fmaf(p, v[k], a * y[k]);
                    if constexpr (STEP == Step::kLast) finish(x, call, row, col, v);
                    else store_row(x.x[from ^ 1], row, col, x.np, v);
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_fence_after();
        tmem_free<kTmemColumns>(tmem);
    }
}

// --------------------------------------------------- moments, norms, images

// u of element i from the gradient and the new momentum.
template <int T>
__device__ __forceinline__ float update_of(const MatrixItem& x, const MatrixGroup& g, float coef,
                                           float grad, float m) {
    if (x.m_buf == nullptr) return grad;
    return g.nesterov ? fmaf(g.mu, m, g.one_mu * (grad * coef)) : m;
}

// The momentum, and each part's sum of the update's squares.
template <int T>
__global__ void __launch_bounds__(256) matrix_moments(const __grid_constant__ MatrixTable t,
                                                      const MatrixCall call) {
    using S = typename Elem<T>::Store;
    __shared__ double warp_sum[8];
    pdl_enter();
    if (skip_step(call.skip)) return;
    const int k = find(t.part0, t.count, blockIdx.x);
    const MatrixItem& x = t.item[k];
    const MatrixGroup& g = call.group[x.group];
    const int part = blockIdx.x - t.part0[k], parts = t.part0[k + 1] - t.part0[k];
    const float coef = call.coef != nullptr ? __ldg(call.coef) : 1.0f;
    const int64_t n = static_cast<int64_t>(x.m) * x.n;
    const S* grad = static_cast<const S*>(x.grad);
    float sum = 0.0f;
    for (int64_t i = static_cast<int64_t>(part) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(parts) * 256) {
        const float d = elem_to_f32<T>(grad[i]);
        float m = 0.0f;
        if (x.m_buf != nullptr) {
            m = fmaf(g.mu, x.m_buf[i], g.one_mu * (d * coef));
            x.m_buf[i] = m;
        }
        const float u = update_of<T>(x, g, coef, d, m);
        sum = fmaf(u, u, sum);
    }
    double s = sum;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 8; ++w) s += warp_sum[w];
    x.part[part] = s;
}

// X's image: a block of it per thread block.
template <int T>
__global__ void __launch_bounds__(256) matrix_image(const __grid_constant__ MatrixTable t,
                                                    const MatrixCall call) {
    using S = typename Elem<T>::Store;
    __shared__ double warp_sum[8];
    pdl_enter();
    if (skip_step(call.skip)) return;
    const int k = find(t.image0, t.count, blockIdx.x);
    const MatrixItem& x = t.item[k];
    const MatrixGroup& g = call.group[x.group];
    const int parts = t.part0[k + 1] - t.part0[k];
    double s = threadIdx.x < parts ? x.part[threadIdx.x] : 0.0;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += warp_sum[w];
    // a sum that is not finite leaves nothing finite
    const float scale = s <= 1.7976931348623157e308
                            ? static_cast<float>(kScaleX / (sqrt(s) + call.eps))
                            : __int_as_float(0x7FFFFFFF);
    const float coef = call.coef != nullptr ? __ldg(call.coef) : 1.0f;
    const S* grad = static_cast<const S*>(x.grad);
    const int block = blockIdx.x - t.image0[k], wide = x.np / 64;
    const int row0 = block / wide * 128, col0 = block % wide * 64;
    char* to = static_cast<char*>(x.x[0]) + static_cast<int64_t>(block) * kBlockBytes;
    for (int q = threadIdx.x; q < 1024; q += 256) {
        // eight columns of a row; consecutive threads along what memory has in a row
        const int r = x.tall ? q % 128 : q / 8, c = x.tall ? q / 128 * 8 : q % 8 * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = row0 + r, col = col0 + c + j;
            v[j] = 0.0f;
            if (row < x.m && col < x.n) {
                const int64_t i = x.tall ? static_cast<int64_t>(col) * x.m + row
                                         : static_cast<int64_t>(row) * x.n + col;
                v[j] = scale * update_of<T>(x, g, coef, elem_to_f32<T>(grad[i]),
                                            x.m_buf != nullptr ? x.m_buf[i] : 0.0f);
            }
        }
        uint4 hi, lo;
        split_pair(v[0], v[1], &hi.x, &lo.x);
        split_pair(v[2], v[3], &hi.y, &lo.y);
        split_pair(v[4], v[5], &hi.z, &lo.z);
        split_pair(v[6], v[7], &hi.w, &lo.w);
        char* p = to + swizzled(r, c);
        *reinterpret_cast<uint4*>(p) = hi;
        *reinterpret_cast<uint4*>(p + kBlockBytes / 2) = lo;
    }
}

template <Step STEP>
cudaError_t go_product(const MatrixTable& t, const MatrixCall& c, int from, cudaStream_t stream) {
    constexpr bool sym = STEP == Step::kGram || STEP == Step::kPoly;
    const uint32_t tiles = sym ? t.sym0[t.count] : t.full0[t.count];
    const uint32_t sms = static_cast<uint32_t>(device_sms());
    constexpr int smem = kStages * kStageBytes + 1024;
    cudaError_t e = cudaFuncSetAttribute(matrix_product<STEP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_after(matrix_product<STEP>, dim3(tiles < sms ? tiles : sms), dim3(kMatrixThreads),
                     smem, stream, t, c, from, tma_wait_limit());
    note_launch();
    return e;
}

}  // namespace

cudaError_t read_matrix_status(unsigned int* status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_matrix_status, sizeof(unsigned int));
    if (e != cudaSuccess || !clear) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_matrix_status, &zero, sizeof(unsigned int));
}

cudaError_t launch_matrices(const MatrixTable& t, const MatrixCall& c, int grad_type,
                            cudaStream_t stream) {
    cudaError_t e = by_type(grad_type, [&](auto type) {
        constexpr int T = decltype(type)::value;
        const cudaError_t first =
            launch_after(matrix_moments<T>, dim3(t.part0[t.count]), dim3(256), 0, stream, t, c);
        note_launch();
        if (first != cudaSuccess) return first;
        const cudaError_t second =
            launch_after(matrix_image<T>, dim3(t.image0[t.count]), dim3(256), 0, stream, t, c);
        note_launch();
        return second;
    });
    for (int k = 0; e == cudaSuccess && k < c.rounds; ++k) {
        e = go_product<Step::kGram>(t, c, k & 1, stream);
        if (e == cudaSuccess) e = go_product<Step::kPoly>(t, c, k & 1, stream);
        if (e != cudaSuccess) return e;
        e = k + 1 < c.rounds ? go_product<Step::kApply>(t, c, k & 1, stream)
                             : go_product<Step::kLast>(t, c, k & 1, stream);
    }
    return e;
}

}  // namespace shardstep
