// Layer norm over the rows of a matrix, and its gradients.
//
//   xh = (x - mean) r,  r = 1 / sqrt(mean((x - mean)^2) + eps),  out = xh w + b
//   g = d w,  d_x = r (g - mean(g) - xh mean(g xh))
//   d_w = sum over rows of d xh,  d_b = sum over rows of d
//
// Both passes are bound by memory: forward reads x and writes out, backward
// reads x and d and writes d_x; a row stays in registers between its sums and
// its results, so nothing is read twice.  The variance is formed from the
// differences from the mean, not from a sum of squares, so a row far from zero
// keeps its bits.  All sums are fp32 (a thread's terms, then a tree over the
// threads).
//
// Backward, a thread holds the same columns of every row it meets, so their
// d_w and d_b stay in its registers until the block's last row; the blocks'
// sums then go to the workspace and layer_norm_columns adds them in the blocks'
// order.  The grid goes by the sizes and the number of SMs alone, so equal
// calls give equal bits.
//
// Rows too wide for registers (over 16384 columns forward and 8192 backward, or
// 8192 and 4096 where rows are not aligned) are read again for each sum (layer_norm_wide, layer_norm_wide_grad,
// layer_norm_wide_columns).
#include <algorithm>

#include "elem.cuh"

namespace shardstep {
namespace {

constexpr int kNormThreads = 512;   // most threads of a block; whole groups of rows
constexpr uint32_t kFull = 0xFFFFFFFFu;

// Sums of two values over a group of `size` threads (32, 64, .., 512) that take
// one row: shuffles, then one word per warp.  `words` holds 2 x 2 words per
// warp of the block: two banks in turn, so that one barrier a sum is enough.
struct Group {
    int size, warp, first_warp, id;
    float2* words;
    int bank;
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
    }
    __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            a += __shfl_xor_sync(kFull, a, d);
            b += __shfl_xor_sync(kFull, b, d);
        }
        if (size == 32) return make_float2(a, b);
        float2* w = words + bank * (kNormThreads / 32);
        bank ^= 1;
        if (threadIdx.x % 32 == 0) w[warp] = make_float2(a, b);
        sync();
        float2 t = make_float2(0.0f, 0.0f);
        for (int k = 0; k < size / 32; ++k) {
            const float2 v = w[first_warp + k];
            t.x += v.x;
            t.y += v.y;
        }
        return t;
    }
};
__device__ __forceinline__ Group group_of(int size, float2* words) {
    const int g = threadIdx.x / size;
    return Group{size, static_cast<int>(threadIdx.x / 32), g * size / 32, g, words, 0};
}

// The N elements of a row from column c on; those past its end are zeros, and
// are not read.  TAIL: whether a row may end inside a vector.
template <int T, int N, bool TAIL>
__device__ __forceinline__ void load_part(const typename Elem<T>::Store* p, int c, int cols,
                                          float* f) {
    if (!TAIL || c + N <= cols) {
        load_elems<T, N>(p + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = c + j < cols ? elem_to_f32<T>(p[c + j]) : 0.0f;
    }
}
template <int T, int N, bool TAIL>
__device__ __forceinline__ void store_part(typename Elem<T>::Store* p, int c, int cols,
                                           const float* f) {
    if (!TAIL || c + N <= cols) {
        store_elems<T, N>(p + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c + j < cols) p[c + j] = elem_from_f32<T>(f[j]);
    }
}

// V vectors of N elements per thread.
template <int T, int TW, int N, int V, bool TAIL>
__global__ void __launch_bounds__(kNormThreads) layer_norm_rows(const NormRows a, int size) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    Group g = group_of(size, words);
    const int t = threadIdx.x % size, groups = blockDim.x / size;
    const int cols = static_cast<int>(a.cols);
    pdl_enter();
    const float n = static_cast<float>(a.cols);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * groups) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        float f[V][N];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c < cols) {
                load_part<T, N, TAIL>(x, c, cols, f[k]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) f[k][j] = 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) s += f[k][j];
        const float mean = __fdiv_rn(g.sum(s, 0.0f).x, n);   // no rounded 1 / n: rows far from 0
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (TAIL && c + j >= cols) continue;
                f[k][j] -= mean;
                q = fmaf(f[k][j], f[k][j], q);
            }
        }
        const float var = __fdiv_rn(g.sum(q, 0.0f).x, n);
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
        if (t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = r;
        }
        S* out = static_cast<S*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
            float w[N], b[N];
            if (a.w != nullptr) load_part<TW, N, TAIL>(static_cast<const W*>(a.w), c, cols, w);
            if (a.b != nullptr) load_part<TW, N, TAIL>(static_cast<const W*>(a.b), c, cols, b);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float y = f[k][j] * r;
                if (a.w != nullptr) y *= w[j];
                if (a.b != nullptr) y += b[j];
                f[k][j] = y;
            }
            store_part<T, N, TAIL>(out, c, cols, f[k]);
        }
    }
}

// Backward.  Dynamic shared memory: the groups' column sums, where a block has
// more than one group.
template <int T, int TW, int N, int V, bool TAIL, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_rows_grad(const NormGradRows a, int size) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    extern __shared__ float sums[];
    Group g = group_of(size, words);
    const int t = threadIdx.x % size, groups = blockDim.x / size;
    const int cols = static_cast<int>(a.cols);
    pdl_enter();
    const float inv = 1.0f / static_cast<float>(a.cols);
    float dw[V][N] = {}, db[V][N] = {};
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * groups) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        const S* d = static_cast<const S*>(a.d) + row * a.d_stride;
        float xh[V][N], f[V][N];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c < cols) {
                load_part<T, N, TAIL>(x, c, cols, xh[k]);
                load_part<T, N, TAIL>(d, c, cols, f[k]);
            }
        }
        const float mean = __ldg(a.mean + row), r = __ldg(a.rstd + row);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
            float w[N];
            if (a.w != nullptr) load_part<TW, N, TAIL>(static_cast<const W*>(a.w), c, cols, w);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                xh[k][j] = (xh[k][j] - mean) * r;
                dw[k][j] = fmaf(f[k][j], xh[k][j], dw[k][j]);
                db[k][j] += f[k][j];
                if (a.w != nullptr) f[k][j] *= w[j];
                s1 += f[k][j];
                s2 = fmaf(f[k][j], xh[k][j], s2);
            }
        }
        if (a.d_x == nullptr) continue;
        const float2 m = g.sum(s1, s2);
        const float c1 = m.x * inv, c2 = m.y * inv;
        S* dx = static_cast<S*>(a.d_x) + row * a.d_x_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
#pragma unroll
            for (int j = 0; j < N; ++j)
                f[k][j] = r * (f[k][j] - c1 - xh[k][j] * c2);
            store_part<T, N, TAIL>(dx, c, cols, f[k]);
        }
    }
    if (a.piece == nullptr) return;
    // the groups' sums, added in the groups' order
    float* piece = a.piece + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (int q = 0; q < groups; ++q) {
        if (q > 0) __syncthreads();
        if (g.id != q) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (TAIL && c + j >= cols) continue;
                if (q > 0) {
                    dw[k][j] += sums[c + j];
                    db[k][j] += sums[a.cols + c + j];
                }
                float* to = q + 1 < groups ? sums : piece;
                to[c + j] = dw[k][j];
                to[a.cols + c + j] = db[k][j];
            }
        }
    }
}

// d_w and d_b from the blocks' sums: 32 columns per block, a warp takes every
// eighth of the pieces, the warps' sums are added in their order.
template <int TW>
__global__ void __launch_bounds__(256)
    layer_norm_columns(const float* piece, int pieces, int64_t cols, void* d_w, void* d_b,
                       int accumulate) {
    using W = typename Elem<TW>::Store;
    __shared__ float part[8][32];
    pdl_enter();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // of 2 * cols
    float s = 0.0f;
    if (c < 2 * cols) {
        const float* p = piece + c;
        int q = warp;
        for (; q + 24 < pieces; q += 32) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = p[static_cast<int64_t>(q + 8 * k) * 2 * cols];
#pragma unroll
            for (int k = 0; k < 4; ++k) s += f[k];
        }
        for (; q < pieces; q += 8) s += p[static_cast<int64_t>(q) * 2 * cols];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= 2 * cols) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += part[k][lane];
    W* to = static_cast<W*>(c < cols ? d_w : d_b);
    if (to == nullptr) return;
    to += c < cols ? c : c - cols;
    if (accumulate) s += elem_to_f32<TW>(*to);
    *to = elem_from_f32<TW>(s);
}

// ------------------------------------------------------- rows of any width

template <int T, int TW>
__global__ void __launch_bounds__(kNormThreads) layer_norm_wide(const NormRows a) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    Group g = group_of(kNormThreads, words);
    pdl_enter();
    const float n = static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) s += elem_to_f32<T>(x[c]);
        const float mean = __fdiv_rn(g.sum(s, 0.0f).x, n);   // no rounded 1 / n: rows far from 0
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
            const float y = elem_to_f32<T>(x[c]) - mean;
            q = fmaf(y, y, q);
        }
        const float var = __fdiv_rn(g.sum(q, 0.0f).x, n);
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = r;
        }
        S* out = static_cast<S*>(a.out) + row * a.out_stride;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
            float y = (elem_to_f32<T>(x[c]) - mean) * r;
            if (a.w != nullptr) y *= elem_to_f32<TW>(static_cast<const W*>(a.w)[c]);
            if (a.b != nullptr) y += elem_to_f32<TW>(static_cast<const W*>(a.b)[c]);
            out[c] = elem_from_f32<T>(y);
        }
    }
}

template <int T, int TW>
__global__ void __launch_bounds__(kNormThreads) layer_norm_wide_grad(const NormGradRows a) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    Group g = group_of(kNormThreads, words);
    pdl_enter();
    const float inv = 1.0f / static_cast<float>(a.cols);
    const W* w = static_cast<const W*>(a.w);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        const S* d = static_cast<const S*>(a.d) + row * a.d_stride;
        S* dx = static_cast<S*>(a.d_x) + row * a.d_x_stride;
        const float mean = __ldg(a.mean + row), r = __ldg(a.rstd + row);
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
            const float f = elem_to_f32<T>(d[c]) * (w != nullptr ? elem_to_f32<TW>(w[c]) : 1.0f);
            s1 += f;
            s2 = fmaf(f, (elem_to_f32<T>(x[c]) - mean) * r, s2);
        }
        const float2 m = g.sum(s1, s2);
        const float c1 = m.x * inv, c2 = m.y * inv;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
            const float f = elem_to_f32<T>(d[c]) * (w != nullptr ? elem_to_f32<TW>(w[c]) : 1.0f);
            const float xh = (elem_to_f32<T>(x[c]) - mean) * r;
            dx[c] = elem_from_f32<T>(r * (f - c1 - xh * c2));
        }
    }
}

// Column sums of a share of the rows, a thread per column.
template <int T>
__global__ void __launch_bounds__(256) layer_norm_wide_columns(const NormGradRows a) {
    using S = typename Elem<T>::Store;
    pdl_enter();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = elem_to_f32<T>(static_cast<const S*>(a.d)[row * a.d_stride + c]);
        const float x = elem_to_f32<T>(static_cast<const S*>(a.x)[row * a.x_stride + c]);
        dw = fmaf(d, (x - __ldg(a.mean + row)) * __ldg(a.rstd + row), dw);
        db += d;
    }
    float* piece = a.piece + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    piece[c] = dw;
    piece[a.cols + c] = db;
}

// ----------------------------------------------------------------- launches

// Threads that take one row of `held` elements each; 0: too wide.
int fit_group(int64_t cols, int most, int held) {
    for (int s = 32; s <= most; s *= 2)
        if (static_cast<int64_t>(s) * held >= cols) return s;
    return 0;
}

// A thread holds up to 32 elements of a row in vectors (4 of 16 bits, 8 of fp32),
// or 16 single ones where rows are not aligned; backward, with their columns'
// sums, 32 or 8 (up to 200 and 128 registers), 256 or 512 threads to a block.
int fit_rows(int64_t cols, bool vec) { return fit_group(cols, kNormThreads, vec ? 32 : 16); }
int grad_threads(bool vec) { return vec ? 256 : 512; }
int fit_grad(int64_t cols, bool vec) { return fit_group(cols, grad_threads(vec), vec ? 32 : 8); }

template <int T, int TW>
cudaError_t go_rows(const NormRows& a, bool vec, cudaStream_t stream) {
    const int size = fit_rows(a.cols, vec);
    const int64_t most = static_cast<int64_t>(device_sms()) * 8;
    if (size == 0)
        return launch_after(layer_norm_wide<T, TW>,
                            dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                            dim3(kNormThreads), 0, stream, a);
    const int threads = size > 128 ? size : 128;
    const int64_t blocks = (a.rows + threads / size - 1) / (threads / size);
    const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
    constexpr int N = Elem<T>::kVec;
    const auto go = [&](auto* kernel) {
        return launch_after(kernel, grid, dim3(threads), 0, stream, a, size);
    };
    return !vec              ? go(layer_norm_rows<T, TW, 1, 16, false>)
           : a.cols % N == 0 ? go(layer_norm_rows<T, TW, N, 32 / N, false>)
                             : go(layer_norm_rows<T, TW, N, 32 / N, true>);
}

template <int T, int TW>
cudaError_t go_rows_grad(const NormGradRows& a, int size, int blocks, bool vec,
                         cudaStream_t stream) {
    constexpr int N = Elem<T>::kVec;
    const int threads = grad_threads(vec);
    const size_t smem = threads > size ? sizeof(float) * 2 * a.cols : 0;   // 32 KB at most
    const auto go = [&](auto* kernel) {
        return launch_after(kernel, dim3(blocks), dim3(threads), smem, stream, a, size);
    };
    return !vec              ? go(layer_norm_rows_grad<T, TW, 1, 8, false, 512>)
           : a.cols % N == 0 ? go(layer_norm_rows_grad<T, TW, N, 32 / N, false, 256>)
                             : go(layer_norm_rows_grad<T, TW, N, 32 / N, true, 256>);
}

template <int T, int TW>
cudaError_t go_grad(const NormGradRows& a, void* d_w, void* d_b, int accumulate, bool vec,
                    cudaStream_t stream) {
    const int size = fit_grad(a.cols, vec);
    const int pieces = norm_pieces(a.rows, a.cols, vec);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && size != 0) {
        e = go_rows_grad<T, TW>(a, size, pieces, vec, stream);
        note_launch();
    } else if (a.rows > 0) {
        if (a.d_x != nullptr) {
            const int64_t most = static_cast<int64_t>(device_sms()) * 4;
            e = launch_after(layer_norm_wide_grad<T, TW>,
                             dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                             dim3(kNormThreads), 0, stream, a);
            note_launch();
        }
        if (e == cudaSuccess && a.piece != nullptr) {
            e = launch_after(layer_norm_wide_columns<T>,
                             dim3(static_cast<unsigned>((a.cols + 255) / 256), pieces), dim3(256),
                             0, stream, a);
            note_launch();
        }
    }
    if (e != cudaSuccess || a.piece == nullptr) return e;
    e = launch_after(layer_norm_columns<TW>, dim3(static_cast<unsigned>((2 * a.cols + 31) / 32)),
                     dim3(256), 0, stream, static_cast<const float*>(a.piece), pieces, a.cols, d_w,
                     d_b, accumulate);
    note_launch();
    return e;
}

// Weights have the rows' type or fp32.
template <typename F>
cudaError_t by_types(int type, int w_type, F&& f) {
    return by_type(type, [&](auto t) {
        return w_type == kGradF32 ? f(t, Const<kGradF32>()) : f(t, t);
    });
}

}  // namespace

// Blocks of the backward pass, each of which leaves one row of column sums.
int norm_pieces(int64_t rows, int64_t cols, bool vec) {
    const int size = fit_grad(cols, vec);
    if (rows == 0) return 0;
    if (size == 0) return static_cast<int>(rows < 64 ? rows : 64);
    const int groups = grad_threads(vec) / size;
    const int64_t most = std::min(device_sms(), kNormPieces);
    const int64_t need = (rows + groups - 1) / groups;
    return static_cast<int>(need < most ? need : most);
}

cudaError_t launch_layer_norm(const NormRows& a, int type, int w_type, bool vec,
                              cudaStream_t stream) {
    const cudaError_t e = by_types(type, w_type, [&](auto t, auto w) {
        return go_rows<decltype(t)::value, decltype(w)::value>(a, vec, stream);
    });
    note_launch();
    return e;
}

cudaError_t launch_layer_norm_grad(const NormGradRows& a, int type, int w_type, void* d_w,
                                   void* d_b, int accumulate, bool vec, cudaStream_t stream) {
    return by_types(type, w_type, [&](auto t, auto w) {
        return go_grad<decltype(t)::value, decltype(w)::value>(a, d_w, d_b, accumulate, vec,
                                                               stream);
    });
}

}  // namespace shardstep
