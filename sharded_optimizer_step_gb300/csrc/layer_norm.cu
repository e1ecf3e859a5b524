// Layer norm over the rows of a matrix, and its gradients.
//
//   xh = (x - mean) r,  r = 1 / sqrt(mean((x - mean)^2) + eps),  out = xh w + b
//   g = d w,  d_x = r (g - mean(g) - xh mean(g xh))
//   d_w = sum over rows of d xh,  d_b = sum over rows of d
//
// Both passes move each row once: forward reads x and writes out, backward reads x
// and d and writes d_x.  The variance is formed from the differences from the mean,
// not from a sum of squares, so a row far from zero keeps its bits.  All sums are fp32
// (a thread's terms, then a tree over the threads).
//
// Forward, a row stays in registers as it is in memory (layer_norm_vectors: 16384 rows
// of 4096 bf16 in 58 to 61 us, 4.4 TB/s; 20 instructions an element and 6 blocks a SM,
// bound by their latency).  Backward, rows come through shared memory some 190 KB ahead
// (layer_norm_staged_grad and layer_norm_columns: 82 to 85 us together, 4.8 TB/s; 27
// instructions an element, issue slots 53% busy, 16 warps a SM for their registers).  Where
// only the results' rows take no vectors, consecutive threads write consecutive elements:
// forward by turning each warp's, backward from the shared rows (with turned ones 27.5 us at
// 999 x 5003 fp32 and 137 at 16384 x 4096 bf16 instead of 23.7 and 112: there are no
// registers for it).  A thread holds the same columns of every row it meets, so their d_w and
// d_b stay in its registers until the block's last row; the blocks' sums then go to the
// workspace and layer_norm_columns adds them in the blocks' order.  The grid goes by the
// sizes and the number of SMs alone, so equal calls give equal bits.
//
// Rows that are not 16-byte aligned take single elements (layer_norm_elements, up to
// 8192 columns forward and 4096 backward); wider rows (over 16384 forward and 8192
// backward where they are aligned) are read again for each sum (layer_norm_wide,
// layer_norm_wide_grad, layer_norm_wide_columns).
#include <algorithm>

#include "elem.cuh"
#include "pairs.cuh"
#include "tma.cuh"

namespace shardstep {
namespace {

constexpr int kNormThreads = 512;   // most threads of a block; whole groups of rows
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ unsigned int g_norm_status;

// Sums of one or two values over a group of `size` threads (32, 64, .., 512) that take
// one row: shuffles, then a word or two per warp.  `words` holds 2 x 2 words per
// warp of the block: two banks in turn, so that one barrier a sum is enough.
// ALONE: the group is its block.  (A barrier whose number is not known when the kernel
// is compiled takes all sixteen of a block, and an SM has 64.)
template <bool ALONE>
struct Group {
    int size, warp, first_warp, id;
    float2* words;
    int bank;
    __device__ __forceinline__ void sync() const {
        if constexpr (ALONE) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
    }
    __device__ __forceinline__ float sum(float a) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) a += __shfl_xor_sync(kFull, a, d);
        if (size == 32) return a;
        float* w = reinterpret_cast<float*>(words + bank * (blockDim.x / 32));
        bank ^= 1;
        if (threadIdx.x % 32 == 0) w[warp] = a;
        sync();
        float t = 0.0f;
        for (int k = 0; k < size / 32; ++k) t += w[first_warp + k];
        return t;
    }
    __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            a += __shfl_xor_sync(kFull, a, d);
            b += __shfl_xor_sync(kFull, b, d);
        }
        if (size == 32) return make_float2(a, b);
        float2* w = words + bank * (blockDim.x / 32);
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
template <bool ALONE>
__device__ __forceinline__ Group<ALONE> group_of(int size, float2* words) {
    const int g = ALONE ? 0 : threadIdx.x / size;
    return Group<ALONE>{size, static_cast<int>(threadIdx.x / 32), g * size / 32, g, words, 0};
}

// A row as it is in memory: V vectors of N elements per thread (N 1: elements), and
// two of its values at a time.
template <int T, int N>
struct Raw {
    uint4 v;
    __device__ __forceinline__ Pair pair(int j) const {
        if constexpr (T == kGradF32) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            return make_pair(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if constexpr (T == kGradF16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                return make_pair(f.x, f.y);
            } else {
                return make_pair(bf16_lo(w[j]), bf16_hi(w[j]));
            }
        }
    }
};
template <int TW, int N>
__device__ __forceinline__ void load_weights(const void* p, int c, Pair* w) {
    float f[N];
    load_elems<TW, N>(static_cast<const typename Elem<TW>::Store*>(p) + c, f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) w[j] = make_pair(f[2 * j], f[2 * j + 1]);
}

// A warp's 32 vectors of a row, `c` this lane's column, into elements: consecutive lanes
// write consecutive ones below `cols`.  All lanes of the warp call it.  (999 rows of 5003
// fp32 between padded ones and packed ones: forward 13.2 us; 17.9 where whole rows wait in
// shared memory to be written element by element, 27 where they are read that way too.)
template <int T, int N>
__device__ __forceinline__ void store_turned(typename Elem<T>::Store* row, int c, int cols,
                                             const float* f, uint4* turn) {
    const int lane = threadIdx.x % 32;
    uint4* mine = turn + threadIdx.x / 32 * 32;
    mine[lane] = pack16<T>(f);
    __syncwarp();
    const auto* from = reinterpret_cast<const typename Elem<T>::Store*>(mine);
    const int first = c - lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (first + 32 * i + lane < cols) row[first + 32 * i + lane] = from[32 * i + lane];
    __syncwarp();
}

// Rows of vectors: kept as they are in memory (16 registers for 32 elements of 16
// bits), so that twice as many rows are on their way as with fp32 copies of them.
// TAIL: a row ends inside a vector, whose elements go to the first threads one each.
// WHOLE: out's rows take vectors; else a warp turns its 32 vectors into elements through
// shared memory, so that consecutive lanes write consecutive ones.
template <int T, int TW, bool ALONE, bool TAIL, bool WHOLE>
__global__ void __launch_bounds__(ALONE ? kNormThreads : 128,
                                  T == kGradF32 ? 1 : ALONE ? 2 : WHOLE ? 8 : 6)
    layer_norm_vectors(const NormRows a, int size) {
    using S = typename Elem<T>::Store;
    constexpr int N = Elem<T>::kVec, V = 32 / N;
    __shared__ float2 words[2 * kNormThreads / 32];
    __shared__ uint4 turn[WHOLE ? 1 : ALONE ? kNormThreads : 128];
    Group<ALONE> g = group_of<ALONE>(size, words);
    const int t = ALONE ? threadIdx.x : threadIdx.x % 32;
    const int groups = ALONE ? 1 : blockDim.x / 32;
    const float n = static_cast<float>(a.cols);
    const int cols = static_cast<int>(a.cols) / N * N;           // in whole vectors
    const bool mine = TAIL && cols + t < static_cast<int>(a.cols);
    pdl_enter();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id;
    if (row >= a.rows) return;   // a whole warp, or no one of the block
    const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
    Raw<T, N> raw[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = (t + k * size) * N;
        raw[k].v = c < cols ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
    float end = mine ? elem_to_f32<T>(x[cols + t]) : 0.0f;
    Pair sum = make_pair(end, 0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) sum = add2(sum, raw[k].pair(j));
    // no rounded 1 / n: rows far from 0
    const float mean = __fdiv_rn(g.sum(floats(sum).x + floats(sum).y), n);
    const Pair off = make_pair(-mean, -mean);
    if (mine) end -= mean;
    sum = make_pair(end * end, 0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if ((t + k * size) * N >= cols) continue;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const Pair d = add2(raw[k].pair(j), off);
            sum = fma2(d, d, sum);
        }
    }
    const float var = __fdiv_rn(g.sum(floats(sum).x + floats(sum).y), n);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
    if (t == 0) {
        a.mean[row] = mean;
        a.rstd[row] = r;
    }
    S* out = static_cast<S*>(a.out) + row * a.out_stride;
    const Pair r2 = make_pair(r, r);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = (t + k * size) * N;
        if (WHOLE ? c >= cols : c - threadIdx.x % 32 * N >= cols) continue;   // or the warp's
        Pair y[N / 2], w[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) y[j] = mul2(add2(raw[k].pair(j), off), r2);
        if (a.w != nullptr && (WHOLE || c < cols)) {
            load_weights<TW, N>(a.w, c, w);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) y[j] = mul2(y[j], w[j]);
        }
        if (a.b != nullptr && (WHOLE || c < cols)) {
            load_weights<TW, N>(a.b, c, w);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) y[j] = add2(y[j], w[j]);
        }
        float f[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            f[2 * j] = floats(y[j]).x;
            f[2 * j + 1] = floats(y[j]).y;
        }
        if constexpr (WHOLE) {
            store_elems<T, N>(out + c, f);
        } else {
            store_turned<T, N>(out, c, cols, f, turn);
        }
    }
    if (!mine) return;
    using W = typename Elem<TW>::Store;
    end *= r;
    if (a.w != nullptr) end *= elem_to_f32<TW>(static_cast<const W*>(a.w)[cols + t]);
    if (a.b != nullptr) end += elem_to_f32<TW>(static_cast<const W*>(a.b)[cols + t]);
    out[cols + t] = elem_from_f32<T>(end);
}

// Rows that are not aligned: V single elements per thread.
template <int T, int TW, int V>
__global__ void __launch_bounds__(kNormThreads) layer_norm_elements(const NormRows a, int size) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    Group<false> g = group_of<false>(size, words);
    const int t = threadIdx.x % size, groups = blockDim.x / size;
    const int cols = static_cast<int>(a.cols);
    pdl_enter();
    const float n = static_cast<float>(a.cols);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * groups) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        float f[V];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = t + k * size;
            f[k] = c < cols ? elem_to_f32<T>(x[c]) : 0.0f;
            s += f[k];
        }
        const float mean = __fdiv_rn(g.sum(s), n);   // no rounded 1 / n: rows far from 0
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (t + k * size >= cols) continue;
            f[k] -= mean;
            q = fmaf(f[k], f[k], q);
        }
        const float var = __fdiv_rn(g.sum(q), n);
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
        if (t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = r;
        }
        S* out = static_cast<S*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = t + k * size;
            if (c >= cols) continue;
            float y = f[k] * r;
            if (a.w != nullptr) y *= elem_to_f32<TW>(static_cast<const W*>(a.w)[c]);
            if (a.b != nullptr) y += elem_to_f32<TW>(static_cast<const W*>(a.b)[c]);
            out[c] = elem_from_f32<T>(y);
        }
    }
}

// Its backward pass.  Dynamic shared memory: the groups' column sums, where a block has
// more than one group.
template <int T, int TW, int V>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_elements_grad(const NormGradRows a, int size) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    extern __shared__ float sums[];
    Group<false> g = group_of<false>(size, words);
    const int t = threadIdx.x % size, groups = blockDim.x / size;
    const int cols = static_cast<int>(a.cols);
    pdl_enter();
    const float inv = 1.0f / static_cast<float>(a.cols);
    float dw[V] = {}, db[V] = {};
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * groups) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        const S* d = static_cast<const S*>(a.d) + row * a.d_stride;
        const float mean = __ldg(a.mean + row), r = __ldg(a.rstd + row);
        float xh[V], f[V];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = t + k * size;
            if (c >= cols) continue;
            xh[k] = (elem_to_f32<T>(x[c]) - mean) * r;
            f[k] = elem_to_f32<T>(d[c]);
            dw[k] = fmaf(f[k], xh[k], dw[k]);
            db[k] += f[k];
            if (a.w != nullptr) f[k] *= elem_to_f32<TW>(static_cast<const W*>(a.w)[c]);
            s1 += f[k];
            s2 = fmaf(f[k], xh[k], s2);
        }
        if (a.d_x == nullptr) continue;
        const float2 m = g.sum(s1, s2);
        const float c1 = m.x * inv, c2 = m.y * inv;
        S* dx = static_cast<S*>(a.d_x) + row * a.d_x_stride;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (t + k * size < cols)
                dx[t + k * size] = elem_from_f32<T>(r * (f[k] - c1 - xh[k] * c2));
    }
    if (a.piece == nullptr) return;
    // the groups' sums, added in the groups' order
    float* piece = a.piece + static_cast<int64_t>(blockIdx.x) * 2 * a.pitch;
    for (int q = 0; q < groups; ++q) {
        if (q > 0) __syncthreads();
        if (g.id != q) continue;
        const bool last = q + 1 == groups;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = t + k * size;
            if (c >= cols) continue;
            if (q > 0) {
                dw[k] += sums[c];
                db[k] += sums[cols + c];
            }
            (last ? piece : sums)[c] = dw[k];
            (last ? piece + a.pitch : sums + cols)[c] = db[k];
        }
    }
}

// Backward with rows on their way through shared memory: each group of threads has
// `depth` slots of its own for rows of x and d, which its first thread fills by bulk
// copies as soon as all have done with a row, so that some 190 KB a SM are in flight
// whatever the threads do.  The row is read twice from shared memory, once for the
// sums and once for d_x: in registers it would leave room for half the threads.  After
// a wait that ran out a block goes on without waiting (its barriers need all threads),
// with the status word set.
constexpr int kStagedThreads = 512;
constexpr int kStagedBytes = 216 * 1024;
// Rows of 16 bits that end inside a vector take a few registers more.
constexpr int staged_threads(int type, bool tail) {
    return tail && type != kGradF32 ? 384 : kStagedThreads;
}
struct StagedShape {
    int size, groups, depth;
};
// WHOLE: d_x's rows take vectors; else consecutive threads write consecutive elements.
// WARPS: each warp is a group (sixteen of them: their sums one after another would take 4 of
// 16 us at 4096 rows of 768).
template <int T, int TW, int N, bool TAIL, bool WHOLE, bool WARPS>
__global__ void __launch_bounds__(staged_threads(T, TAIL), 1)
    layer_norm_staged_grad(const NormGradRows a, const StagedShape sh,
                           unsigned long long limit_ns) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    constexpr int V = 32 / N;
    extern __shared__ __align__(128) char slots[];
    __shared__ float2 words[2 * kNormThreads / 32];
    __shared__ uint64_t full[kStagedThreads / 32 * 4];     // up to four slots a group
    __shared__ float tails[TAIL ? 2 * N * kStagedThreads / 32 : 1];   // sums of the row's end
    const int size = WARPS ? 32 : sh.size;
    Group<false> g = group_of<false>(size, words);
    const int t = threadIdx.x % size;
    const int cols = static_cast<int>(a.cols) / N * N;           // in whole vectors
    const int wide = TAIL ? cols + N : cols;                     // of a slot
    // the elements after them: the first threads', one each
    const int tail = cols + t;
    const bool has = TAIL && tail < static_cast<int>(a.cols);
    const uint32_t row_bytes = wide * sizeof(S);
    // the weights in fp32, then the slots
    float* weights = reinterpret_cast<float*>(slots);
    char* mine = slots + (a.w != nullptr ? 4 * wide : 0) +
                 static_cast<size_t>(g.id) * sh.depth * 2 * row_bytes;
    uint64_t* bar = full + g.id * sh.depth;
    if (t == 0)
        for (int k = 0; k < sh.depth; ++k) mbar_init(bar + k, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_enter();
    if (a.w != nullptr)
        for (int c = threadIdx.x; c < wide; c += blockDim.x)
            weights[c] = c < a.cols ? elem_to_f32<TW>(static_cast<const W*>(a.w)[c]) : 0.0f;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * sh.groups + g.id;
    const int64_t next = static_cast<int64_t>(gridDim.x) * sh.groups;
    const int64_t rows = first < a.rows ? (a.rows - first + next - 1) / next : 0;
    const auto fetch = [&](int64_t j) {                          // the group's j-th row
        const int64_t row = first + j * next;
        const int slot = static_cast<int>(j % sh.depth);
        char* to = mine + slot * 2 * row_bytes;
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        const S* d = static_cast<const S*>(a.d) + row * a.d_stride;
        uint32_t bytes = row_bytes;
        if (TAIL && row + 1 == a.rows) {
            // what follows the last row may not be read: its end goes by itself
            bytes = cols * sizeof(S);
            for (int c = cols; c < a.cols; ++c) {
                reinterpret_cast<S*>(to)[c] = x[c];
                reinterpret_cast<S*>(to + row_bytes)[c] = d[c];
            }
        }
        mbar_expect_tx(bar + slot, 2 * bytes);
        if (TAIL && bytes == 0) return;
        bulk_load(to, x, bytes, bar + slot);
        bulk_load(to + row_bytes, d, bytes, bar + slot);
    };
    int64_t fetched = 0;
    if (t == 0)
        for (; fetched < sh.depth && fetched < rows; ++fetched) fetch(fetched);
    const float inv = 1.0f / static_cast<float>(a.cols);
    bool late = false;
    Pair dw[V][N / 2], db[V][N / 2];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) dw[k][i] = db[k][i] = make_pair(0.0f, 0.0f);
    if (has) tails[2 * (g.id * N + t)] = tails[2 * (g.id * N + t) + 1] = 0.0f;
    int slot = 0, phase = 0;
    float next_mean = rows > 0 ? __ldg(a.mean + first) : 0.0f;
    float next_r = rows > 0 ? __ldg(a.rstd + first) : 0.0f;
    for (int64_t j = 0; j < rows; ++j) {
        const int64_t row = first + j * next;
        const float mean = next_mean, r = next_r;
        if (j + 1 < rows) {
            next_mean = __ldg(a.mean + row + next);
            next_r = __ldg(a.rstd + row + next);
        }
        const Pair off = make_pair(-mean, -mean), r2 = make_pair(r, r);
        if (!late && !mbar_wait(bar + slot, phase, limit_ns)) {
            late = true;
            atomicOr(&g_norm_status, kStatusConsumerTimeout);
        }
        const S* x = reinterpret_cast<const S*>(mine + slot * 2 * row_bytes);
        const S* d = reinterpret_cast<const S*>(mine + slot * 2 * row_bytes + row_bytes);
        Pair s1 = make_pair(0.0f, 0.0f), s2 = s1;
        if (has) {
            const float xh = (elem_to_f32<T>(x[tail]) - mean) * r;
            float f = elem_to_f32<T>(d[tail]);
            float* own = tails + 2 * (g.id * N + t);
            own[0] = fmaf(f, xh, own[0]);
            own[1] += f;
            if (a.w != nullptr) f *= weights[tail];
            s1 = make_pair(f, 0.0f);
            s2 = make_pair(f * xh, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
            Raw<T, N> rx{*reinterpret_cast<const uint4*>(x + c)};
            Raw<T, N> rd{*reinterpret_cast<const uint4*>(d + c)};
            Pair w[N / 2];
            if (a.w != nullptr) load_weights<kGradF32, N>(weights, c, w);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const Pair xh = mul2(add2(rx.pair(i), off), r2);
                Pair f = rd.pair(i);
                dw[k][i] = fma2(f, xh, dw[k][i]);
                db[k][i] = add2(db[k][i], f);
                if (a.w != nullptr) f = mul2(f, w[i]);
                s1 = add2(s1, f);
                s2 = fma2(f, xh, s2);
            }
        }
        const float2 m = g.sum(floats(s1).x + floats(s1).y, floats(s2).x + floats(s2).y);
        // all threads are here: none reads the row before any more (a warp's shuffles alone
        // order no reads of shared memory before the next copy into it)
        if constexpr (WARPS) __syncwarp();
        if (t == 0 && !late && j > 0 && fetched < rows) fetch(fetched++);
        if (a.d_x != nullptr) {
            // r (f - c1 - xh c2) = r f + (x - mean) (-r r c2) - r c1
            const float c1 = -r * (m.x * inv), c2 = -r * (r * (m.y * inv));
            S* dx = static_cast<S*>(a.d_x) + row * a.d_x_stride;
            const auto element = [&](int c) {
                float y = elem_to_f32<T>(d[c]);
                if (a.w != nullptr) y *= weights[c];
                dx[c] = elem_from_f32<T>(fmaf(y, r, fmaf(elem_to_f32<T>(x[c]) - mean, c2, c1)));
            };
            if constexpr (WHOLE) {
                const Pair k1 = make_pair(c1, c1), k2 = make_pair(c2, c2);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int c = (t + k * size) * N;
                    if (c >= cols) continue;
                    Raw<T, N> rx{*reinterpret_cast<const uint4*>(x + c)};
                    Raw<T, N> rd{*reinterpret_cast<const uint4*>(d + c)};
                    Pair w[N / 2];
                    if (a.w != nullptr) load_weights<kGradF32, N>(weights, c, w);
                    float f[N];
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        Pair y = rd.pair(i);
                        if (a.w != nullptr) y = mul2(y, w[i]);
                        y = fma2(y, r2, fma2(add2(rx.pair(i), off), k2, k1));
                        f[2 * i] = floats(y).x;
                        f[2 * i + 1] = floats(y).y;
                    }
                    store_elems<T, N>(dx + c, f);
                }
                if (has) element(tail);
            } else {
#pragma unroll 4
                for (int c = t; c < static_cast<int>(a.cols); c += size) element(c);
            }
        }
        if (++slot == sh.depth) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (late && t == 0)      // copies in flight land before the block's memory goes
        for (int64_t j = fetched > sh.depth ? fetched - sh.depth : 0; j < fetched; ++j)
            if (!mbar_wait(bar + j % sh.depth, (j / sh.depth) & 1, kDrainNs))
                atomicOr(&g_norm_status, kStatusDrainTimeout);
    if (a.piece == nullptr) return;
    if constexpr (WARPS) {
        // the warps' sums to where their rows were (8 bytes a column: two slots of 16 bits
        // or one of fp32), then added in the warps' order
        __syncwarp();
        float* to = reinterpret_cast<float*>(mine);
        if (has) {
            to[tail] = tails[2 * (g.id * N + t)];
            to[wide + tail] = tails[2 * (g.id * N + t) + 1];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
            float fw[N], fb[N];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                fw[2 * i] = floats(dw[k][i]).x;
                fw[2 * i + 1] = floats(dw[k][i]).y;
                fb[2 * i] = floats(db[k][i]).x;
                fb[2 * i + 1] = floats(db[k][i]).y;
            }
            store_elems<kGradF32, N>(to + c, fw);
            store_elems<kGradF32, N>(to + wide + c, fb);
        }
        __syncthreads();
        const float* from = reinterpret_cast<const float*>(slots + (a.w != nullptr ? 4 * wide : 0));
        const int each = static_cast<int>(sh.depth * 2 * row_bytes / sizeof(float));
        for (int c = threadIdx.x; c < 2 * wide; c += blockDim.x) {
            const int col = c < wide ? c : c - wide;
            if (col >= static_cast<int>(a.cols)) continue;
            float sum = from[c];
#pragma unroll 4
            for (int q = 1; q < sh.groups; ++q) sum += from[q * each + c];
            a.piece[(2 * static_cast<int64_t>(blockIdx.x) + (c >= wide)) * a.pitch + col] = sum;
        }
        return;
    }
    // the groups' sums, added in the groups' order, where the rows were
    float* sums = reinterpret_cast<float*>(slots + (a.w != nullptr ? 4 * wide : 0));
    float* piece = a.piece + static_cast<int64_t>(blockIdx.x) * 2 * a.pitch;
    for (int q = 0; q < sh.groups; ++q) {
        __syncthreads();
        if (g.id != q) continue;
        const bool last = q + 1 == sh.groups;
        if (has) {
            float* to = (last ? piece : sums) + tail;
            to[0] = tails[2 * (g.id * N + t)] + (q > 0 ? sums[tail] : 0.0f);
            to[last ? a.pitch : wide] =
                tails[2 * (g.id * N + t) + 1] + (q > 0 ? sums[wide + tail] : 0.0f);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (t + k * size) * N;
            if (c >= cols) continue;
            float fw[N], fb[N];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                fw[2 * i] = floats(dw[k][i]).x;
                fw[2 * i + 1] = floats(dw[k][i]).y;
                fb[2 * i] = floats(db[k][i]).x;
                fb[2 * i + 1] = floats(db[k][i]).y;
            }
            if (q > 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    fw[i] += sums[c + i];
                    fb[i] += sums[wide + c + i];
                }
            }
            float* to = (last ? piece : sums) + c;
            store_elems<kGradF32, N>(to, fw);
            store_elems<kGradF32, N>(to + (last ? a.pitch : wide), fb);
        }
    }
}

// d_w and d_b from the blocks' sums: 32 columns per block, a warp takes every
// sixteenth of the pieces, the warps' sums are added in their order.
template <int TW>
__global__ void __launch_bounds__(512)
    layer_norm_columns(const float* piece, int pieces, int64_t cols, int64_t pitch, void* d_w,
                       void* d_b, int accumulate) {
    using W = typename Elem<TW>::Store;
    __shared__ float part[16][32];
    pdl_enter();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // of 2 * pitch
    const int64_t c = at < pitch ? at : at - pitch;
    const bool live = at < 2 * pitch && c < cols;
    float s = 0.0f;
    if (live) {
#pragma unroll
        for (int k = 0; k < kNormPieces / 16; ++k) {
            const int q = warp + 16 * k;
            if (q < pieces) s += piece[static_cast<int64_t>(q) * 2 * pitch + at];
        }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !live) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += part[k][lane];
    W* to = static_cast<W*>(at < pitch ? d_w : d_b);
    if (to == nullptr) return;
    to += c;
    if (accumulate) s += elem_to_f32<TW>(*to);
    *to = elem_from_f32<TW>(s);
}

// ------------------------------------------------------- rows of any width

template <int T, int TW>
__global__ void __launch_bounds__(kNormThreads) layer_norm_wide(const NormRows a) {
    using S = typename Elem<T>::Store;
    using W = typename Elem<TW>::Store;
    __shared__ float2 words[2 * kNormThreads / 32];
    Group<true> g = group_of<true>(kNormThreads, words);
    pdl_enter();
    const float n = static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const S* x = static_cast<const S*>(a.x) + row * a.x_stride;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) s += elem_to_f32<T>(x[c]);
        const float mean = __fdiv_rn(g.sum(s), n);   // no rounded 1 / n: rows far from 0
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
            const float y = elem_to_f32<T>(x[c]) - mean;
            q = fmaf(y, y, q);
        }
        const float var = __fdiv_rn(g.sum(q), n);
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
    Group<true> g = group_of<true>(kNormThreads, words);
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
    float* piece = a.piece + static_cast<int64_t>(blockIdx.y) * 2 * a.pitch;
    piece[c] = dw;
    piece[a.pitch + c] = db;
}

// ----------------------------------------------------------------- launches

// Whole warps that take one row, `held` elements to a thread; 0: too wide.  (As few as
// hold it, not a power of two of them: 8192 rows of 5120 bf16 take 38.8 us instead of
// 46.7, backward 59.4 instead of 69.1.)
int fit_group(int64_t cols, int most, int held) {
    const int64_t s = std::max<int64_t>(1, (cols + 32 * held - 1) / (32 * held)) * 32;
    return s <= most ? static_cast<int>(s) : 0;
}
// A thread holds up to 32 elements of a row in vectors (4 of 16 bits, 8 of fp32; what
// follows the last whole vector goes to the first threads besides), or 16 single ones
// where rows are not aligned; backward, with their columns' sums, 32 or 8.
int64_t in_vectors(int64_t cols, int type) {
    return type == kGradF32 ? cols / 4 * 4 : cols / 8 * 8;
}
int fit_rows(int64_t cols, int type, bool vec) {
    return vec ? fit_group(in_vectors(cols, type), kNormThreads, 32)
               : fit_group(cols, kNormThreads, 16);
}
int fit_grad(int64_t cols, int type, bool vec) {
    return vec ? fit_group(in_vectors(cols, type), 256, 32) : fit_group(cols, kNormThreads, 8);
}

// The groups of a block and their slots: as many groups as leave three slots each (or
// two, in rows of 32 KB and more).
StagedShape staged_shape(int64_t cols, int type, int threads) {
    StagedShape s{fit_grad(cols, type, true), 0, 0};
    const int64_t wide = (cols + 7) / 8 * 8;         // as much as the kernel takes, or more
    const int64_t slot = 2 * wide * (type == kGradF32 ? 4 : 2);     // a row of x and one of d
    const int64_t room = kStagedBytes - 4 * wide;    // beside the weights
    const int64_t most = std::max<int64_t>(1, room / (3 * slot));
    // where few rows fit, more threads to each; a group of several warps has one of 15
    // barriers
    s.size = static_cast<int>(std::max<int64_t>(s.size, threads / most / 32 * 32));
    s.groups = static_cast<int>(std::min<int64_t>(threads / s.size, most));
    if (s.size > 32 && s.groups > 15) s.groups = 15;
    s.depth = static_cast<int>(std::min<int64_t>(4, room / (s.groups * slot)));
    return s;
}
template <typename Kernel, typename Args>
cudaError_t go_staged(Kernel* kernel, const Args& a, const StagedShape& s, int blocks,
                      cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedBytes);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(blocks), dim3(s.groups * s.size), kStagedBytes, stream, a, s,
                        tma_wait_limit());
}
template <int T, int TW>
cudaError_t go_rows(const NormRows& a, bool vec, bool whole, cudaStream_t stream) {
    const int size = fit_rows(a.cols, T, vec);
    const int64_t most = static_cast<int64_t>(device_sms()) * 8;
    if (size == 0)
        return launch_after(layer_norm_wide<T, TW>,
                            dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                            dim3(kNormThreads), 0, stream, a);
    // rows of vectors: four warps with a row each, or a block to a row
    const int threads = size > 128 || (vec && size > 32) ? size : 128 / size * size;
    const int64_t blocks = (a.rows + threads / size - 1) / (threads / size);
    const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
    constexpr int N = Elem<T>::kVec;
    const auto go = [&](auto* kernel) {
        return launch_after(kernel, grid, dim3(threads), 0, stream, a, size);
    };
    if (!vec) return go(layer_norm_elements<T, TW, 16>);
    const auto vectors = [&](auto alone, auto tail) {
        constexpr bool A = decltype(alone)::value, E = decltype(tail)::value;
        return whole ? go(layer_norm_vectors<T, TW, A, E, true>)
                     : go(layer_norm_vectors<T, TW, A, E, false>);
    };
    if (a.cols % N == 0)
        return size > 32 ? vectors(Const<true>(), Const<false>())
                         : vectors(Const<false>(), Const<false>());
    return size > 32 ? vectors(Const<true>(), Const<true>()) : vectors(Const<false>(), Const<true>());
}

StagedShape grad_shape(int64_t cols, int type) {
    const int es = type == kGradF32 ? 4 : 2;
    return staged_shape(cols, type, staged_threads(type, cols * es % 16 != 0));
}
// Blocks of the backward pass, each of which leaves one row of column sums:
// at most kNormPieces.
int norm_pieces(int64_t rows, int64_t cols, int type, bool vec) {
    const int size = fit_grad(cols, type, vec);
    if (rows == 0) return 0;
    if (size == 0) return static_cast<int>(rows < 64 ? rows : 64);
    const int groups = vec ? grad_shape(cols, type).groups : kNormThreads / size;
    const int64_t most = std::min(device_sms(), kNormPieces);
    const int64_t need = (rows + groups - 1) / groups;
    return static_cast<int>(need < most ? need : most);
}

template <int T, int TW>
cudaError_t go_staged_grad(const NormGradRows& a, int blocks, bool whole, cudaStream_t stream) {
    constexpr int N = Elem<T>::kVec;
    const StagedShape s = grad_shape(a.cols, T);
    const auto go = [&](auto tail, auto warps) {
        constexpr bool E = decltype(tail)::value, P = decltype(warps)::value;
        return whole
                   ? go_staged(layer_norm_staged_grad<T, TW, N, E, true, P>, a, s, blocks, stream)
                   : go_staged(layer_norm_staged_grad<T, TW, N, E, false, P>, a, s, blocks, stream);
    };
    if (a.cols % N == 0)
        return s.size == 32 ? go(Const<false>(), Const<true>()) : go(Const<false>(), Const<false>());
    return s.size == 32 ? go(Const<true>(), Const<true>()) : go(Const<true>(), Const<false>());
}
template <int T, int TW>
cudaError_t go_elements_grad(const NormGradRows& a, int size, int blocks, cudaStream_t stream) {
    const size_t smem = kNormThreads >= 2 * size ? sizeof(float) * 2 * a.cols : 0;   // 16 KB at most
    return launch_after(layer_norm_elements_grad<T, TW, 8>, dim3(blocks),
                        dim3(kNormThreads / size * size), smem, stream, a, size);
}

template <int T, int TW>
cudaError_t go_grad(const NormGradRows& a, void* d_w, void* d_b, int accumulate, bool vec,
                    bool whole, cudaStream_t stream) {
    const int size = fit_grad(a.cols, T, vec);
    const int pieces = norm_pieces(a.rows, a.cols, T, vec);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && size != 0) {
        e = vec ? go_staged_grad<T, TW>(a, pieces, whole, stream)
                : go_elements_grad<T, TW>(a, size, pieces, stream);
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
    e = launch_after(layer_norm_columns<TW>, dim3(static_cast<unsigned>((2 * a.pitch + 31) / 32)),
                     dim3(512), 0, stream, static_cast<const float*>(a.piece), pieces, a.cols,
                     a.pitch, d_w, d_b, accumulate);
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

cudaError_t read_norm_status(unsigned int* status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_norm_status, sizeof(unsigned int));
    if (e != cudaSuccess || !clear) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_norm_status, &zero, sizeof(unsigned int));
}

const char* layer_norm_kernel(int64_t cols, int type, bool vec, bool whole) {
    if (fit_rows(cols, type, vec) == 0) return "layer_norm_wide";
    return !vec    ? "layer_norm_elements"
           : whole ? "layer_norm_vectors" : "layer_norm_vectors, turned";
}
const char* layer_norm_grad_kernel(const NormGradRows& a, int type, bool vec, bool whole) {
    if (a.rows == 0) return "layer_norm_columns";
    if (fit_grad(a.cols, type, vec) == 0)
        return a.d_x != nullptr ? "layer_norm_wide_grad" : "layer_norm_wide_columns";
    return !vec    ? "layer_norm_elements_grad"
           : whole ? "layer_norm_staged_grad" : "layer_norm_staged_grad, by elements";
}

cudaError_t launch_layer_norm(const NormRows& a, int type, int w_type, bool vec, bool whole,
                              cudaStream_t stream) {
    const cudaError_t e = by_types(type, w_type, [&](auto t, auto w) {
        return go_rows<decltype(t)::value, decltype(w)::value>(a, vec, whole, stream);
    });
    note_launch();
    return e;
}

cudaError_t launch_layer_norm_grad(const NormGradRows& a, int type, int w_type, void* d_w,
                                   void* d_b, int accumulate, bool vec, bool whole,
                                   cudaStream_t stream) {
    return by_types(type, w_type, [&](auto t, auto w) {
        return go_grad<decltype(t)::value, decltype(w)::value>(a, d_w, d_b, accumulate, vec,
                                                               whole, stream);
    });
}

}  // namespace shardstep
