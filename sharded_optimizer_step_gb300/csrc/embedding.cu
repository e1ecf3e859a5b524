// The token embedding and its gradient.
//
//   out[i]      = scale * table[ids[i]]
//   d_table[v] (+)= scale * sum over i with ids[i] == v of d_out[i]
//
// An id outside [0, vocab) reads nothing, gives a row of zeros and adds to no
// gradient, so padded batches need no mask.  Both passes are bound by memory:
// the lookup moves every row once each way, the gradient reads every row of
// d_out once and writes every row of d_table once (those that occur, twice over,
// when it adds).
//
// The gradient's sums must not depend on the order in which blocks run, and a
// few ids make up much of a text, so the tokens are sorted by id first (stable:
// equal ids keep the tokens' order) and the sorted list is cut into equal
// chunks, whatever the ids are:
//
//   embedding_sort   block b owns the ids [b r, (b + 1) r).  It scans all ids
//                    twice (8 bytes a token and block from L2; up to 32768
//                    tokens the second time from shared memory): once to
//                    count its own and those below its range, which gives it
//                    its place in the sorted list without any other block's
//                    answer, once to place them.
//   embedding_sum    a chunk of sorted tokens times a slice of columns per
//                    block; sums in fp32 in the tokens' order.  A run of equal
//                    ids within a chunk is written at once, pieces of runs that
//                    go on across chunks are kept.  Further blocks write the
//                    rows that do not occur.
//   embedding_join   adds the pieces of each such run in the chunks' order.
//
// Chunk lengths go by the sizes alone, so equal calls give equal bits.
//
// Measured: the lookup of 16384 rows of 4096 bf16 takes 30 us (268 MB; ids that occur
// again are read from L2).  The gradient of 16384 rows of 4096 bf16 over 32000 ids: the
// sort 12 us (8 for 4096 tokens; its latency: two passes over the ids, 32 warps a
// block, a block an SM), the sums 58 (396 MB at 6.8 TB/s, the rate of a plain copy), the
// join 6: what is over the bytes' time is the sort, in which memory is idle, and the join.
#include <atomic>

#include "elem.cuh"

namespace shardstep {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortHeld = 32768;   // tokens whose ids a block keeps after its first scan
constexpr int kSortBytes = sizeof(uint32_t) * kSortWarps * kEmbedSortRange +
                           sizeof(int16_t) * kSortHeld;     // of shared memory at most
constexpr int kIdsAhead = 4;       // loads of ids in flight per thread
constexpr int kRowsAhead = 8;      // rows of d_out in flight per thread
constexpr int kPiecesAhead = 16;   // of the pieces of a run
// Rows that take no vectors are zeroed by vectors from their first 16-byte boundary on if
// they are longer than this (32000 of 2047 fp32: the gradient takes 47 us instead of 79;
// 50257 of 769 bf16 45 instead of 41).
constexpr int kShortRow = 1024;

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
    return ids64 ? __ldg(static_cast<const long long*>(ids) + i)
                 : static_cast<int64_t>(__ldg(static_cast<const int*>(ids) + i));
}

// ----------------------------------------------------------------- lookup

template <int TYPE, int N, int TOKENS>
__global__ void __launch_bounds__(256) embedding_lookup(const EmbedArgs a) {
    using S = typename Elem<TYPE>::Store;
    pdl_enter();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * TOKENS;
    int64_t id[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
        id[t] = first + t < a.n ? load_id(a.ids, a.ids64, first + t) : -1;
    const S* table = static_cast<const S*>(a.table);
    S* out = static_cast<S*>(a.rows);
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * N; c < a.dim;
         c += static_cast<int64_t>(blockDim.x) * N) {
        float f[TOKENS][N];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            if (id[t] >= 0 && id[t] < a.vocab) {
                load_elems<TYPE, N>(table + id[t] * a.table_stride + c, f[t]);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) f[t][k] = 0.0f;
            }
        }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            const bool live = id[t] >= 0 && id[t] < a.vocab;   // 0 * inf is not 0
#pragma unroll
            for (int k = 0; k < N; ++k) f[t][k] = live ? f[t][k] * a.scale : 0.0f;
            if (first + t < a.n) store_elems<TYPE, N>(out + (first + t) * a.row_stride + c, f[t]);
        }
    }
}

// ------------------------------------------------------------------- sort

__global__ void __launch_bounds__(kSortThreads) embedding_sort(const EmbedArgs a,
                                                               const EmbedSort s) {
    extern __shared__ uint32_t counts[];   // [warp][id - lo], then each pair's next place
    __shared__ uint32_t below_sum, warp_sum[kSortWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * s.range;
    const int64_t left = a.vocab - lo;
    const int own = static_cast<int>(left < s.range ? left : s.range);
    for (int k = threadIdx.x; k < kSortWarps * s.range; k += kSortThreads) counts[k] = 0;
    if (threadIdx.x == 0) below_sum = 0;
    pdl_enter();
    __syncthreads();

    // each warp takes a run of consecutive tokens
    const int64_t per = (a.n + kSortThreads - 1) / kSortThreads * 32;
    const int64_t begin = warp * per < a.n ? warp * per : a.n;
    const int64_t end = begin + per < a.n ? begin + per : a.n;
    uint32_t* mine = counts + warp * s.range;
    // what a token is to this block: its place in the range, or -1
    int16_t* held = reinterpret_cast<int16_t*>(counts + kSortWarps * s.range);
    const bool hold = a.n <= kSortHeld;
    uint32_t below = 0;
    for (int64_t i = begin + lane; i < end; i += kIdsAhead * 32) {
        int64_t id[kIdsAhead];
#pragma unroll
        for (int k = 0; k < kIdsAhead; ++k)
            id[k] = i + 32 * k < end ? load_id(a.ids, a.ids64, i + 32 * k) : -1;
#pragma unroll
        for (int k = 0; k < kIdsAhead; ++k) {
            const bool in = id[k] >= lo && id[k] < lo + own;
            below += id[k] >= 0 && id[k] < lo;
            if (in) atomicAdd(mine + (id[k] - lo), 1u);
            if (hold && i + 32 * k < end)
                held[i + 32 * k] = static_cast<int16_t>(in ? id[k] - lo : -1);
        }
    }
    below = __reduce_add_sync(0xFFFFFFFFu, below);
    if (lane == 0 && below) atomicAdd(&below_sum, below);
    __syncthreads();

    // places: by id, then by warp; a thread takes `each` consecutive ids
    const int each = (s.range + kSortThreads - 1) / kSortThreads;
    const int k0 = threadIdx.x * each;
    uint32_t total = 0;
    for (int k = k0; k < k0 + each && k < own; ++k)
        for (int w = 0; w < kSortWarps; ++w) total += counts[w * s.range + k];
    uint32_t upto = total;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    uint32_t at = below_sum + upto - total;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int k = k0; k < k0 + each && k < own; ++k) {
        s.row_start[lo + k] = at;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = counts[w * s.range + k];
            counts[w * s.range + k] = at;
            at += c;
        }
    }
    if (lo + own == a.vocab && k0 < own && k0 + each >= own) s.row_start[a.vocab] = at;
    __syncthreads();

    const auto place_tokens = [&](int64_t i, int slot) {
        const uint32_t live = __ballot_sync(0xFFFFFFFFu, slot >= 0);
        if (live == 0) return;
        if (slot >= 0) {
            const uint32_t peers = __match_any_sync(live, slot);
            const uint32_t rank = __popc(peers & ((1u << lane) - 1));
            const uint32_t place = mine[slot] + rank;
            s.token[place] = static_cast<int32_t>(i);
            s.id[place] = static_cast<int32_t>(lo + slot);
            __syncwarp(live);
            if (rank == 0) mine[slot] += __popc(peers);
        }
        __syncwarp();
    };
    if (hold) {
        for (int64_t i = begin + lane; i - lane < end; i += 32)
            place_tokens(i, i < end ? held[i] : -1);
        return;
    }
    for (int64_t i = begin + lane; i - lane < end; i += kIdsAhead * 32) {
        int64_t id[kIdsAhead];
#pragma unroll
        for (int k = 0; k < kIdsAhead; ++k)
            id[k] = i + 32 * k < end ? load_id(a.ids, a.ids64, i + 32 * k) : -1;
#pragma unroll
        for (int k = 0; k < kIdsAhead; ++k)
            place_tokens(i + 32 * k, id[k] >= lo && id[k] < lo + own
                                         ? static_cast<int>(id[k] - lo) : -1);
    }
}

// -------------------------------------------------------------------- sum

// Row v of the gradient from its sum.
template <int TOUT, int N>
__device__ __forceinline__ void finish_row(const EmbedArgs& a, int64_t v, int64_t c, float* sum) {
    using S = typename Elem<TOUT>::Store;
    S* p = static_cast<S*>(a.table) + v * a.table_stride + c;
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] *= a.scale;
    if (a.accumulate) {
        float old[N];
        load_elems<TOUT, N>(p, old);
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] += old[k];
    }
    store_elems<TOUT, N>(p, sum);
}
template <int N>
__device__ __forceinline__ void keep_piece(float* p, const float* sum) {
    if constexpr (N == 1) {
        *p = sum[0];
    } else {
#pragma unroll
        for (int k = 0; k < N / 4; ++k)
            reinterpret_cast<uint4*>(p)[k] = pack4f(sum + 4 * k);
    }
}

template <int T, int N>
struct RawElems {          // as they are in memory: a vector, or one element
    using Type = uint4;
};
template <int T>
struct RawElems<T, 1> {
    using Type = typename Elem<T>::Store;
};

template <int TIN, int TOUT, int N>
__global__ void __launch_bounds__(256) embedding_sum(const EmbedArgs a, const EmbedSort s) {
    using S = typename Elem<TIN>::Store;
    using Raw = typename RawElems<TIN, N>::Type;
    __shared__ int32_t token[kEmbedChunkMax], id[kEmbedChunkMax];
    __shared__ uint32_t start[kEmbedZeroRows + 1];
    __shared__ int32_t before, after;
    pdl_enter();
    // units of sums and of zeros in turn, so that loads and stores mix
    const int64_t units = static_cast<int64_t>(s.chunks) * s.slices;
    const int64_t zeros = gridDim.x - units, both = units < zeros ? units : zeros;
    const int64_t b = blockIdx.x;
    const bool zero_rows = b < 2 * both ? b % 2 : units < zeros;
    const int64_t unit = b < 2 * both ? b / 2 : b - both;
    if (zero_rows) {   // rows that do not occur
        const int64_t v0 = unit * kEmbedZeroRows;
        const int count = static_cast<int>(a.vocab - v0 < kEmbedZeroRows ? a.vocab - v0
                                                                         : kEmbedZeroRows);
        if (threadIdx.x <= count) start[threadIdx.x] = s.row_start[v0 + threadIdx.x];
        __syncthreads();
        const float zero[N] = {};
        for (int v = 0; v < count; ++v) {
            if (start[v] != start[v + 1]) continue;
            typename Elem<TOUT>::Store* row =
                static_cast<typename Elem<TOUT>::Store*>(a.table) + (v0 + v) * a.table_stride;
            if (N > 1 || a.dim <= kShortRow) {
                for (int64_t c = static_cast<int64_t>(threadIdx.x) * N; c < a.dim;
                     c += static_cast<int64_t>(blockDim.x) * N)
                    store_elems<TOUT, N>(row + c, zero);
            } else {       // vectors from the row's first 16-byte boundary on
                constexpr int V = Elem<TOUT>::kVec;
                const int64_t skew = reinterpret_cast<uintptr_t>(row) / (16 / V) % V;
                const int64_t head = skew == 0 ? 0 : a.dim < V - skew ? a.dim : V - skew;
                const int64_t last = head + (a.dim - head) / V * V;
                for (int64_t c = head + static_cast<int64_t>(threadIdx.x) * V; c < last;
                     c += static_cast<int64_t>(blockDim.x) * V)
                    *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
                if (threadIdx.x < head) store_elems<TOUT, 1>(row + threadIdx.x, zero);
                if (last + threadIdx.x < a.dim) store_elems<TOUT, 1>(row + last + threadIdx.x, zero);
            }
        }
        return;
    }
    const int64_t chunk = unit / s.slices;
    const uint32_t live = s.row_start[a.vocab];   // tokens in the list
    const int64_t first = chunk * s.chunk;
    if (first >= live) return;
    const int count = static_cast<int>(live - first < s.chunk ? live - first : s.chunk);
    for (int k = threadIdx.x; k < count; k += blockDim.x) {
        token[k] = s.token[first + k];
        id[k] = s.id[first + k];
    }
    if (threadIdx.x == 0) {
        before = first > 0 ? s.id[first - 1] : -1;
        after = first + count < live ? s.id[first + count] : -1;
    }
    __syncthreads();
    const int64_t c = (unit % s.slices * static_cast<int64_t>(blockDim.x) + threadIdx.x) * N;
    if (c >= a.dim) return;
    const S* rows = static_cast<const S*>(a.rows) + c;
    float* piece = s.piece + 2 * chunk * a.dim + c;
    float sum[N] = {};
    for (int j0 = 0; j0 < count; j0 += kRowsAhead) {
        Raw raw[kRowsAhead];
#pragma unroll
        for (int j = 0; j < kRowsAhead; ++j)
            if (j0 + j < count)
                raw[j] = __ldcs(reinterpret_cast<const Raw*>(rows + token[j0 + j] * a.row_stride));
#pragma unroll
        for (int j = 0; j < kRowsAhead; ++j) {
            if (j0 + j >= count) continue;
            const int at = j0 + j, v = id[at];
            float f[N];
            if constexpr (N == 1) f[0] = elem_to_f32<TIN>(raw[j]);
            else unpack16<TIN>(raw[j], f);
#pragma unroll
            for (int k = 0; k < N; ++k) sum[k] += f[k];
            if (at + 1 < count && id[at + 1] == v) continue;
            // the run ends here: with what came before, alone, or to be continued
            if (v == before) keep_piece<N>(piece, sum);
            else if (at + 1 == count && v == after) keep_piece<N>(piece + a.dim, sum);
            else finish_row<TOUT, N>(a, v, c, sum);
#pragma unroll
            for (int k = 0; k < N; ++k) sum[k] = 0.0f;
        }
    }
}

// The runs that begin in a chunk and go on after it: its second piece, then the
// first pieces of the chunks up to the run's end.
template <int TOUT, int N>
__global__ void __launch_bounds__(256) embedding_join(const EmbedArgs a, const EmbedSort s) {
    pdl_enter();
    const int64_t chunk = blockIdx.x;
    const uint32_t live = s.row_start[a.vocab];
    const int64_t next = (chunk + 1) * s.chunk;
    if (next >= live) return;
    const int32_t v = s.id[next - 1];
    if (s.id[next] != v) return;
    if (s.row_start[v] < chunk * s.chunk) return;      // began before this chunk
    const int64_t c = (blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x) * N;
    if (c >= a.dim) return;
    const int64_t last = (s.row_start[v + 1] - 1) / s.chunk;
    const float* p = s.piece + c;
    float sum[N];
    load_elems<kGradF32, N>(p + (2 * chunk + 1) * a.dim, sum);
    for (int64_t q = chunk + 1; q <= last; q += kPiecesAhead) {
        float f[kPiecesAhead][N];
#pragma unroll
        for (int j = 0; j < kPiecesAhead; ++j)
            if (q + j <= last) load_elems<kGradF32, N>(p + 2 * (q + j) * a.dim, f[j]);
#pragma unroll
        for (int j = 0; j < kPiecesAhead; ++j) {
            if (q + j > last) continue;
#pragma unroll
            for (int k = 0; k < N; ++k) sum[k] += f[j][k];
        }
    }
    finish_row<TOUT, N>(a, v, c, sum);
}

int threads_for(int64_t vectors) {
    return vectors >= 256 ? 256 : static_cast<int>((vectors + 31) / 32 * 32);
}

template <int TYPE, int N>
cudaError_t go_lookup(const EmbedArgs& a, cudaStream_t stream) {
    const dim3 block(threads_for((a.dim + N - 1) / N));
    // one token per block until every SM has some
    if (a.n <= 4 * static_cast<int64_t>(device_sms()))
        return launch_after(embedding_lookup<TYPE, N, 1>, dim3(static_cast<unsigned>(a.n)), block,
                            0, stream, a);
    return launch_after(embedding_lookup<TYPE, N, 4>, dim3(static_cast<unsigned>((a.n + 3) / 4)),
                        block, 0, stream, a);
}

template <int TIN, int TOUT, int N>
cudaError_t go_sum(const EmbedArgs& a, EmbedSort s, cudaStream_t stream) {
    const dim3 block(threads_for(a.dim / N));
    s.slices = (a.dim / N + block.x - 1) / block.x;
    const int64_t zero =
        a.accumulate ? 0 : (a.vocab + kEmbedZeroRows - 1) / kEmbedZeroRows;
    const int64_t blocks = static_cast<int64_t>(s.chunks) * s.slices + zero;
    cudaError_t e = launch_after(embedding_sum<TIN, TOUT, N>, dim3(static_cast<unsigned>(blocks)),
                                 block, 0, stream, a, s);
    note_launch();
    if (e != cudaSuccess || s.chunks <= 1) return e;   // no run goes on
    // pieces are fp32: four columns a thread
    constexpr int J = N == 1 ? 1 : 4;
    const dim3 threads(threads_for(a.dim / J));
    const int64_t slices = (a.dim / J + threads.x - 1) / threads.x;
    e = launch_after(embedding_join<TOUT, J>,
                     dim3(static_cast<unsigned>(s.chunks - 1), static_cast<unsigned>(slices)),
                     threads, 0, stream, a, s);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_embedding(const EmbedArgs& a, int type, bool vec, cudaStream_t stream) {
    const cudaError_t e = by_type(type, [&](auto t) {
        constexpr int T = decltype(t)::value;
        return vec ? go_lookup<T, Elem<T>::kVec>(a, stream) : go_lookup<T, 1>(a, stream);
    });
    note_launch();
    return e;
}

// A chunk is long enough for some eight blocks per SM of 152, so that few runs are
// cut; it goes by the sizes alone.
EmbedPlan embed_plan(int64_t n, int64_t dim) {
    const int64_t wide = (dim + 2047) / 2048;
    const int64_t t = (n * wide / 1216 + 7) / 8 * 8;
    EmbedPlan p;
    p.chunk = static_cast<int>(t < 8 ? 8 : t > kEmbedChunkMax ? kEmbedChunkMax : t);
    p.chunks = (n + p.chunk - 1) / p.chunk;
    return p;
}

// Raises the sort's limit of shared memory to the most that any call takes, once per
// device: a limit of this call's own would hold for a call of another thread too, and
// the kernel's own words count towards the 48 KB that need none.
static cudaError_t allow_sort() {
    static std::atomic<int> done[256];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 256;
    if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(embedding_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortBytes);
    if (e == cudaSuccess && known) done[dev].store(1, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_embedding_grad(const EmbedArgs& a, EmbedSort s, int in_type, int out_type,
                                  bool vec, cudaStream_t stream) {
    const int sms = device_sms();
    const int64_t fair = (a.vocab + sms - 1) / sms;
    s.range = static_cast<int>(fair < kEmbedSortRange ? fair : kEmbedSortRange);
    const size_t smem = sizeof(uint32_t) * kSortWarps * s.range +
                        (a.n <= kSortHeld ? sizeof(int16_t) * a.n : 0);
    cudaError_t e = allow_sort();
    if (e != cudaSuccess) return e;
    e = launch_after(embedding_sort, dim3(static_cast<unsigned>((a.vocab + s.range - 1) / s.range)),
                     dim3(kSortThreads), smem, stream, a, s);
    note_launch();
    if (e != cudaSuccess) return e;
    return by_type(in_type, [&](auto ti) {
        return by_type(out_type, [&](auto to) {
            constexpr int I = decltype(ti)::value, O = decltype(to)::value;
            // a vector is 16 bytes of d_out; a gradient of fp32 takes two stores for it
            return vec ? go_sum<I, O, Elem<I>::kVec>(a, s, stream) : go_sum<I, O, 1>(a, s, stream);
        });
    });
}

}  // namespace shardstep
