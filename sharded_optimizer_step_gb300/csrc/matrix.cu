// Orthogonalised updates of matrices: the Newton-Schulz quintic iteration
//
//   X = u / (|u| + eps)            (transposed where u is taller than wide)
//   A = X X^T,  X = (a + b A + c A A) X             `rounds` times
//
// over a list of matrices, as such or as an optimizer's step: the momentum and the
// norms (matrix_moments), X's image (matrix_image), and all products of all rounds in
// one launch (matrix_rounds), the last of which steps the weights.
//
// Products.  A round forms A, then P = a + A C with C = b + c A written beside A, then
// P X; no result needs another image than its own operands (a result warp's loads
// would stand at the end of every step: they took 6 of its 12 us).  Everything but X
// is symmetric: its products compute the tiles on and above the diagonal, and where an
// operand lies below it, the tile from above is read the other way round.  Rounds of
// long matrices go two at a time without forming X between them (plan_steps in
// model_api.cpp).
//
// The tensor cores multiply halves; to keep single precision each value v is held as
// two, hi = half(s v) and lo = half(s v - hi) with s a power of two: 22 bits, of which
// three products hi hi + hi lo + lo hi make a product good to about 2^-21.  One product
// of single halves loses 2e-3 to 2e-2 of the result's norm over five rounds, these three
// 1e-6 to 1e-5 (8e-5 where u is one direction), 0.2 to 2.6 times what 32-bit products do.
// s is 2^15 for X and A, whose elements stay below sqrt(2) and 2, 2^13 for C, below 8, 2^14
// for P, below 4, and 2^12 for the product of two of them (the host checks the coefficients
// for it): nothing overflows, and an element of rms 1 / sqrt(m n), the smallest that occurs
// throughout (|a| is 1 or more), has its 22 bits up to m n = 2^30.
//
// What bounds it: three products of halves each, 1718 TFLOP/s of them sustained, so 573
// of the results' own; the operands: an SM takes in 64 bytes a clock, a 128 x 128
// tile's 64 KB in 0.49 us, and a pair's ring of three such stages turns one over in 2.4 us;
// and the sums: 64 of k take a 128 x 64 tile 0.61 us, a 128 x 128 one 0.76 (the products
// 0.45), a pair's 256 x 256 one 1.08 to 1.27.  Eight matrices of 2048 x 2048 run at 477
// (2.88 ms), 14 of a Llama-1B layer pair at 524 counted round by round (9.0 ms: rounds in
// twos do less).  A few small matrices are bound by their chain of 15 to 17 steps, 3 to 5 us
// each beside the products: 0.75 for the first operands, 0.3 to read the sums, 1 to 2 to turn
// them into halves, 0.5 for the stores to be seen, 1.5 until another SM knows (256 x 256:
// 92 to 98 us).
//
// Layout.  All operands live in the workspace as the images of what shared memory
// holds: blocks of 128 rows x 64 columns, 16 KB of hi then 16 KB of lo, rows of 128
// bytes in the tensor cores' 128-byte swizzle.  A tile's operands are then whole
// contiguous pieces, copied by bulk copies without a tensor map, and one block serves
// both as rows of k and as k rows.  Both sides are padded to the tile with zeros, which
// the products keep zero in X.
#include <atomic>

#include "elem.cuh"
#include "tcgen05.cuh"

namespace shardstep {
namespace {

__device__ unsigned int g_matrix_status;

constexpr int kBlockBytes = 32768;            // 128 x 64 halves, hi and lo
constexpr int kRingBytes = 196608;            // of the stages
constexpr int kMostStages = 4;
constexpr int kMostAccs = 4;
// Results on their way out: each result warp's 32 rows x 32 columns of hi or lo.
constexpr int kOutPiece = 2048;
// The tensor cores cut a sum's terms off at its last bits instead of rounding it, so a
// long sum falls short with every product that is added to it.  A sum over k therefore
// goes in pieces of 64, a stage each, which the result warps add up in their registers
// (rounding to nearest), and within a piece the small products, hi lo and lo hi, go
// first: four additions at its full size.  (256 k to a piece, products in turn: errors 3
// to 10 times those of 32-bit products, with 128 up to twice.)

// A tile of results: 128 x 128 by one block, 128 x 64 where tiles are few (a step's
// time is then its last tile's), or 256 x 256 by a pair of blocks, which copies half as
// much for a product.  Each block has 128 rows of it, and for each quarter of them two
// or four result warps with 128 or 32 columns each.  (256 x 128 by a pair was slower
// than 128 x 128 by one block at every size: a stage is too short for the pair's
// signals.)
template <int ROWS, int COLS>
struct Shape {
    static constexpr int kRows = ROWS, kCols = COLS;
    static constexpr int kBlocks = ROWS / 128;
    static constexpr bool kPair = kBlocks == 2;
    static constexpr int kColumns = COLS == 256 ? 128 : 32;     // of a result warp
    static constexpr int kResultWarps = 4 * COLS / kColumns;
    static constexpr int kThreads = 64 + 32 * kResultWarps;
    static constexpr int kAccs = COLS == 256 ? 2 : 4;           // accumulators
    static constexpr int kTmemColumns = kAccs * COLS;
    static constexpr int kArrivals = kBlocks * kResultWarps;    // per tile
    // a stage: 128 rows and this block's columns, 64 k of each, hi and lo
    static constexpr int kRightRows = COLS / kBlocks;
    static constexpr int kRightHalf = kRightRows * 128;         // bytes of hi, and of lo
    static constexpr int kStageBytes = kBlockBytes + 2 * kRightHalf;
    static constexpr int kStages = kRingBytes / kStageBytes;
    // stages from a multiple of 1024 on, then the pieces on their way out
    static constexpr int kDynamicBytes = kRingBytes + kResultWarps * kOutPiece + 1024;
    static_assert(kStages <= kMostStages && kStageBytes % 1024 == 0, "the ring");
};

struct Tile {
    int matrix, step;
    int row, col;            // of the result, in elements
    int k;                   // length of the sum
    uint32_t before;         // tiles of the matrix that have to be done
};
// What a result warp goes by, in shared memory: its registers hold sums.
struct Work {
    Tile tile;
    uint32_t index, step, end;   // of the tile, to the next one, of all
    uint32_t lanes, out;     // its tensor memory, and its piece of shared memory
    int down, across;        // its part of the tile
};

struct Shared {
    uint64_t full[kMostStages], empty[kMostStages];
    uint64_t peer[kMostStages];               // the other block's stage is full
    uint64_t done[kMostAccs], taken[kMostAccs];   // an accumulator is complete / has been read
    uint64_t drain;
    uint32_t tmem;
    Work work[16];                            // of each result warp
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

// Tile `index` of the call: step by step, matrix by matrix.
template <class F>
__device__ __forceinline__ Tile tile_at(const MatrixTable& t, const MatrixCall& call,
                                        uint32_t index) {
    Tile out;
    int lo = 0, hi = call.steps - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (call.step[mid].first <= index) lo = mid;
        else hi = mid - 1;
    }
    out.step = lo;
    const MatrixStep& step = call.step[lo];
    index -= step.first;
    const bool sym = step.flags & kSymmetric;
    const uint32_t* first = sym ? t.sym0 : t.full0;
    out.matrix = find(first, t.count, index);
    const MatrixItem& x = t.item[out.matrix];
    int i = static_cast<int>(index - first[out.matrix]);
    const int side = x.mp / F::kRows, all = x.np / F::kCols;
    constexpr int per = F::kRows / F::kCols;     // tiles on the diagonal of each row of them
    if (sym) {
        int r = 0;
        while (i >= (side - r) * per) i -= (side - r++) * per;
        out.row = r * F::kRows;
        out.col = r * F::kRows + i * F::kCols;
    } else {          // the rows of a column first: they share X's columns
        out.row = i % side * F::kRows;
        out.col = i / side * F::kCols;
    }
    out.k = step.flags & kLeftX ? x.np : x.mp;
    out.before = step.sym_before * (per * side * (side + 1) / 2) + step.full_before * (side * all);
    return out;
}

// Which operands' 64 k from k on come from blocks that hold k along their rows: X
// behind a symmetric matrix, and of a symmetric matrix what lies below the diagonal.
struct Turned {
    bool left, right;
};
template <class F>
__device__ __forceinline__ Turned turned_at(const Tile& at, int flags, int k) {
    const bool x = flags & kLeftX;
    return Turned{!x && k / F::kRows < at.row / F::kRows,
                  (flags & kRightX) || (!x && k / F::kRows < at.col / F::kRows)};
}
// Where 64 k of a row of results lie: in a block's rows, or, turned, in 64 of its rows.
__device__ __forceinline__ const char* operand_at(const void* image, int row, int k, int width,
                                                  bool turned) {
    return turned ? block_at(image, k, row, width) + k % 128 * 128
                  : block_at(image, row, k, width) + row % 128 * 128;
}
// 64 k of 128 or 64 rows, hi then lo: a block (its half of each part), or, turned, 64
// rows of k of one block for each 64 rows.
template <int ROWS>
__device__ __forceinline__ void copy_rows(char* to, const char* from, bool turned,
                                          uint64_t* bar) {
    if (!turned) {
        if constexpr (ROWS == 128) {
            bulk_load(to, from, kBlockBytes, bar);
        } else {
            bulk_load(to, from, 8192, bar);
            bulk_load(to + 8192, from + kBlockBytes / 2, 8192, bar);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < ROWS / 32; ++j)          // hi of all, then lo of all
        bulk_load(to + j * 8192,
                  from + j % (ROWS / 64) * kBlockBytes + j / (ROWS / 64) * (kBlockBytes / 2), 8192,
                  bar);
}

// Waits until `count` warps' parts of a matrix's tiles are written.
__device__ __forceinline__ bool tiles_wait(const unsigned int* counter, uint32_t count,
                                           unsigned long long limit_ns) {
    unsigned long long t0 = 0;
    for (uint32_t k = 0;; ++k) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
        if (v >= count) return true;
        if (k == 0) t0 = now_ns();
        else if (now_ns() - t0 > limit_ns) return false;
    }
}

// ------------------------------------------------------------------ results

// 32 columns of this lane's row, in place: each eight sums become, times scale and
// with `diagonal` added to column `on`, four words of halves hi and four of lo; and
// those become the same of what they stand for.
__device__ __forceinline__ void split_sums(uint32_t* w, float scale, float diagonal, int on) {
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = __uint_as_float(w[k + j]) * scale;
            if (on == k + j) f[j] += diagonal;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) split_pair(f[2 * j], f[2 * j + 1], &w[k + j], &w[k + 4 + j]);
    }
}
__device__ __forceinline__ void split_again(uint32_t* w, float scale, float diagonal, int on) {
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&w[k + j]));
            const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&w[k + 4 + j]));
            float a = (hi.x + lo.x) * scale, b = (hi.y + lo.y) * scale;
            if (on == k + 2 * j) a += diagonal;
            if (on == k + 2 * j + 1) b += diagonal;
            split_pair(a, b, &w[k + j], &w[k + 4 + j]);
        }
    }
}

// Those words to an image's block, `first` 16-byte pieces into its rows.  Through
// shared memory, so that four lanes write 64 bytes of one row (each lane its own row
// would be 32 lines an instruction, 4 us a step).
__device__ __forceinline__ void store_words(char* block, int first, const uint32_t* w,
                                            uint32_t piece) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int q = 0; q < 2; ++q) {                        // hi, lo
        __syncwarp();                                    // what was there has left
#pragma unroll
        for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             piece + lane * 64 + (c ^ lane / 2 % 4) * 16),
                         "r"(w[8 * c + 4 * q]), "r"(w[8 * c + 4 * q + 1]),
                         "r"(w[8 * c + 4 * q + 2]), "r"(w[8 * c + 4 * q + 3])
                         : "memory");
        __syncwarp();
        char* to = block + q * (kBlockBytes / 2) + lane / 4 * 128 +
                   ((first + lane % 4) ^ lane / 4) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {                    // rows 8 i + lane / 4
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(piece + (i * 8 + lane / 4) * 64 +
                               (lane % 4 ^ lane / 8 % 4) * 16)
                         : "memory");
            *reinterpret_cast<uint4*>(to + i * 1024) = v;
        }
    }
}

// Eight columns of the last round's results: an output, or the step of the weights.
__device__ __forceinline__ void finish(const MatrixItem& x, const MatrixCall& c, int row, int col,
                                       const uint32_t* sum, float scale) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(sum[k]) * scale;
    if (row >= x.m || col >= x.n) return;
    const float decay = c.group[x.group].lr_wd;
    if (!x.tall && x.whole) {        // rows of whole vectors
        const int64_t at = static_cast<int64_t>(row) * x.n + col;
        if (x.master != nullptr) {
            float p[8];
            load_elems<kGradF32, 8>(x.master + at, p);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                p[k] -= decay * p[k];
                v[k] = p[k] - x.step * v[k];
            }
            store_elems<kGradF32, 8>(x.master + at, v);
            if (x.out == nullptr) return;
        }
        if (c.out_type == kGradF32)
            store_elems<kGradF32, 8>(static_cast<float*>(x.out) + at, v);
        else if (c.out_type == kGradF16)
            store_elems<kGradF16, 8>(static_cast<uint16_t*>(x.out) + at, v);
        else
            store_elems<kGradBF16, 8>(static_cast<uint16_t*>(x.out) + at, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (col + k >= x.n) continue;
        const int64_t at = x.tall ? static_cast<int64_t>(col + k) * x.m + row
                                  : static_cast<int64_t>(row) * x.n + col + k;
        float r = v[k];
        if (x.master != nullptr) {
            float p = x.master[at];
            p -= decay * p;
            r = p - x.step * r;
            x.master[at] = r;
            if (x.out == nullptr) continue;
        }
        if (c.out_type == kGradF32) static_cast<float*>(x.out)[at] = r;
        else if (c.out_type == kGradF16)
            static_cast<uint16_t*>(x.out)[at] = elem_from_f32<kGradF16>(r);
        else static_cast<uint16_t*>(x.out)[at] = f32_to_bf16(r);
    }
}

// ----------------------------------------------------------------- products

// All rounds in one launch: every SM's block (or pair of blocks) walks the tiles of
// all steps in one fixed order.  A tile waits until its matrix has all tiles of the
// step before, so matrices follow each other through the steps without a barrier
// between them, and no step's last wave leaves SMs idle while another matrix has
// work.  (The launch is cooperative: all blocks are resident, and a tile waits for
// earlier ones only.)
//
// Warp 0 copies operands into a ring of stages, warp 1 issues each stage's products into
// one of a few accumulators, the others add those up and turn the sums into results.  In a
// pair, each block copies its half of both operands; the first block's warp 1 issues the
// products of both, and the second's passes on that its stages are full.  Every wait has a
// limit: past it the block sets the status word, lets its copies and products in flight
// end, frees its tensor memory and returns.
template <class F>
__global__ void __launch_bounds__(F::kThreads, 1)
    matrix_rounds(const __grid_constant__ MatrixTable t, const __grid_constant__ MatrixCall call,
                  unsigned long long limit_ns) {
    constexpr bool kPair = F::kPair;
    constexpr int kStages = F::kStages;
    extern __shared__ char raw[];
    __shared__ Shared sh;
    char* ring =
        reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = kPair ? pair_rank() : 0;
    const uint32_t unit = blockIdx.x / F::kBlocks, units = gridDim.x / F::kBlocks;
    const uint32_t tiles = call.tiles;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
            mbar_init(&sh.peer[s], 1);
        }
        for (int k = 0; k < F::kAccs; ++k) {
            mbar_init(&sh.done[k], 1);
            mbar_init(&sh.taken[k], F::kResultWarps * F::kBlocks);
        }
        mbar_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<kPair, F::kTmemColumns>(&sh.tmem);
    tmem_fence_before();
    if constexpr (kPair) pair_sync();
    else __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    const bool skip = skip_step(call.skip);

    if (!skip && warp == 0) {
        if (lane == 0) {
            uint32_t issued = 0;
            bool ok = true;
            for (uint32_t i = unit; ok && i < tiles; i += units) {
                const Tile at = tile_at<F>(t, call, i);
                const MatrixItem& x = t.item[at.matrix];
                if (at.before > 0)
                    ok = tiles_wait(x.tiles_done, at.before * F::kArrivals, limit_ns);
                if (!ok) break;
                asm volatile("fence.proxy.async.global;" ::: "memory");
                const MatrixStep& step = call.step[at.step];
                const void* left = x.image[step.left];
                const void* right = x.image[step.right];
                const int row = at.row + 128 * rank, col = at.col + F::kRightRows * rank;
                for (int k = 0; k < at.k; k += 64, ++issued) {
                    const uint32_t s = issued % kStages;
                    const Turned turned = turned_at<F>(at, step.flags, k);
                    const char* from_left = operand_at(left, row, k, at.k, turned.left);
                    const char* from_right = operand_at(
                        right, col, k, step.flags & kRightX ? x.np : at.k, turned.right);
                    // formed before the wait, not after it
                    asm volatile("" : "+l"(from_left), "+l"(from_right));
                    if (issued >= kStages &&
                        !mbar_wait(&sh.empty[s], (issued / kStages - 1) & 1, limit_ns)) {
                        ok = false;
                        break;
                    }
                    char* to = ring + s * F::kStageBytes;
                    mbar_expect_tx(&sh.full[s], F::kStageBytes);
                    copy_rows<128>(to, from_left, turned.left, &sh.full[s]);
                    copy_rows<F::kRightRows>(to + kBlockBytes, from_right, turned.right,
                                             &sh.full[s]);
                }
            }
            if (!ok) atomicOr(&g_matrix_status, kStatusProducerTimeout);
            // the last copies of every stage land before the block's memory goes
            for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                if (!mbar_wait(&sh.full[j % kStages], (j / kStages) & 1, kDrainNs))
                    atomicOr(&g_matrix_status, kStatusDrainTimeout);
        }
    } else if (!skip && warp == 1 && rank == 0) {
        // the warp stays together and one lane issues: what the products take is then in
        // uniform registers (moved there from one lane's, 12 products took it 690 clocks)
        const bool one = elect_one();
        uint32_t n = 0;                                   // stages, which are pieces
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity, bool far) {
            return __all_sync(0xFFFFFFFFu, far ? mbar_wait_pair(bar, parity, limit_ns)
                                               : mbar_wait(bar, parity, limit_ns)) != 0;
        };
        for (uint32_t i = unit; ok && i < tiles; i += units) {
            const Tile at = tile_at<F>(t, call, i);
            const int flags = call.step[at.step].flags;
            for (int k = 0; k < at.k; k += 64, ++n) {
                const uint32_t s = n % kStages;
                const uint32_t d = tmem + n % F::kAccs * F::kCols;
                const uint32_t a = smem_addr(ring + s * F::kStageBytes);
                const uint32_t b = a + kBlockBytes;
                const Turned turned = turned_at<F>(at, flags, k);
                const uint32_t form = half_product(F::kRows, F::kCols, turned.left, turned.right);
                // 16 k are 32 bytes along the rows, or 16 rows of 128 bytes
                const uint32_t ah = turned.left ? mn_major(a, 8192) : k_major(a);
                const uint32_t bh = turned.right ? mn_major(b, 8192) : k_major(b);
                const uint32_t next_a = turned.left ? 2048 / 16 : 32 / 16;
                const uint32_t next_b = turned.right ? 2048 / 16 : 32 / 16;
                const uint32_t al = ah + kBlockBytes / 2 / 16, bl = bh + F::kRightHalf / 16;
                if (n >= F::kAccs)
                    ok = wait(&sh.taken[n % F::kAccs], (n / F::kAccs - 1) & 1, kPair);
                if (ok) ok = wait(&sh.full[s], (n / kStages) & 1, false);
                if (kPair && ok) ok = wait(&sh.peer[s], (n / kStages) & 1, true);
                if (!ok) break;
                tmem_fence_after();
                if (one) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mma_half<kPair>(d, ah + q * next_a, bl + q * next_b, form, q > 0);
                        mma_half<kPair>(d, al + q * next_a, bh + q * next_b, form, true);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_half<kPair>(d, ah + q * next_a, bh + q * next_b, form, true);
                    mma_commit<kPair>(&sh.empty[s]);
                    mma_commit<kPair>(&sh.done[n % F::kAccs]);
                }
                __syncwarp();
            }
        }
        if (one) {
            if (!ok) atomicOr(&g_matrix_status, kStatusConsumerTimeout);
            mma_commit<kPair>(&sh.drain);    // the products in flight end before their memory goes
            if (!mbar_wait(&sh.drain, 0, kDrainNs))
                atomicOr(&g_matrix_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (!skip && warp == 1) {
        if (lane == 0) {
            uint32_t used = 0;
            bool ok = true;
            for (uint32_t i = unit; ok && i < tiles; i += units) {
                const Tile at = tile_at<F>(t, call, i);
                for (int k = 0; k < at.k; k += 64, ++used) {
                    const uint32_t s = used % kStages;
                    ok = mbar_wait(&sh.full[s], (used / kStages) & 1, limit_ns);
                    if (!ok) break;
                    arrive_at_first(&sh.peer[s]);
                }
            }
            if (!ok) atomicOr(&g_matrix_status, kStatusConsumerTimeout);
            // the products that the first block has in flight read this block's stages
            if (!mbar_wait(&sh.drain, 0, 2 * kDrainNs + 2 * limit_ns))
                atomicOr(&g_matrix_status, kStatusDrainTimeout);
        }
    } else if (!skip) {
        volatile Work& my = sh.work[warp - 2];
        if (lane == 0) {
            // the quarter of the lanes that this warp may read, and its columns
            my.lanes = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) +
                       (warp - 2) / 4 * F::kColumns;
            my.out = smem_addr(ring) + kRingBytes + (warp - 2) * kOutPiece;
            my.down = 128 * rank + warp % 4 * 32;
            my.across = (warp - 2) / 4 * F::kColumns;
            my.index = unit;
            my.step = units;
            my.end = tiles;
        }
        __syncwarp();
        uint32_t n = 0;
        for (;;) {
            const bool more = my.index < my.end;
            __syncwarp();                                // all have read what lane 0 moves on
            if (!more) break;
            if (lane == 0) {
                const Tile next = tile_at<F>(t, call, my.index);
                my.tile.matrix = next.matrix;
                my.tile.step = next.step;
                my.tile.row = next.row + my.down;        // this warp's
                my.tile.col = next.col + my.across;
                my.tile.k = next.k;
                my.index += my.step;
            }
            __syncwarp();
            volatile Tile& at = my.tile;
            bool ok = true;
            uint32_t sum[F::kColumns];                   // fp32, then halves
#pragma unroll
            for (int k = 0; k < F::kColumns; ++k) sum[k] = 0u;
            for (int k = 0; k < at.k; k += 64, ++n) {
                // every lane waits, so that all of them see the products
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.done[n % F::kAccs],
                                                       (n / F::kAccs) & 1, limit_ns));
                if (!ok) break;
                tmem_fence_after();
                constexpr int kWide = F::kColumns == 128 ? 32 : 8;   // more take more registers
                const uint32_t from = my.lanes + n % F::kAccs * F::kCols;
#pragma unroll
                for (int c = 0; c < F::kColumns; c += kWide) {
                    uint32_t acc[kWide];
                    if constexpr (kWide == 32) tmem_load32(from + c, acc);
                    else tmem_load8(from + c, acc);
#pragma unroll
                    for (int j = 0; j < kWide; ++j)
                        sum[c + j] = __float_as_uint(__uint_as_float(sum[c + j]) +
                                                     __uint_as_float(acc[j]));
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {                         // the next products may come
                    if constexpr (kPair) tmem_read_at_first(&sh.taken[n % F::kAccs]);
                    else mbar_arrive(&sh.taken[n % F::kAccs]);
                }
            }
            const MatrixItem& x = t.item[at.matrix];
            if (!ok) {
                atomicOr(&g_matrix_status, kStatusConsumerTimeout);
                break;
            }
            const MatrixStep& step = call.step[at.step];
            if (step.flags & kLastStep) {
#pragma unroll
                for (int c = 0; c < F::kColumns; c += 8)
                    finish(x, call, at.row + lane, at.col + c, sum + c, step.scale);
                __syncwarp();
                continue;
            }
            // 32 columns at a time: of the result, then of C where it is A
            const int images = step.flags & kWithC ? 2 : 1;
#pragma unroll
            for (int c = 0; c < F::kColumns; c += 32) {
#pragma unroll 1                                             // twice its code takes more registers
                for (int image = 0; image < images; ++image) {
                    int row = threadIdx.x % 32;
                    asm volatile("" : "+r"(row));            // formed here, not kept
                    const int on = at.row + row - at.col - c;   // the column on the diagonal
                    if (image == 0)
                        split_sums(sum + c, step.scale, step.diagonal, on);
                    else
                        split_again(sum + c, call.c_scale, call.c_diagonal, on);
                    store_words(block_at(x.image[image == 0 ? step.out : kC], at.row, at.col + c,
                                         step.out <= kX1 ? x.np : x.mp) +
                                    at.row % 128 * 128,
                                (at.col + c) % 64 / 8, sum + c, my.out);
                }
            }
            // written, for copies as for loads; then another warp of the matrix is done (the
            // release is for all lanes' stores that the warp's barrier puts before it)
            asm volatile("fence.proxy.async.global;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(x.tiles_done)
                             : "memory");
        }
    }
    tmem_fence_before();
    __syncwarp();
    if constexpr (kPair) pair_sync();
    else __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        tmem_free<kPair, F::kTmemColumns>(tmem);
    }
}

// --------------------------------------------------- moments, norms, images

// The update from the gradient and the new momentum.
__device__ __forceinline__ float update_of(const MatrixItem& x, const MatrixGroup& g, float coef,
                                           float grad, float m) {
    if (x.m_buf == nullptr) return grad;
    return g.nesterov ? fmaf(g.mu, m, g.one_mu * (grad * coef)) : m;
}

// N elements from i on: the momentum, and the sum of the update's squares, in fp32 up to
// kSquaresMost (which a warp's 32 sums still take), beyond it each square in double.
constexpr float kSquaresMost = 0x1p120f;
template <int T, int N>
__device__ __forceinline__ void moments_of(const MatrixItem& x, const MatrixGroup& g, float coef,
                                           int64_t i, float* sum, double* large) {
    float d[N], m[N] = {};
    load_elems<T, N>(static_cast<const typename Elem<T>::Store*>(x.grad) + i, d);
    if (x.m_buf != nullptr) {
        load_elems<kGradF32, N>(x.m_buf + i, m);
#pragma unroll
        for (int k = 0; k < N; ++k) m[k] = fmaf(g.mu, m[k], g.one_mu * (d[k] * coef));
        store_elems<kGradF32, N>(x.m_buf + i, m);
    }
    float s = *sum;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        d[k] = update_of(x, g, coef, d[k], m[k]);
        s = fmaf(d[k], d[k], s);
    }
    if (s <= kSquaresMost) {
        *sum = s;
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) *large += static_cast<double>(d[k] * d[k]);
}

// The momentum, and each part's sum of the update's squares.
template <int T>
__global__ void __launch_bounds__(256) matrix_moments(const __grid_constant__ MatrixTable t,
                                                      const __grid_constant__ MatrixCall call) {
    __shared__ double warp_sum[8];
    pdl_enter();
    if (skip_step(call.skip)) return;
    const int k = find(t.part0, t.count, blockIdx.x);
    const MatrixItem& x = t.item[k];
    const MatrixGroup& g = call.group[x.group];
    const int part = blockIdx.x - t.part0[k], parts = t.part0[k + 1] - t.part0[k];
    if (part == 0 && threadIdx.x == 0) *x.tiles_done = 0;
    const float coef = call.coef != nullptr ? __ldg(call.coef) : 1.0f;
    const int64_t n = static_cast<int64_t>(x.m) * x.n;
    const int64_t first = static_cast<int64_t>(part) * 256 + threadIdx.x;
    const int64_t next = static_cast<int64_t>(parts) * 256;
    float sum = 0.0f;
    double large = 0.0;
    int64_t at = 0;                              // elements done in vectors
    if (x.flat) {
        at = n / 8 * 8;
        for (int64_t i = first; i < n / 8; i += next)
            moments_of<T, 8>(x, g, coef, 8 * i, &sum, &large);
    }
    for (int64_t i = at + first; i < n; i += next)
        moments_of<T, 1>(x, g, coef, i, &sum, &large);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (__any_sync(0xFFFFFFFFu, !(large == 0.0))) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) large += __shfl_xor_sync(0xFFFFFFFFu, large, d);
    }
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = sum + large;
    __syncthreads();
    if (threadIdx.x != 0) return;
    double s = 0.0;                     // in double from warp to warp
    for (int w = 0; w < 8; ++w) s += warp_sum[w];
    x.part[part] = s;
}

// X's image: a block of it per thread block.  All loads go out before the norm is
// added up from its parts.
template <int T>
__global__ void __launch_bounds__(256) matrix_image(const __grid_constant__ MatrixTable t,
                                                    const __grid_constant__ MatrixCall call) {
    using S = typename Elem<T>::Store;
    __shared__ float scale;
    __shared__ uint4 out[kBlockBytes / 16];
    pdl_enter();
    if (skip_step(call.skip)) return;
    const int k = find(t.image0, t.count, blockIdx.x);
    const MatrixItem& x = t.item[k];
    const MatrixGroup& g = call.group[x.group];
    const float coef = call.coef != nullptr ? __ldg(call.coef) : 1.0f;
    const S* grad = static_cast<const S*>(x.grad);
    const int block = blockIdx.x - t.image0[k], wide = x.np / 64;
    const int row0 = block / wide * 128, col0 = block % wide * 64;
    const bool whole = x.flat && !x.tall && x.n % 8 == 0;   // eight columns are one vector
    float u[4][8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        // eight columns of a row; consecutive threads along what memory has in a row
        const int q = p * 256 + threadIdx.x;
        const int row = row0 + (x.tall ? q % 128 : q / 8);
        const int col = col0 + (x.tall ? q / 128 * 8 : q % 8 * 8);
        float m[8] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) u[p][j] = 0.0f;
        if (whole) {
            if (row < x.m && col < x.n) {
                const int64_t i = static_cast<int64_t>(row) * x.n + col;
                load_elems<T, 8>(grad + i, u[p]);
                if (x.m_buf != nullptr) load_elems<kGradF32, 8>(x.m_buf + i, m);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (row >= x.m || col + j >= x.n) continue;
                const int64_t i = x.tall ? static_cast<int64_t>(col + j) * x.m + row
                                         : static_cast<int64_t>(row) * x.n + col + j;
                u[p][j] = elem_to_f32<T>(grad[i]);
                if (x.m_buf != nullptr) m[j] = x.m_buf[i];
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[p][j] = update_of(x, g, coef, u[p][j], m[j]);
    }
    // by one warp: an SM has few double-precision units (9.4M elements: the pass takes 27 us,
    // and 37 where every thread forms the scale)
    if (threadIdx.x < 32) {
        const int parts = t.part0[k + 1] - t.part0[k];
        double s = 0.0;
#pragma unroll
        for (int q = 0; q < kMatrixParts / 32; ++q)
            if (threadIdx.x + 32 * q < parts) s += x.part[threadIdx.x + 32 * q];
#pragma unroll
        for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        // a sum that is not finite leaves nothing finite
        if (threadIdx.x == 0)
            scale = s <= 1.7976931348623157e308
                        ? static_cast<float>(kImageScaleX / (sqrt(s) + call.eps))
                        : __int_as_float(0x7FFFFFFF);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int q = p * 256 + threadIdx.x;
        const int r = x.tall ? q % 128 : q / 8, c = x.tall ? q / 128 * 8 : q % 8 * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)       // padding stays zero whatever the scale is
            v[j] = row0 + r < x.m && col0 + c + j < x.n ? scale * u[p][j] : 0.0f;
        uint4 hi, lo;
        split_pair(v[0], v[1], &hi.x, &lo.x);
        split_pair(v[2], v[3], &hi.y, &lo.y);
        split_pair(v[4], v[5], &hi.z, &lo.z);
        split_pair(v[6], v[7], &hi.w, &lo.w);
        const int at = swizzled(r, c) / 16;
        out[at] = hi;
        out[kBlockBytes / 32 + at] = lo;
    }
    __syncthreads();
    // on in the image's order: a tall matrix's threads hold 16 bytes of a row each
    uint4* to = reinterpret_cast<uint4*>(static_cast<char*>(x.image[kX0]) +
                                         static_cast<int64_t>(block) * kBlockBytes);
#pragma unroll
    for (int q = 0; q < kBlockBytes / 16; q += 256) to[q + threadIdx.x] = out[q + threadIdx.x];
}

// Blocks of the rounds' kernel that can be resident at once, by device.
template <class F>
int resident_units() {
    static std::atomic<int> cache[256];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return 0;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (cudaFuncSetAttribute(matrix_rounds<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             F::kDynamicBytes) != cudaSuccess)
        return 0;
    v = device_sms();
    if constexpr (F::kPair) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {2, 1, 1};
        cfg.gridDim = dim3(static_cast<unsigned>(v / 2 * 2));
        cfg.blockDim = dim3(F::kThreads);
        cfg.dynamicSmemBytes = F::kDynamicBytes;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, matrix_rounds<F>, &cfg) != cudaSuccess)
            return 0;
        v = clusters < v / 2 ? clusters : v / 2;
    }
    if (v > 0) cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

template <class F>
cudaError_t go_rounds(const MatrixTable& t, const MatrixCall& c, cudaStream_t stream) {
    const uint32_t most = c.most;
    const int fit = resident_units<F>();
    if (fit < 1) return cudaErrorLaunchOutOfResources;
    const uint32_t units = most < static_cast<uint32_t>(fit) ? most : static_cast<uint32_t>(fit);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {2, 1, 1};
    cfg.gridDim = dim3(units * F::kBlocks);
    cfg.blockDim = dim3(F::kThreads);
    cfg.dynamicSmemBytes = F::kDynamicBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = F::kPair ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, matrix_rounds<F>, t, c, tma_wait_limit());
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
    if (e != cudaSuccess) return e;
    return t.shape == 2   ? go_rounds<Shape<256, 256>>(t, c, stream)
           : t.shape == 1 ? go_rounds<Shape<128, 128>>(t, c, stream)
                          : go_rounds<Shape<128, 64>>(t, c, stream);
}

}  // namespace shardstep
