// Internal interface between the host-side C ABI (api.cpp) and the kernel
// translation units.  Plain C++; no device code.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "shardstep.h"

namespace shardstep {

// fp32 per-step scalars of the AdamW update (derived in double, on the host
// or by the state-advance kernel).  With `dev` set, each kernel replaces the
// eight values at its start by the eight floats at dev (the scalars of a
// device-resident step state, in this field order).
struct AdamScalars {
    float lr_wd, beta1, omb1, beta2, omb2, step_size, sqrt_bc2, eps;
    const float* dev;
};
static_assert(offsetof(shardstep_adamw_state_t, scalars) == 24, "state layout");

// The device-resident step state (api.cpp / step.cu): init writes step t's
// powers (and scalars for t >= 1), advance moves t to t + 1.
cudaError_t launch_adamw_state_set(shardstep_adamw_state_t* state, int64_t step, double b1p,
                                   double b2p, double lr, double beta1, double beta2, double eps,
                                   double wd, cudaStream_t stream);
cudaError_t launch_adamw_state_advance(shardstep_adamw_state_t* state, double lr, double beta1,
                                       double beta2, double eps, double wd,
                                       const unsigned int* skip, cudaStream_t stream);

// How the reduce turns the N_d rank slices into a mean: the slices are summed
// in groups of `group` consecutive ranks (group == N_d: one rank-order sum;
// 1 < group < N_d: hybrid sharding, group sums first, then across groups),
// then the total is divided by N_d, correctly rounded (div_nd: a multiply by
// the exact reciprocal when N_d is a power of two, else a multiply by
// inv_nd = RN(1/N_d) and one fma correction).
// With `scaled` set, the mean is then multiplied by inv_scale, the gradient
// scaler's 1/s, which each kernel computes at start from the device word
// *scale (resolve_scale).
struct MeanOp {
    float inv_nd;
    float nd;
    int pow2;
    int group;
    float inv_scale;
    int scaled;
    const float* scale;
};

// Gradient element types the fused kernels read (the C ABI's dtype codes).
constexpr int kGradBF16 = SHARDSTEP_DTYPE_BF16;
constexpr int kGradF32 = SHARDSTEP_DTYPE_F32;
constexpr int kGradF16 = SHARDSTEP_DTYPE_F16;

struct PtrTable {
    const void* p[SHARDSTEP_MAX_ND];
};

// One contiguous byte range to copy (src == nullptr: fill with zeros).
constexpr int kMaxCopySegs = 64;
struct CopySeg {
    const char* src;
    char* dst;
    int64_t bytes;
    int64_t chunk0;  // first chunk index of this segment in the launch
    int64_t body;    // vectors of `width` bytes after the head
    int32_t width;   // 16, 8, 4, 2 or 1
    int32_t head;    // bytes before dst is `width`-aligned
};
struct CopyTable {
    CopySeg s[kMaxCopySegs];
    int32_t n;
    int64_t total_chunks;
};
constexpr int kCopyVecsPerChunk = 1024;  // 256 threads x 4

// Byte ranges for the aligned copy: source, destination and size all
// multiples of 16 bytes; cut into chunks of kAlignedChunk bytes, one block
// each.
constexpr int kAlignedChunk = 16384;
struct AlignedSeg {
    const char* src;
    char* dst;
    int64_t bytes;
    int64_t chunk0;  // first chunk index of this range in the launch
};
struct AlignedTable {
    AlignedSeg s[kMaxCopySegs];
    int32_t n;
    int64_t total_chunks;
};

// Launches `kernel` as a programmatic dependent of the previous kernel in
// `stream`: it may start while that kernel drains.  Only for launches whose
// kernel neither reads nor writes anything the previous kernel writes, and
// which wait (pdl_wait) for it before they end.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// Whether kernels go out as programmatic dependent launches
// (shardstep_set_dependent_launch; api.cpp).
bool dependent_launches();

// Launches `kernel` as a programmatic dependent of the previous kernel in the
// stream when dependent launches are on, else as an ordinary launch.  The
// kernel must begin with pdl_enter() (it waits for its predecessor before it
// touches memory), so stream order holds whatever the predecessor is.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent_launches() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// Launch bookkeeping (api.cpp).
void note_launch();
int device_sms();                                   // SMs of the current device (cached)
int resident_blocks(const void* kernel, int threads);  // per SM, cached per kernel

// Launchers (return the CUDA error of the launch).
// `skip` (may be null): a device word; when it holds a non-zero value at
// launch the kernel changes nothing (the gradient scaler's skipped step).
cudaError_t launch_rs_adamw_cast(const PtrTable& tab, int nd, int grad_type, int64_t S,
                                 float* master, float* m, float* v, uint16_t* out,
                                 const AdamScalars& c, const MeanOp& mo,
                                 const unsigned int* skip, bool vec, cudaStream_t stream);
// TMA-staged kernels (step_tma.cu).  Each needs every source 16-byte aligned,
// at least kTmaMinElements elements and two stages in shared memory (the
// *_fits checks: the fused step's stage holds N_d slices + 3 state arrays,
// the all-reduce's and the check's N_d slices).  set_tma_stage_limit fixes
// the stages per launch (0: about 128 KB of tiles in flight per SM; returns
// the previous setting).
bool tma_step_fits(int nd, int grad_type);
bool tma_reduce_fits(int nd, int grad_type);
int set_tma_stage_limit(int stages);
// The TMA-staged kernels' wait limit in ns (0: the default of two seconds);
// read at each launch.  Returns the previous limit.
int64_t set_tma_wait_ns(int64_t ns);
unsigned long long tma_wait_limit();
// The status word of the staged loss kernels (token_loss.cu).
cudaError_t read_loss_status(unsigned int* status, bool clear);
cudaError_t launch_rs_adamw_cast_tma(const PtrTable& tab, int nd, int grad_type, int64_t S,
                                     float* master, float* m, float* v, uint16_t* out,
                                     const AdamScalars& c, const MeanOp& mo,
                                     const unsigned int* skip, cudaStream_t stream);
cudaError_t launch_accumulate_tma(const uint16_t* g, float* acc, int64_t n, float scale,
                                  bool first, cudaStream_t stream);
// pdl: launch as a programmatic dependent of the previous bucket's kernel
// (later buckets of one ddp_bucket_allreduce_avg call).
cudaError_t launch_allreduce_avg_tma(const PtrTable& tab, int nd, int64_t n, uint16_t* out,
                                     const MeanOp& mo, bool pdl, cudaStream_t stream);
cudaError_t launch_nonfinite_check_tma(const PtrTable& tab, int nd, int grad_type, int64_t S,
                                       const MeanOp& mo, unsigned int* found,
                                       cudaStream_t stream);
// Gradient scaler (step.cu): the non-finite check of the unscaled mean and
// the scale update.
cudaError_t launch_nonfinite_check(const PtrTable& tab, int nd, int grad_type, int64_t S,
                                   const MeanOp& mo, unsigned int* found, bool vec,
                                   cudaStream_t stream);
cudaError_t launch_scaler_update(float* scale, int* tracker, unsigned int* found,
                                 float growth, float backoff, int interval, cudaStream_t stream);
cudaError_t read_device_status(unsigned int* status, bool clear);
int device_smem_optin();  // max dynamic shared memory per block (cached)
constexpr int64_t kTmaMinElements = 4096;

cudaError_t launch_allreduce_avg(const PtrTable& tab, int nd, int64_t n, uint16_t* out,
                                 const MeanOp& mo, bool vec, bool pdl, cudaStream_t stream);
// The segments of one FSDP2 step launch (launch_rs_adamw_cast_segs): segment
// s covers local elements [lo[s], lo[s] + n[s]) and reads the N_d slices
// p[po[s] + q] (po[s] < 0: padding rows, every contribution +0, no
// pointers); b0[s] is its first block, b0[ns] the launch's block count.
// About 2.9 KB as a kernel parameter.
constexpr int kSegMax = 32;
constexpr int kSegPtrMax = 256;
struct SegTable {
    const void* p[kSegPtrMax];
    int64_t lo[kSegMax];
    int64_t n[kSegMax];
    int64_t b0[kSegMax + 1];
    int32_t po[kSegMax];
    int ns;
};
// Blocks one segment of n elements takes in launch_rs_adamw_cast_segs.
int64_t seg_blocks(int64_t n);
// One launch over the table's segments: the fused step's reduce (rank
// order), mean, AdamW and cast; every segment 16-byte aligned in the state
// and 8-byte (16-bit slices) or 16-byte (fp32 slices) in its slices.
cudaError_t launch_rs_adamw_cast_segs(const SegTable& st, int nd, int grad_type, float* master,
                                      float* m, float* v, uint16_t* out, const AdamScalars& c,
                                      const MeanOp& mo, cudaStream_t stream);
// AdamW with a zero gradient over n elements (FSDP2 padding rows).
cudaError_t launch_adamw_zero_grad(int64_t n, float* master, float* m, float* v, uint16_t* out,
                                   const AdamScalars& c, cudaStream_t stream);
// The DDP all-reduce average fused with the replicated AdamW + cast over n
// bucketed elements (step.cu); mean_out may be null.  `vec`: state 16-byte,
// gradients, mean_out and out 8-byte aligned.
cudaError_t launch_ddp_allreduce_adamw_cast(const PtrTable& tab, int nd, int64_t n,
                                            uint16_t* mean_out, float* master, float* m,
                                            float* v, uint16_t* out, const AdamScalars& c,
                                            const MeanOp& mo, bool vec, cudaStream_t stream);
// Division self-check (step.cu): counts into *mismatches the fp32 patterns
// for which the reduce's division by N_d differs from IEEE division and
// lowers *first_bad to the smallest of them.
cudaError_t launch_mean_division_check(const MeanOp& mo, unsigned long long* mismatches,
                                       unsigned int* first_bad, cudaStream_t stream);
// The copy launchers' `pdl`: launch as a programmatic dependent of the
// previous kernel in the stream.  `wait_first`: the kernel waits for that
// predecessor before it touches memory (the first launch of a call, whose
// predecessor is unknown); without it the kernel waits only before it ends
// (a later launch of the same batch of disjoint copies, so that it overlaps
// the previous one's drain; the batch's last kernel still completes after
// all of them).
cudaError_t launch_copy(const CopyTable& t, bool pdl, bool wait_first, cudaStream_t stream);
// Aligned copy (copy.cu): one block per 16 KB chunk of 16-byte vectors.
cudaError_t launch_copy16(const AlignedTable& t, bool pdl, bool wait_first, cudaStream_t stream);
// Realigning copy (copy.cu): like copy16, but every source starts 1..15
// bytes past a 16-byte boundary (destinations and sizes 16-byte multiples).
cudaError_t launch_copy16_shift(const AlignedTable& t, bool pdl, bool wait_first,
                                cudaStream_t stream);
cudaError_t launch_accumulate(const uint16_t* g, float* acc, int64_t n, float scale, bool first,
                              bool vec, cudaStream_t stream);
// The last micro-batch's accumulation fused into the step (accum_step.cu):
// fp32 accumulator slices `acc`, bf16 last micro-batch slices `last`; `vec`:
// accumulators and state 16-byte aligned, bf16 slices and output 8-byte.
cudaError_t launch_accum_rs_adamw_cast(const PtrTable& acc, const PtrTable& last, int nd,
                                       int64_t S, float scale, float* master, float* m,
                                       float* v, uint16_t* out, const AdamScalars& c,
                                       const MeanOp& mo, bool vec, cudaStream_t stream);

// ------------------------------------------------- lists of tensors
// (tensors.cu; host side in tuning_api.cpp)

// The AdamW hyper-parameter groups of one launch.
constexpr int kMaxGroups = SHARDSTEP_MAX_GROUPS;
// Tensors of one launch: the table travels as a kernel parameter, whose limit
// is 32764 bytes; the smaller capacity keeps the parameter block of the usual
// short lists small.
constexpr int kTensorsSmall = 32;
constexpr int kTensorsLarge = 400;
// Elements that share one scale of the 8-bit moments.
constexpr int kMomentBlock = SHARDSTEP_MOMENT_BLOCK;

// A launch's blocks in up to kNear runs of 2^near_shift, so that a block looks for
// its tensor among those of its run, mostly one.
constexpr int kNear = 128;
template <int CAP>
struct TensorTable {
    const void* grad[CAP];
    float* master[CAP];
    void* m[CAP];
    void* v[CAP];
    float* m_scale[CAP];
    float* v_scale[CAP];
    void* param[CAP];
    int64_t n[CAP];
    uint32_t b0[CAP + 1];   // first block of each tensor; b0[count] = the launch's blocks
    uint16_t group[CAP];
    uint8_t vec[CAP];       // every array of the tensor takes 16-byte accesses
    uint16_t near[kNear + 1];   // the tensor of block k << near_shift (the last one: of the end)
    int32_t near_shift;
    int32_t count;
};
struct GroupScalars {
    AdamScalars c[kMaxGroups];
    float inv_sqrt_bc2[kMaxGroups];   // RN(1 / c[g].sqrt_bc2), host scalars only
    float neg_zero;                   // -0.0f, unknown to the compiler
};
// Elements one block of the list kernels covers.
constexpr int kListChunk32 = 2048;
constexpr int kListChunk8 = 8 * kMomentBlock;

template <int CAP>
cudaError_t launch_tensors_adamw(const TensorTable<CAP>& t, int grad_type, int param_type,
                                 int bits, const GroupScalars& gs, const float* coef,
                                 const unsigned int* skip, cudaStream_t stream);
cudaError_t launch_moments_decode(const uint8_t* m, const float* m_scale, const uint8_t* v,
                                  const float* v_scale, int64_t n, float* m_out, float* v_out,
                                  bool vec, cudaStream_t stream);
cudaError_t launch_moments_encode(const float* m_in, const float* v_in, int64_t n, uint8_t* m,
                                  float* m_scale, uint8_t* v, float* v_scale, bool vec,
                                  cudaStream_t stream);

template <int CAP>
struct NormTable {
    const void* p[CAP];
    int64_t n[CAP];
    uint32_t b0[CAP + 1];   // first chunk of each tensor; b0[count] = the launch's chunks
    uint8_t vec[CAP];
    int32_t count;
};
constexpr int kNormSmall = 64;
constexpr int kNormLarge = 1200;
constexpr int kNormChunk = 8192;      // elements of one chunk
constexpr int kNormMaxBlocks = 1024;  // partial sums in the workspace
// The norm's workspace: an arrival counter, then one double per block.
struct NormWork {
    unsigned int arrived;
    unsigned int pad_[3];
    double partial[kNormMaxBlocks];
};
struct NormArgs {
    NormWork* ws;
    const float* scale;       // may be null: 1
    float max_norm;
    float* out;               // {norm, factor}
    unsigned int* found;      // may be null
    int first, last;          // this launch starts / ends the call
};
template <int CAP>
cudaError_t launch_tensors_norm(const NormTable<CAP>& t, int type, const NormArgs& a, int blocks,
                                cudaStream_t stream);

// ---------------------------------------------------- losses over tokens
// (token_loss.cu; host side in tuning_api.cpp)

constexpr int kLossMaxBlocks = 1024;
// The workspace of the token losses; the preference loss's per-token and
// per-sequence words follow it.
constexpr int kPairsPerLaunch = 1024;
struct LossWork {
    unsigned int arrived;
    unsigned int pad_[3];
    double total[4];                        // carried from launch to launch
    double partial[kLossMaxBlocks][4];      // the blocks' sums
    unsigned int rows_done[kPairsPerLaunch];  // of each pair; zero between launches
    double pair_loss[kPairsPerLaunch][3];     // of each pair: loss, margin, margin > 0
};
struct TokenArgs {
    const void* x;          // logits, row i at x + i * x_stride
    int64_t x_stride;       // elements
    void* grad;             // or null: forward only
    int64_t g_stride;
    const void* ids;
    int ids64;
    const float* w;         // or null: ones
    const float* ref;
    float* logps;
    int64_t n, v;
    float grad_scale;
    const float* loss_scale;  // or null
    float norm;               // 0: the sum of the weights (policy)
    float* stats;
    LossWork* ws;
};
struct PolicyArgs {
    const float* old;
    const float* adv;
    float lo, hi, kl;
};
// The sequences of one launch of the preference loss: pairs 2 p, 2 p + 1 are
// its rows [start[2 p], start[2 p + 1]) and [start[2 p + 1], start[2 p + 2]).
template <int CAP>
struct PairTable {
    int32_t start[2 * CAP + 1];
    int32_t pairs;
};
constexpr int kPairsSmall = 64;   // 520 bytes of kernel parameter; the other 8 KB
using PairTableLarge = PairTable<kPairsPerLaunch>;
struct PreferenceArgs {
    float beta, smoothing;
    float* log_ratios;      // 2 per pair
    float* row_ref;         // per token: what its exponents refer to
    float* row_sum;         // per token: the sum of its exponentials
    float* term;            // per token: w (a - ref); of the policy loss c, or null
    int32_t* seq;           // per token: its sequence within the launch
    float* coef;            // per sequence: d loss / d a at weight 1; null: policy
    int first, last;        // this launch starts / ends the call
};
// Whether a row of v elements fits the staged policy kernel's shared memory.
bool loss_row_fits(int64_t v, int dtype);
// A call's rows go in launches of at most this many (loss_rows_per_launch), so
// that a block's share of them fits its shared memory.
constexpr int kShareRows = 1024;   // per SM
int64_t loss_rows_per_launch();
// The policy loss forward and backward; the rows fit and can be staged.
cudaError_t launch_policy_staged(const TokenArgs& a, const PolicyArgs& pol, int64_t begin,
                                 int64_t end, int dtype, cudaStream_t stream);
// Forward; with p.term also p.term, p.row_ref and p.row_sum for the backward pass.
cudaError_t launch_policy_forward(const TokenArgs& a, const PolicyArgs& pol,
                                  const PreferenceArgs& p, int64_t begin, int64_t end, int dtype,
                                  cudaStream_t stream);
cudaError_t launch_preference_forward(const TokenArgs& a, const PreferenceArgs& p,
                                      const PairTableLarge& t, int64_t begin, int64_t end,
                                      int dtype, cudaStream_t stream);
// The gradient from what a forward pass has left.  staged: the gradient's rows
// start at the logits' rows' offsets from 16-byte boundaries.
cudaError_t launch_loss_backward(const TokenArgs& a, const PreferenceArgs& p, int64_t begin,
                                 int64_t end, int dtype, bool staged, cudaStream_t stream);

// ------------------------------------------- embedding and layer norm
// (embedding.cu, layer_norm.cu; host side in model_api.cpp)

// Token i's row at rows + i * row_stride (the lookup's output, the gradient's
// d_out), id v's at table + v * table_stride (the table, or its gradient).
struct EmbedArgs {
    void* table;
    int64_t table_stride;   // elements, as row_stride
    void* rows;
    int64_t row_stride;
    const void* ids;
    int ids64;
    int accumulate;
    int64_t n, vocab, dim;
    float scale;
};
constexpr int kEmbedChunkMax = 512;    // sorted tokens of a chunk
constexpr int kEmbedSortRange = 1024;  // ids of a sorting block
constexpr int kEmbedZeroRows = 16;     // rows that a block looks through for absent ids
struct EmbedPlan {
    int chunk;              // sorted tokens per block
    int64_t chunks;
};
EmbedPlan embed_plan(int64_t n, int64_t dim);
// The gradient's workspace.
struct EmbedSort {
    int32_t* token;         // sorted by id; n each
    int32_t* id;
    uint32_t* row_start;    // vocab + 1: each id's first place in the list
    float* piece;           // 2 * dim per chunk: of a run from before, of one that goes on
    int range, chunk;
    int64_t chunks, slices;
};
cudaError_t launch_embedding(const EmbedArgs& a, int type, bool vec, cudaStream_t stream);
cudaError_t launch_embedding_grad(const EmbedArgs& a, EmbedSort s, int in_type, int out_type,
                                  bool vec, cudaStream_t stream);

struct NormRows {
    const void* x;
    int64_t x_stride;       // elements, as all strides
    void* out;
    int64_t out_stride;
    const void *w, *b;      // or null
    float *mean, *rstd;
    int64_t rows, cols;
    float eps;
};
struct NormGradRows {
    const void* x;
    int64_t x_stride;
    const void* d;
    int64_t d_stride;
    void* d_x;              // or null
    int64_t d_x_stride;
    const void* w;          // or null
    const float *mean, *rstd;
    float* piece;           // 2 * pitch per block, or null: no d_w, d_b
    int64_t rows, cols, pitch;
};
// Blocks of the backward pass, each of which leaves one row of column sums; at
// most kNormPieces.
constexpr int kNormPieces = 160;
cudaError_t read_norm_status(unsigned int* status, bool clear);
// vec: the rows that are read, the weights and the bias take vectors; whole: the rows
// that are written do.
cudaError_t launch_layer_norm(const NormRows& a, int type, int w_type, bool vec, bool whole,
                              cudaStream_t stream);
cudaError_t launch_layer_norm_grad(const NormGradRows& a, int type, int w_type, void* d_w,
                                   void* d_b, int accumulate, bool vec, bool whole,
                                   cudaStream_t stream);
// The kernels that these launch for the rows.
const char* layer_norm_kernel(int64_t cols, int type, bool vec, bool whole);
const char* layer_norm_grad_kernel(const NormGradRows& a, int type, bool vec, bool whole);

// ------------------------------------------------ matrices' updates
// (matrix.cu; host side in model_api.cpp)

constexpr int kMatrices = 64;        // of one group: a launch's table
constexpr int kMatrixParts = 256;    // sums of squares of one matrix
// The images of a matrix in the workspace: X twice, then symmetric ones of its short
// side: A = X X^T, C = b + c A, P = a + A C twice, A P, and the product of the P.
enum MatrixImage { kX0, kX1, kA, kC, kP0, kP1, kZ, kQ, kImages };
struct MatrixItem {
    const void* grad;                // m x n, or n x m where tall
    float* master;                   // null: `out` takes the orthogonal matrix
    float* m_buf;                    // momentum, or null
    void* out;                       // the parameter (may be null), or the result
    void* image[kImages];
    double* part;
    unsigned int* tiles_done;        // result warps of all steps so far
    float step;                      // learning rate times the matrix's factor
    int32_t m, n, mp, np;            // m <= n, and padded to the tile
    int16_t tall, group;
    int32_t whole;                   // master and out take whole vectors of 8 along rows
    int32_t flat;                    // grad and m_buf take whole vectors of 8
};
constexpr int kMatrixTiles[3][2] = {{128, 64}, {128, 128}, {256, 256}};
struct MatrixTable {
    MatrixItem item[kMatrices];
    uint32_t sym0[kMatrices + 1];    // first tile of the symmetric products
    uint32_t full0[kMatrices + 1];   // of the others
    uint32_t part0[kMatrices + 1];   // first sum of squares
    uint32_t image0[kMatrices + 1];  // first image block of x
    int32_t count;
    int32_t shape;                   // of the tiles: kMatrixTiles[shape]
    int32_t twos;                    // rounds are taken two at a time
};
struct MatrixGroup {
    float lr_wd, mu, one_mu;
    int nesterov;
};
// One product of the rounds, of all matrices: out = scale left right + diagonal.
enum MatrixStepFlags {
    kSymmetric = 1,       // its tiles on and above the diagonal only
    kLeftX = 2,           // rows of X on the left
    kRightX = 4,          // X behind a symmetric matrix
    kWithC = 8,           // write C beside A
    kLastStep = 16,       // the result itself
};
struct MatrixStep {
    uint32_t first;                  // tile of the call
    float scale, diagonal;           // of the values as the images hold them
    uint16_t sym_before, full_before;   // steps that have to be done, of either kind
    uint8_t left, right, out, flags;
};
constexpr int kMatrixSteps = 256;
constexpr float kImageScaleX = 32768.0f;   // what X's images hold X times
struct MatrixCall {
    MatrixGroup group[kMaxGroups];
    const float* coef;
    const unsigned int* skip;
    float a, b, c, eps;
    int rounds, out_type;
    float c_scale, c_diagonal;       // C from A, as the images hold them
    uint32_t tiles, most;            // of all steps, of the largest
    int steps;
    MatrixStep step[kMatrixSteps];
};
cudaError_t launch_matrices(const MatrixTable& t, const MatrixCall& c, int grad_type,
                            cudaStream_t stream);
cudaError_t read_matrix_status(unsigned int* status, bool clear);

// Host helpers of api.cpp for the other translation units: the last error of
// the calling thread, the name shardstep_last_kernel reports, the per-step
// scalars.
int ready_fail(int code, const char* fmt, ...);
int ready_ok();
void record_kernel(const char* fmt, ...);
AdamScalars host_adam_scalars(const shardstep_adamw_t& hp);

}  // namespace shardstep
