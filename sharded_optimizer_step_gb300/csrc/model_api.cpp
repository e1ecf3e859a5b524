// Host side of the embedding (token_embedding*), layer norm (rows_layer_norm*)
// and the matrices' updates (matrices_*, tensors_muon_step): argument checks, the
// products that make up the rounds, the tables that travel with each launch, and
// dispatch.  Nothing here allocates
// device memory or keeps a pointer.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <numeric>
#include <vector>

#include "checks.h"
#include "internal.h"
#include "shardstep.h"

namespace shardstep {
namespace {

int64_t span(int64_t rows, int64_t cols, int64_t stride, int es) {
    return rows > 0 ? ((rows - 1) * stride + cols) * es : 0;
}
// Whether every row starts on a 16-byte boundary.
bool rows_aligned(const void* p, int64_t stride, int64_t rows, int es) {
    return aligned(p, 16) && (rows <= 1 || stride * es % 16 == 0);
}
bool stride_ok(int64_t stride, int64_t rows, int64_t cols) {
    return stride >= cols && (rows == 0 || stride <= (int64_t{1} << 60) / rows);
}
int cuda_fail(const char* what, cudaError_t e) {
    return ready_fail(SHARDSTEP_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

// -------------------------------------------------------------- embedding

bool embed_sizes(int64_t n, int64_t vocab, int64_t dim) {
    return n >= 0 && n <= INT32_MAX && vocab >= 1 && vocab < INT32_MAX && dim >= 1 &&
           dim <= (int64_t{1} << 23);
}

// The checks that both directions share.
int check_embedding(const void* table, int64_t table_stride, int64_t vocab, int64_t dim,
                    const void* ids, int32_t id_bytes, int64_t n, float scale, const void* rows,
                    int64_t row_stride, int es_table, int es_rows) {
    if (es_table == 0 || es_rows == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype");
    if (id_bytes != 4 && id_bytes != 8)
        return ready_fail(SHARDSTEP_ERR_INVALID, "id_bytes must be 4 or 8");
    if (!embed_sizes(n, vocab, dim))
        return ready_fail(SHARDSTEP_ERR_INVALID, "n, vocab or dim out of range");
    if (!std::isfinite(scale)) return ready_fail(SHARDSTEP_ERR_INVALID, "scale is not finite");
    if (!stride_ok(table_stride, vocab, dim) || !stride_ok(row_stride, n, dim))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a row stride is out of range");
    if (!table || (n > 0 && (!ids || !rows)))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a NULL array");
    if (!aligned(table, es_table) || !aligned(rows, es_rows) || !aligned(ids, id_bytes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an array is misaligned");
    return SHARDSTEP_OK;
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// --------------------------------------------------------------- matrices

constexpr int64_t kSideMax = int64_t{1} << 20;
constexpr int64_t kGroupBytes = int64_t{2} << 30;

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }
constexpr int64_t kMatrixWords = kMatrixParts * sizeof(double) + 128;   // sums and a counter
// A matrix's part of the workspace: two images of X, six of symmetric matrices, the
// words (with either tile).
int64_t matrix_bytes(int64_t rows, int64_t cols) {
    const int64_t m = padded(std::min(rows, cols), 256), n = padded(std::max(rows, cols), 256);
    return 8 * m * n + 24 * m * m + kMatrixWords;
}
bool side_ok(int64_t n) { return n >= 0 && n <= kSideMax; }

struct Sides {
    int64_t rows, cols;
};
// The end of the group that starts at `at`, and its workspace.
template <typename F>
int32_t group_end(const F& sides, int32_t n, int32_t at, int64_t* bytes) {
    int count = 0;
    *bytes = 0;
    for (; at < n; ++at) {
        const Sides s = sides(at);
        if (s.rows == 0 || s.cols == 0) continue;
        const int64_t b = matrix_bytes(s.rows, s.cols);
        if (count == kMatrices || (count > 0 && *bytes + b > kGroupBytes)) break;
        *bytes += b;
        ++count;
    }
    return at;
}
template <typename F>
int64_t workspace_for(const F& sides, int32_t n) {
    int64_t most = 0;
    for (int32_t at = 0; at < n;) {
        int64_t bytes;
        at = group_end(sides, n, at, &bytes);
        most = std::max(most, bytes);
    }
    return most;
}

// The largest magnitude of a x + b x^3 + c x^5 over [0, hi].
double quintic_most(double a, double b, double c, double hi) {
    const auto f = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
    double most = f(hi);
    // where a + 3 b t + 5 c t^2 = 0, t = x^2
    const double q = 9 * b * b - 20 * a * c;
    const auto at = [&](double t) {
        if (t > 0 && t < hi * hi) most = std::max(most, f(std::sqrt(t)));
    };
    if (c != 0 && q >= 0) {
        at((-3 * b + std::sqrt(q)) / (10 * c));
        at((-3 * b - std::sqrt(q)) / (10 * c));
    } else if (c == 0 && b != 0) {
        at(-a / (3 * b));
    }
    return most;
}
// The largest magnitude of a + b t + c t^2 over [0, hi].
double square_most(double a, double b, double c, double hi) {
    const auto f = [&](double t) { return std::fabs(a + t * (b + t * c)); };
    double most = std::max(f(0.0), f(hi));
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < hi) most = std::max(most, f(-b / (2 * c)));
    return most;
}

int take_quintic(const shardstep_quintic_t* q, MatrixCall* call) {
    if (q == nullptr) return ready_fail(SHARDSTEP_ERR_INVALID, "quintic is NULL");
    if (q->rounds < 1 || q->rounds > 64)
        return ready_fail(SHARDSTEP_ERR_INVALID, "rounds must be 1..64 (got %d)", q->rounds);
    if (!std::isfinite(q->a) || !std::isfinite(q->b) || !std::isfinite(q->c) ||
        !(q->eps >= 0) || !std::isfinite(q->eps))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a coefficient or eps is out of range");
    if (std::fabs(q->a) < 1)      // small singular values shrink by it in every round
        return ready_fail(SHARDSTEP_ERR_INVALID,
                          "|a| is below 1: values shrink below what halves hold");
    double hi = 1.0;
    for (int32_t k = 0; k < q->rounds; ++k) {
        // X and A are held times 2^15 in halves, which end at 65504, b + c A times 2^13
        // and a + b A + c A A times 2^14
        if (!(hi <= 1.39) || !(square_most(q->b, q->c, 0.0, hi * hi) <= 7.9) ||
            !(square_most(q->a, q->b, q->c, hi * hi) <= 3.9))
            return ready_fail(SHARDSTEP_ERR_INVALID,
                              "the coefficients let values grow past what round %d holds", k + 1);
        hi = std::max(hi, quintic_most(q->a, q->b, q->c, hi));
    }
    call->a = static_cast<float>(q->a);
    call->b = static_cast<float>(q->b);
    call->c = static_cast<float>(q->c);
    call->eps = static_cast<float>(q->eps);
    call->rounds = q->rounds;
    return SHARDSTEP_OK;
}

// The matrices [at, end) of the list; false: all are empty.
template <typename F>
bool take_group(const F& item, int32_t at, int32_t end, MatrixTable* t) {
    t->count = 0;
    for (; at < end; ++at) {
        MatrixItem x{};
        int64_t rows, cols;
        item(at, &x, &rows, &cols);
        if (rows == 0 || cols == 0) continue;
        x.tall = rows > cols;
        x.whole = std::max(rows, cols) % 8 == 0 && aligned(x.master, 16) && aligned(x.out, 16);
        x.flat = aligned(x.grad, 16) && aligned(x.m_buf, 16);
        x.m = static_cast<int32_t>(std::min(rows, cols));
        x.n = static_cast<int32_t>(std::max(rows, cols));
        t->item[t->count++] = x;
    }
    return t->count > 0;
}

// The products of all rounds.  One round at a time these are A = X X^T, P = a + A C and
// X = P X.  Rounds can also be taken two at a time without forming X in between, since
// everything is a polynomial in A: A' = (P X)(P X)^T = (A P) P, the next P from it, and
// X = P' P X.  That is 2 products with X and 5 without instead of 4 and 2: for 5 rounds of
// an m x n matrix 9 m^2 n + 11 m^3 (products of symmetric matrices half) instead of
// 15 m^2 n + 5 m^3.  Errors of the products between grow where X's own round would have
// settled them, so the last round is always by itself.  Five rounds are then off by up to
// 1.8 times what 32-bit products are at a short side of 512 and 1.2 from 1024 on (round by
// round 0.8), but 2.2 to 5.5 times at sides of 64 to 256 (1 to 2), which go round by round;
// with two rounds at the end up to 2.7 times, with three at once up to 10.
void plan_steps(MatrixCall* call, bool segments) {
    double scale[kImages];
    scale[kX0] = scale[kX1] = scale[kA] = scale[kZ] = kImageScaleX;
    scale[kC] = kImageScaleX / 4;
    scale[kP0] = scale[kP1] = kImageScaleX / 2;
    scale[kQ] = kImageScaleX / 8;              // its elements are below 3.9 squared
    call->c_scale = static_cast<float>(call->c * scale[kC] / scale[kA]);
    call->c_diagonal = static_cast<float>(call->b * scale[kC]);
    int sym = 0, full = 0;
    call->steps = 0;
    const auto add = [&](int left, int right, int out, int flags) {
        MatrixStep& s = call->step[call->steps++];
        s = MatrixStep{};
        s.left = static_cast<uint8_t>(left);
        s.right = static_cast<uint8_t>(right);
        s.out = static_cast<uint8_t>(out);
        s.flags = static_cast<uint8_t>(flags);
        s.scale = static_cast<float>((flags & kLastStep ? 1.0 : scale[out]) /
                                     (scale[left] * scale[right]));
        s.diagonal = right == kC ? static_cast<float>(call->a * scale[out]) : 0.0f;
        s.sym_before = static_cast<uint16_t>(sym);
        s.full_before = static_cast<uint16_t>(full);
        ++(flags & kSymmetric ? sym : full);
    };
    int x = kX0;
    for (int done = 0; done < call->rounds;) {
        const int take = segments && call->rounds - done > 2 ? 2 : 1;
        add(x, x, kA, kSymmetric | kLeftX | kWithC);
        add(kA, kC, kP0, kSymmetric);
        if (take == 2) {
            add(kA, kP0, kZ, kSymmetric);
            add(kZ, kP0, kA, kSymmetric | kWithC);
            add(kA, kC, kP1, kSymmetric);
            add(kP1, kP0, kQ, kSymmetric);
        }
        done += take;
        add(take == 2 ? kQ : kP0, x, x ^ 1,
            kRightX | (done == call->rounds ? kLastStep : 0));
        x ^= 1;
    }
}

constexpr int32_t kSegmentSide = 512;   // the shortest side for rounds in twos
constexpr double kTileUs[3] = {0.61, 0.76, 1.08}, kLevelUs[3] = {3.2, 4.2, 7.1};
// About how many microseconds the steps take: a tile's 64 of k kTileUs (a 256 x 256 tile
// takes a pair 1.08: it copies half as much per product), and a step its longest tile and
// kLevelUs from the last results to the next products, or the tiles' share per SM; within
// 3 to 7% of 17 lists measured with each tile and grouping.  So the larger tile is taken
// where there are enough of them for all pairs (12 matrices of 1024 x 1024 take 679 us with
// it and 803 and 1179 with the smaller ones, 4 of them 375, 308 and 396, one 347, 249 and
// 205), and rounds in twos for long matrices (1024 x 4096 403 us and 488 without,
// 2048 x 8192 1167 and 1540; but 4 of 1024 x 1024 322 and 308).
double steps_cost(const MatrixTable& t, const MatrixCall& call, int shape, int sms) {
    const int64_t high = kMatrixTiles[shape][0], wide = kMatrixTiles[shape][1];
    const double each = kTileUs[shape], units = static_cast<double>(sms / (high / 128));
    double total = 0.0;
    for (int s = 0; s < call.steps; ++s) {
        double work = 0.0, longest = 0.0;
        const int flags = call.step[s].flags;
        for (int j = 0; j < t.count; ++j) {
            const int64_t mp = padded(t.item[j].m, high), np = padded(t.item[j].n, wide);
            const double side = static_cast<double>(mp / high);
            const double k = each * static_cast<double>((flags & kLeftX ? np : mp) / 64);
            work += k * (flags & kSymmetric
                             ? side * (side + 1) / 2 * static_cast<double>(high / wide)
                             : side * static_cast<double>(np / wide));
            longest = std::max(longest, k);
        }
        total += std::max(work / units + longest / 3, longest + kLevelUs[shape]);
    }
    return total;
}

// Tiles, workspace and the launches' bounds.
void lay_out(MatrixTable* t, MatrixCall* call, char* ws) {
    const int sms = device_sms();
    double best = 0.0;
    bool segments = false;
    int32_t shortest = INT32_MAX;
    for (int j = 0; j < t->count; ++j) shortest = std::min(shortest, t->item[j].m);
    for (const bool split : {false, true}) {
        if (split && shortest < kSegmentSide) continue;
        plan_steps(call, split);
        for (int shape = 0; shape < 3; ++shape) {
            const double cost = steps_cost(*t, *call, shape, sms);
            if ((split || shape) && cost >= best) continue;
            best = cost;
            segments = split;
            t->shape = shape;
        }
    }
    plan_steps(call, segments);
    t->twos = segments;
    const int64_t high = kMatrixTiles[t->shape][0], across = kMatrixTiles[t->shape][1];
    // the longest tiles first, so that the last ones to end are short
    std::sort(t->item, t->item + t->count, [](const MatrixItem& a, const MatrixItem& b) {
        return a.m != b.m ? a.m > b.m : a.n > b.n;
    });
    uint32_t sym = 0, full = 0, part = 0, image = 0;
    for (int j = 0; j < t->count; ++j) {
        MatrixItem& x = t->item[j];
        x.mp = static_cast<int32_t>(padded(x.m, high));
        x.np = static_cast<int32_t>(padded(x.n, across));
        const int64_t wide = 4 * static_cast<int64_t>(x.mp) * x.np;
        const int64_t square = 4 * static_cast<int64_t>(x.mp) * x.mp;
        x.image[kX0] = ws;
        x.image[kX1] = ws + wide;
        for (int i = kA; i < kImages; ++i) x.image[i] = ws + 2 * wide + (i - kA) * square;
        x.part = reinterpret_cast<double*>(ws + 2 * wide + (kImages - kA) * square);
        x.tiles_done = reinterpret_cast<unsigned int*>(x.part + kMatrixParts);
        ws += matrix_bytes(x.m, x.n);
        t->sym0[j] = sym;
        t->full0[j] = full;
        t->part0[j] = part;
        t->image0[j] = image;
        const uint32_t side = static_cast<uint32_t>(x.mp / high);
        sym += side * (side + 1) / 2 * static_cast<uint32_t>(high / across);
        full += side * static_cast<uint32_t>(x.np / across);
        part += static_cast<uint32_t>(std::min<int64_t>(
            kMatrixParts, (static_cast<int64_t>(x.m) * x.n + 4095) / 4096));
        image += static_cast<uint32_t>(x.mp / 128) * (x.np / 64);
    }
    t->sym0[t->count] = sym;
    t->full0[t->count] = full;
    t->part0[t->count] = part;
    t->image0[t->count] = image;
    call->tiles = call->most = 0;
    for (int k = 0; k < call->steps; ++k) {
        MatrixStep& s = call->step[k];
        const uint32_t tiles = s.flags & kSymmetric ? sym : full;
        s.first = call->tiles;
        call->tiles += tiles;
        call->most = std::max(call->most, tiles);
    }
}

template <typename S, typename F>
int run_groups(const S& sides, const F& item, int32_t n, MatrixCall* call, int grad_dtype,
               void* workspace, const char* what, cudaStream_t stream) {
    std::unique_ptr<MatrixTable> t(new MatrixTable);
    for (int32_t at = 0; at < n;) {
        int64_t bytes;
        const int32_t end = group_end(sides, n, at, &bytes);
        if (take_group(item, at, end, t.get())) {
            lay_out(t.get(), call, static_cast<char*>(workspace));
            const cudaError_t e = launch_matrices(*t, *call, grad_dtype, stream);
            if (e != cudaSuccess) return cuda_fail(what, e);
            record_kernel("matrix_rounds<%d, %d>%s", kMatrixTiles[t->shape][0],
                          kMatrixTiles[t->shape][1], t->twos ? ", rounds in twos" : "");
        }
        at = end;
    }
    return SHARDSTEP_OK;
}

int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
    if (need > 0 && workspace == nullptr)
        return ready_fail(SHARDSTEP_ERR_INVALID, "workspace is NULL");
    if (!aligned(workspace, 16)) return ready_fail(SHARDSTEP_ERR_INVALID, "workspace misaligned");
    if (bytes < need)
        return ready_fail(SHARDSTEP_ERR_INVALID, "the workspace needs %lld bytes, got %lld",
                          static_cast<long long>(need), static_cast<long long>(bytes));
    return SHARDSTEP_OK;
}

}  // namespace
}  // namespace shardstep

using namespace shardstep;

extern "C" {

int token_embedding(const void* table, int64_t table_stride, int32_t dtype, int64_t vocab,
                    int64_t dim, const void* ids, int32_t id_bytes, int64_t n, float scale,
                    void* out, int64_t out_stride, void* stream) {
    const int es = elem_size(dtype);
    if (int rc = check_embedding(table, table_stride, vocab, dim, ids, id_bytes, n, scale, out,
                                 out_stride, es, es);
        rc != SHARDSTEP_OK)
        return rc;
    if (n == 0) return ready_ok();
    FewRanges reads, writes;
    reads.add(table, span(vocab, dim, table_stride, es));
    reads.add(ids, n * id_bytes);
    writes.add(out, span(n, dim, out_stride, es));
    if (int rc = check_ranges(reads, writes); rc != SHARDSTEP_OK) return rc;
    EmbedArgs a{};
    a.table = const_cast<void*>(table);
    a.table_stride = table_stride;
    a.rows = out;
    a.row_stride = out_stride;
    a.ids = ids;
    a.ids64 = id_bytes == 8;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.scale = scale;
    const bool vec = rows_aligned(table, table_stride, vocab, es) &&
                     rows_aligned(out, out_stride, n, es) && dim * es % 16 == 0;
    const cudaError_t e = launch_embedding(a, dtype, vec, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("embedding", e);
    record_kernel("embedding_lookup<%s> (%s)", dtype_name(dtype), vec ? "vectors" : "elements");
    return ready_ok();
}

int64_t token_embedding_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
    if (!embed_sizes(n, vocab, dim)) return -1;
    return 2 * round16(4 * n) + round16(4 * (vocab + 1)) +
           8 * dim * embed_plan(n, dim).chunks;
}

int token_embedding_grad(const void* d_out, int64_t d_out_stride, int32_t dtype, const void* ids,
                         int32_t id_bytes, int64_t n, float scale, void* grad,
                         int64_t grad_stride, int32_t grad_dtype, int64_t vocab, int64_t dim,
                         int32_t accumulate, void* workspace, int64_t workspace_bytes,
                         void* stream) {
    const int es = elem_size(dtype), gs = elem_size(grad_dtype);
    if (int rc = check_embedding(grad, grad_stride, vocab, dim, ids, id_bytes, n, scale, d_out,
                                 d_out_stride, gs, es);
        rc != SHARDSTEP_OK)
        return rc;
    const int64_t need = token_embedding_grad_workspace_bytes(n, vocab, dim);
    if (int rc = check_workspace(workspace, workspace_bytes, need); rc != SHARDSTEP_OK) return rc;
    if (n == 0 && accumulate) return ready_ok();
    FewRanges reads, writes;
    reads.add(d_out, span(n, dim, d_out_stride, es));
    reads.add(ids, n * id_bytes);
    writes.add(grad, span(vocab, dim, grad_stride, gs));
    writes.add(workspace, need);
    if (int rc = check_ranges(reads, writes); rc != SHARDSTEP_OK) return rc;
    EmbedArgs a{};
    a.table = grad;
    a.table_stride = grad_stride;
    a.rows = const_cast<void*>(d_out);
    a.row_stride = d_out_stride;
    a.ids = ids;
    a.ids64 = id_bytes == 8;
    a.accumulate = accumulate != 0;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.scale = scale;
    const EmbedPlan plan = embed_plan(n, dim);
    char* ws = static_cast<char*>(workspace);
    EmbedSort s{};
    s.token = reinterpret_cast<int32_t*>(ws);
    s.id = reinterpret_cast<int32_t*>(ws += round16(4 * n));
    s.row_start = reinterpret_cast<uint32_t*>(ws += round16(4 * n));
    s.piece = reinterpret_cast<float*>(ws + round16(4 * (vocab + 1)));
    s.chunk = plan.chunk;
    s.chunks = plan.chunks;
    // blocks of the sums, if every slice is of 256 single columns, and of the zeros
    if (plan.chunks * ((dim + 255) / 256) + vocab / kEmbedZeroRows + 1 > INT32_MAX)
        return ready_fail(SHARDSTEP_ERR_INVALID, "n x dim or vocab too large for one launch");
    // a vector of d_out stands over as many elements of grad
    const int per = 16 / es;
    const int at_grad = std::min(16, per * gs);
    const bool vec = rows_aligned(d_out, d_out_stride, n, es) && dim % per == 0 &&
                     aligned(grad, at_grad) && (vocab == 1 || grad_stride * gs % at_grad == 0);
    const cudaError_t e = launch_embedding_grad(a, s, dtype, grad_dtype, vec,
                                                static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("embedding gradient", e);
    record_kernel("embedding_sum<%s, %s> (%s)", dtype_name(dtype), dtype_name(grad_dtype),
                  vec ? "vectors" : "elements");
    return ready_ok();
}

// ------------------------------------------------------------- layer norm

int rows_layer_norm(const void* x, int64_t x_stride, int32_t dtype, int64_t rows, int64_t cols,
                    const void* weight, const void* bias, int32_t weight_dtype, float eps,
                    void* out, int64_t out_stride, float* mean, float* rstd, void* stream) {
    const int es = elem_size(dtype), ws = elem_size(weight_dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype %d", dtype);
    if (weight_dtype != dtype && weight_dtype != SHARDSTEP_DTYPE_F32)
        return ready_fail(SHARDSTEP_ERR_INVALID, "weight_dtype must be dtype or fp32");
    if (rows < 0 || rows > (int64_t{1} << 32) || cols < 1 || cols > (int64_t{1} << 24))
        return ready_fail(SHARDSTEP_ERR_INVALID, "rows or cols out of range");
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return ready_fail(SHARDSTEP_ERR_INVALID, "eps must be finite and >= 0");
    if (!stride_ok(x_stride, rows, cols) || !stride_ok(out_stride, rows, cols))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a row stride is out of range");
    if (rows == 0) return ready_ok();
    if (!x || !out || !mean || !rstd) return ready_fail(SHARDSTEP_ERR_INVALID, "a NULL array");
    if (!aligned(x, es) || !aligned(out, es) || !aligned(weight, ws) || !aligned(bias, ws) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an array is misaligned");
    FewRanges reads, writes;
    reads.add(x, span(rows, cols, x_stride, es));
    reads.add(weight, weight ? cols * ws : 0);
    reads.add(bias, bias ? cols * ws : 0);
    writes.add(out, span(rows, cols, out_stride, es));
    writes.add(mean, rows * 4);
    writes.add(rstd, rows * 4);
    if (int rc = check_ranges(reads, writes); rc != SHARDSTEP_OK) return rc;
    const NormRows a{x, x_stride, out, out_stride, weight, bias, mean, rstd, rows, cols, eps};
    const bool vec =
        rows_aligned(x, x_stride, rows, es) && aligned(weight, 16) && aligned(bias, 16);
    const bool whole = rows_aligned(out, out_stride, rows, es);
    const cudaError_t e = launch_layer_norm(a, dtype, weight_dtype, vec, whole,
                                            static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("layer norm", e);
    record_kernel("%s <%s>", layer_norm_kernel(cols, dtype, vec, whole), dtype_name(dtype));
    return ready_ok();
}

int64_t rows_layer_norm_workspace_bytes(int64_t cols) {
    if (cols < 1 || cols > (int64_t{1} << 24)) return -1;
    return 8 * ((cols + 7) / 8 * 8) * kNormPieces;
}

int rows_layer_norm_grad(const void* d_out, int64_t d_out_stride, const void* x,
                         int64_t x_stride, int32_t dtype, int64_t rows, int64_t cols,
                         const float* mean, const float* rstd, const void* weight,
                         int32_t weight_dtype, void* d_x, int64_t d_x_stride, void* d_weight,
                         void* d_bias, int32_t accumulate, void* workspace,
                         int64_t workspace_bytes, void* stream) {
    const int es = elem_size(dtype), ws = elem_size(weight_dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype %d", dtype);
    if (weight_dtype != dtype && weight_dtype != SHARDSTEP_DTYPE_F32)
        return ready_fail(SHARDSTEP_ERR_INVALID, "weight_dtype must be dtype or fp32");
    if (rows < 0 || rows > (int64_t{1} << 32) || cols < 1 || cols > (int64_t{1} << 24))
        return ready_fail(SHARDSTEP_ERR_INVALID, "rows or cols out of range");
    if (!stride_ok(x_stride, rows, cols) || !stride_ok(d_out_stride, rows, cols) ||
        (d_x && !stride_ok(d_x_stride, rows, cols)))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a row stride is out of range");
    const bool columns = d_weight != nullptr || d_bias != nullptr;
    const int64_t need = columns ? rows_layer_norm_workspace_bytes(cols) : 0;
    if (rows > 0 && (!x || !d_out || !mean || !rstd))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a NULL array");
    if (!aligned(x, es) || !aligned(d_out, es) || !aligned(d_x, es) || !aligned(weight, ws) ||
        !aligned(d_weight, ws) || !aligned(d_bias, ws) || !aligned(mean, 4) || !aligned(rstd, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an array is misaligned");
    if (int rc = check_workspace(workspace, workspace_bytes, need); rc != SHARDSTEP_OK) return rc;
    if (!columns && (rows == 0 || d_x == nullptr)) return ready_ok();
    if (rows == 0 && accumulate) return ready_ok();
    FewRanges reads, writes;
    reads.add(x, span(rows, cols, x_stride, es));
    reads.add(d_out, span(rows, cols, d_out_stride, es));
    reads.add(weight, weight ? cols * ws : 0);
    reads.add(mean, rows * 4);
    reads.add(rstd, rows * 4);
    writes.add(d_x, d_x ? span(rows, cols, d_x_stride, es) : 0);
    writes.add(d_weight, d_weight ? cols * ws : 0);
    writes.add(d_bias, d_bias ? cols * ws : 0);
    writes.add(workspace, need);
    if (int rc = check_ranges(reads, writes); rc != SHARDSTEP_OK) return rc;
    const NormGradRows a{x,    x_stride, d_out, d_out_stride,
                         d_x,  d_x_stride, weight, mean, rstd,
                         columns ? static_cast<float*>(workspace) : nullptr, rows, cols,
                         (cols + 7) / 8 * 8};
    const bool vec = rows_aligned(x, x_stride, rows, es) &&
                     rows_aligned(d_out, d_out_stride, rows, es) && aligned(weight, 16);
    const bool whole = d_x == nullptr || rows_aligned(d_x, d_x_stride, rows, es);
    const cudaError_t e =
        launch_layer_norm_grad(a, dtype, weight_dtype, d_weight, d_bias, accumulate != 0, vec,
                               whole, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("layer norm gradient", e);
    record_kernel("%s <%s>", layer_norm_grad_kernel(a, dtype, vec, whole), dtype_name(dtype));
    return ready_ok();
}

// --------------------------------------------------------------- matrices

int64_t matrices_workspace_bytes(const int64_t* rows, const int64_t* cols, int32_t n) {
    if (n < 0 || (n > 0 && (!rows || !cols))) return -1;
    for (int32_t i = 0; i < n; ++i)
        if (!side_ok(rows[i]) || !side_ok(cols[i])) return -1;
    return workspace_for([&](int32_t i) { return Sides{rows[i], cols[i]}; }, n);
}

int matrices_orthogonalize(const void* const* in, void* const* out, const int64_t* rows,
                           const int64_t* cols, int32_t n, int32_t in_dtype, int32_t out_dtype,
                           const shardstep_quintic_t* quintic, void* workspace,
                           int64_t workspace_bytes, void* stream) try {
    const int es = elem_size(in_dtype), os = elem_size(out_dtype);
    if (es == 0 || os == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype");
    if (n < 0) return ready_fail(SHARDSTEP_ERR_INVALID, "n must be >= 0");
    MatrixCall call{};
    if (int rc = take_quintic(quintic, &call); rc != SHARDSTEP_OK) return rc;
    call.out_type = out_dtype;
    if (n == 0) return ready_ok();
    if (!in || !out || !rows || !cols) return ready_fail(SHARDSTEP_ERR_INVALID, "a NULL array");
    std::vector<Range> reads, writes;
    reads.reserve(n);
    writes.reserve(n + 1);
    for (int32_t i = 0; i < n; ++i) {
        if (!side_ok(rows[i]) || !side_ok(cols[i]))
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: a side is out of range", i);
        const int64_t numel = rows[i] * cols[i];
        if (numel == 0) continue;
        if (!in[i] || !out[i] || !aligned(in[i], es) || !aligned(out[i], os))
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: NULL or misaligned", i);
        add_range(reads, in[i], numel * es);
        add_range(writes, out[i], numel * os);
    }
    const auto sides = [&](int32_t i) { return Sides{rows[i], cols[i]}; };
    const int64_t need = workspace_for(sides, n);
    if (int rc = check_workspace(workspace, workspace_bytes, need); rc != SHARDSTEP_OK) return rc;
    add_range(writes, workspace, need);
    if (int rc = check_ranges(&reads, &writes); rc != SHARDSTEP_OK) return rc;
    const auto item = [&](int32_t i, MatrixItem* x, int64_t* r, int64_t* c) {
        x->grad = in[i];
        x->out = out[i];
        *r = rows[i];
        *c = cols[i];
    };
    if (int rc = run_groups(sides, item, n, &call, in_dtype, workspace, "orthogonalize",
                            static_cast<cudaStream_t>(stream));
        rc != SHARDSTEP_OK)
        return rc;
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

int tensors_muon_step(const shardstep_matrix_t* ms, int32_t n, int32_t grad_dtype,
                      int32_t param_dtype, const shardstep_muon_t* hp, int32_t n_groups,
                      const shardstep_quintic_t* quintic, const float* grad_coef,
                      const uint32_t* skip, void* workspace, int64_t workspace_bytes,
                      void* stream) try {
    const int es = elem_size(grad_dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown grad dtype %d", grad_dtype);
    if (param_dtype != SHARDSTEP_DTYPE_BF16 && param_dtype != SHARDSTEP_DTYPE_F16)
        return ready_fail(SHARDSTEP_ERR_INVALID, "param dtype %d is not bf16 or fp16",
                          param_dtype);
    if (n < 0) return ready_fail(SHARDSTEP_ERR_INVALID, "n must be >= 0");
    if (n_groups < 1) return ready_fail(SHARDSTEP_ERR_INVALID, "n_groups must be >= 1");
    if (n_groups > kMaxGroups)
        return ready_fail(SHARDSTEP_ERR_CAPACITY, "n_groups %d > %d", n_groups, kMaxGroups);
    if (hp == nullptr) return ready_fail(SHARDSTEP_ERR_INVALID, "hp is NULL");
    if (grad_coef && !aligned(grad_coef, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "grad_coef misaligned");
    if (skip && !aligned(skip, 4)) return ready_fail(SHARDSTEP_ERR_INVALID, "skip misaligned");
    MatrixCall call{};
    if (int rc = take_quintic(quintic, &call); rc != SHARDSTEP_OK) return rc;
    call.out_type = param_dtype;
    call.coef = grad_coef;
    call.skip = skip;
    for (int32_t g = 0; g < n_groups; ++g) {
        const shardstep_muon_t& h = hp[g];
        if (!std::isfinite(h.lr) || !std::isfinite(h.weight_decay) ||
            !(h.momentum >= 0 && h.momentum < 1) || !(h.match_rms >= 0) ||
            !std::isfinite(h.match_rms))
            return ready_fail(SHARDSTEP_ERR_INVALID, "hp[%d]: a value is out of range", g);
        call.group[g] = MatrixGroup{static_cast<float>(h.lr * h.weight_decay),
                                    static_cast<float>(h.momentum),
                                    static_cast<float>(1 - h.momentum), h.nesterov != 0};
    }
    if (n == 0) return ready_ok();
    if (ms == nullptr) return ready_fail(SHARDSTEP_ERR_INVALID, "matrices is NULL");
    std::vector<Range> reads, writes;
    reads.reserve(n + 2);
    writes.reserve(3 * static_cast<size_t>(n) + 1);
    add_range(reads, grad_coef, grad_coef ? 4 : 0);
    add_range(reads, skip, skip ? 4 : 0);
    for (int32_t i = 0; i < n; ++i) {
        const shardstep_matrix_t& t = ms[i];
        if (!side_ok(t.rows) || !side_ok(t.cols))
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: a side is out of range", i);
        if (t.group < 0 || t.group >= n_groups)
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: group %d out of range", i,
                              t.group);
        const int64_t numel = t.rows * t.cols;
        if (numel == 0) continue;
        if (!t.grad || !t.master || !t.m)
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: a NULL array", i);
        if (!aligned(t.grad, es) || !aligned(t.master, 4) || !aligned(t.m, 4) ||
            !aligned(t.param, 2))
            return ready_fail(SHARDSTEP_ERR_INVALID, "matrix %d: an array misaligned", i);
        add_range(reads, t.grad, numel * es);
        add_range(writes, t.master, numel * 4);
        add_range(writes, t.m, numel * 4);
        add_range(writes, t.param, t.param ? numel * 2 : 0);
    }
    const auto sides = [&](int32_t i) { return Sides{ms[i].rows, ms[i].cols}; };
    const int64_t need = workspace_for(sides, n);
    if (int rc = check_workspace(workspace, workspace_bytes, need); rc != SHARDSTEP_OK) return rc;
    add_range(writes, workspace, need);
    if (int rc = check_ranges(&reads, &writes); rc != SHARDSTEP_OK) return rc;
    const auto item = [&](int32_t i, MatrixItem* x, int64_t* r, int64_t* c) {
        const shardstep_matrix_t& t = ms[i];
        const shardstep_muon_t& h = hp[t.group];
        x->grad = t.grad;
        x->master = t.master;
        x->m_buf = t.m;
        x->out = t.param;
        x->group = static_cast<int16_t>(t.group);
        const double rows = static_cast<double>(t.rows), cols = static_cast<double>(t.cols);
        x->step = static_cast<float>(
            h.lr * (h.match_rms > 0 ? h.match_rms * std::sqrt(std::max(rows, cols))
                                    : std::sqrt(std::max(1.0, rows / std::max(cols, 1.0)))));
        *r = t.rows;
        *c = t.cols;
    };
    if (int rc = run_groups(sides, item, n, &call, grad_dtype, workspace, "muon step",
                            static_cast<cudaStream_t>(stream));
        rc != SHARDSTEP_OK)
        return rc;
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

}  // extern "C"
