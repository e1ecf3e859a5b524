// Host side of the losses over tokens (token_*) and of the entry points over
// lists of tensors (tensors_*): argument checks, the tables that travel with
// each launch, and dispatch.  Nothing here allocates device memory or keeps a
// pointer.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "internal.h"
#include "shardstep.h"

namespace shardstep {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int32_t dtype) {
    return dtype == SHARDSTEP_DTYPE_F32                                        ? 4
           : dtype == SHARDSTEP_DTYPE_BF16 || dtype == SHARDSTEP_DTYPE_F16 ? 2
                                                                               : 0;
}
const char* dtype_name(int dtype) {
    return dtype == SHARDSTEP_DTYPE_F32 ? "f32" : dtype == SHARDSTEP_DTYPE_F16 ? "f16" : "bf16";
}

struct Range {
    uintptr_t lo, hi;
};
void add_range(std::vector<Range>& v, const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0) v.push_back(Range{a, a + static_cast<uintptr_t>(bytes)});
}
void sort_ranges(std::vector<Range>& v) {
    const auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
}
// Whether any two of the sorted ranges share a byte.
bool self_overlap(const std::vector<Range>& v) {
    for (size_t k = 1; k < v.size(); ++k)
        if (v[k].lo < v[k - 1].hi) return true;
    return false;
}
// Whether a range of `reads` shares a byte with one of `writes` (both sorted;
// the writes disjoint).
bool cross_overlap(const std::vector<Range>& reads, const std::vector<Range>& writes) {
    size_t w = 0;
    for (const Range& r : reads) {
        while (w < writes.size() && writes[w].hi <= r.lo) ++w;
        if (w < writes.size() && writes[w].lo < r.hi) return true;
    }
    return false;
}

// The scalars of every group, from the host's hyper-parameters or from the
// device-resident step states.
int take_groups(const shardstep_adamw_t* hp, const shardstep_adamw_state_t* const* states,
                bool on_device, int32_t n_groups, GroupScalars* gs) {
    if (n_groups < 1) return ready_fail(SHARDSTEP_ERR_INVALID, "n_groups must be >= 1");
    if (n_groups > kMaxGroups)
        return ready_fail(SHARDSTEP_ERR_CAPACITY, "n_groups %d > %d", n_groups, kMaxGroups);
    if (on_device ? states == nullptr : hp == nullptr)
        return ready_fail(SHARDSTEP_ERR_INVALID, on_device ? "states is NULL" : "hp is NULL");
    for (int32_t g = 0; g < n_groups; ++g) {
        AdamScalars& c = gs->c[g];
        if (on_device) {
            if (states[g] == nullptr || !aligned(states[g], 8))
                return ready_fail(SHARDSTEP_ERR_INVALID, "states[%d] is NULL or misaligned", g);
            c = AdamScalars{};
            c.dev = reinterpret_cast<const float*>(reinterpret_cast<const char*>(states[g]) +
                                                   offsetof(shardstep_adamw_state_t, scalars));
        } else {
            if (hp[g].step < 1)
                return ready_fail(SHARDSTEP_ERR_INVALID, "hp[%d].step must be >= 1", g);
            // groups that differ only in lr and decay are the rule: the beta
            // powers' running products are the same ones then
            c = host_adam_scalars(hp[g]);
            gs->inv_sqrt_bc2[g] = 1.0f / c.sqrt_bc2;
        }
    }
    return SHARDSTEP_OK;
}

// `reads`: the words and states that the step reads besides the gradients.
int check_tensors(const void* const* grads, const shardstep_tensor_t* ts, int32_t n, int gs,
                  int bits, int32_t n_groups, std::vector<Range> reads) {
    std::vector<Range> writes;
    reads.reserve(reads.size() + n);
    writes.reserve(static_cast<size_t>(n) * (bits == 8 ? 6 : 4));
    const int ms = bits == 8 ? 1 : 4;
    for (int32_t i = 0; i < n; ++i) {
        const shardstep_tensor_t& t = ts[i];
        if (t.numel < 0) return ready_fail(SHARDSTEP_ERR_INVALID, "tensor %d: numel < 0", i);
        if (t.group < 0 || t.group >= n_groups)
            return ready_fail(SHARDSTEP_ERR_INVALID, "tensor %d: group %d out of range", i,
                              t.group);
        if (t.numel == 0) continue;
        if (t.numel > (int64_t{1} << 40))
            return ready_fail(SHARDSTEP_ERR_INVALID, "tensor %d: too large", i);
        if (!grads[i] || !t.master || !t.m || !t.v || (bits == 8 && (!t.m_scale || !t.v_scale)))
            return ready_fail(SHARDSTEP_ERR_INVALID, "tensor %d: a NULL array", i);
        if (!aligned(grads[i], gs) || !aligned(t.master, 4) || !aligned(t.m, ms) ||
            !aligned(t.v, ms) || (t.param && !aligned(t.param, 2)) ||
            (bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
            return ready_fail(SHARDSTEP_ERR_INVALID, "tensor %d: an array misaligned", i);
        add_range(reads, grads[i], t.numel * gs);
        add_range(writes, t.master, t.numel * 4);
        add_range(writes, t.m, t.numel * ms);
        add_range(writes, t.v, t.numel * ms);
        if (t.param) add_range(writes, t.param, t.numel * 2);
        if (bits == 8) {
            const int64_t blocks = (t.numel + kMomentBlock - 1) / kMomentBlock;
            add_range(writes, t.m_scale, blocks * 4);
            add_range(writes, t.v_scale, blocks * 4);
        }
    }
    sort_ranges(reads);
    sort_ranges(writes);
    if (self_overlap(writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "two of the tensors' outputs overlap");
    if (cross_overlap(reads, writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an input overlaps an output");
    return SHARDSTEP_OK;
}

bool tensor_vec(const void* grad, const shardstep_tensor_t& t, int bits) {
    return aligned(grad, 16) && aligned(t.master, 16) && aligned(t.m, bits == 8 ? 8 : 16) &&
           aligned(t.v, bits == 8 ? 8 : 16) && (t.param == nullptr || aligned(t.param, 16));
}

constexpr uint32_t kMaxLaunchBlocks = 0x7FFFFFFFu;

// Launches tensors [at, ...) as far as the table and the grid go; *at moves on.
template <int CAP>
int launch_some(const void* const* grads, const shardstep_tensor_t* ts, int32_t n, int32_t* at,
                int grad_type, int param_type, int bits, const GroupScalars& gs, const float* coef,
                const uint32_t* skip, cudaStream_t stream) {
    std::unique_ptr<TensorTable<CAP>> tab(new TensorTable<CAP>);
    const int64_t chunk = bits == 8 ? kListChunk8 : kListChunk32;
    int k = 0;
    uint64_t blocks = 0;
    int32_t i = *at;
    for (; i < n && k < CAP; ++i) {
        const shardstep_tensor_t& t = ts[i];
        if (t.numel == 0) continue;
        const uint64_t b = static_cast<uint64_t>((t.numel + chunk - 1) / chunk);
        if (blocks + b > kMaxLaunchBlocks) break;
        tab->grad[k] = grads[i];
        tab->master[k] = t.master;
        tab->m[k] = t.m;
        tab->v[k] = t.v;
        tab->m_scale[k] = t.m_scale;
        tab->v_scale[k] = t.v_scale;
        tab->param[k] = t.param;
        tab->n[k] = t.numel;
        tab->b0[k] = static_cast<uint32_t>(blocks);
        tab->group[k] = static_cast<uint16_t>(t.group);
        tab->vec[k] = tensor_vec(grads[i], t, bits);
        blocks += b;
        ++k;
    }
    *at = i;
    if (k == 0) return SHARDSTEP_OK;
    tab->b0[k] = static_cast<uint32_t>(blocks);
    tab->count = k;
    tab->near_shift = 0;
    while ((blocks - 1) >> tab->near_shift >= kNear) ++tab->near_shift;
    for (int r = 0, at_tensor = 0; r <= kNear; ++r) {
        const uint64_t b = static_cast<uint64_t>(r) << tab->near_shift;
        while (at_tensor < k - 1 && b >= tab->b0[at_tensor + 1]) ++at_tensor;
        tab->near[r] = static_cast<uint16_t>(at_tensor);
    }
    const cudaError_t e =
        launch_tensors_adamw<CAP>(*tab, grad_type, param_type, bits, gs, coef, skip, stream);
    if (e != cudaSuccess)
        return ready_fail(SHARDSTEP_ERR_CUDA, "tensors_adamw launch: %s", cudaGetErrorString(e));
    record_kernel("tensors_adamw%d<%d tensors, %s>", bits, CAP, dtype_name(grad_type));
    return SHARDSTEP_OK;
}

int adamw_step(const void* const* grads, const shardstep_tensor_t* ts, int32_t n,
               int32_t grad_dtype, int32_t param_dtype, int32_t bits, const shardstep_adamw_t* hp,
               const shardstep_adamw_state_t* const* states, bool on_device, int32_t n_groups,
               const float* coef, const uint32_t* skip, void* stream) try {
    const int es = elem_size(grad_dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown grad dtype %d", grad_dtype);
    if (param_dtype != SHARDSTEP_DTYPE_BF16 && param_dtype != SHARDSTEP_DTYPE_F16)
        return ready_fail(SHARDSTEP_ERR_INVALID, "param dtype %d is not bf16 or fp16",
                          param_dtype);
    if (bits != 8 && bits != 32)
        return ready_fail(SHARDSTEP_ERR_INVALID, "state_bits must be 8 or 32 (got %d)", bits);
    if (n < 0) return ready_fail(SHARDSTEP_ERR_INVALID, "n must be >= 0");
    if (coef && !aligned(coef, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "grad_coef misaligned");
    if (skip && !aligned(skip, 4)) return ready_fail(SHARDSTEP_ERR_INVALID, "skip misaligned");
    GroupScalars gs{};
    gs.neg_zero = -0.0f;
    if (int rc = take_groups(hp, states, on_device, n_groups, &gs); rc != SHARDSTEP_OK) return rc;
    if (n == 0) return ready_ok();
    if (ts == nullptr || grads == nullptr)
        return ready_fail(SHARDSTEP_ERR_INVALID, "tensors / grads is NULL");
    std::vector<Range> reads;
    add_range(reads, coef, coef ? 4 : 0);
    add_range(reads, skip, skip ? 4 : 0);
    for (int32_t g = 0; on_device && g < n_groups; ++g)
        add_range(reads, states[g], sizeof(shardstep_adamw_state_t));
    if (int rc = check_tensors(grads, ts, n, es, bits, n_groups, std::move(reads));
        rc != SHARDSTEP_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int32_t at = 0; at < n;) {
        const int rc = n - at <= kTensorsSmall
                           ? launch_some<kTensorsSmall>(grads, ts, n, &at, grad_dtype, param_dtype,
                                                        bits, gs, coef, skip, s)
                           : launch_some<kTensorsLarge>(grads, ts, n, &at, grad_dtype, param_dtype,
                                                        bits, gs, coef, skip, s);
        if (rc != SHARDSTEP_OK) return rc;
    }
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

int check_moments(const void* m, const float* ms, const void* v, const float* vs, int64_t n,
                  const float* fm, const float* fv, bool codes_written) {
    if (!m || !ms || !v || !vs || !fm || !fv)
        return ready_fail(SHARDSTEP_ERR_INVALID, "a NULL array");
    if (!aligned(ms, 4) || !aligned(vs, 4) || !aligned(fm, 4) || !aligned(fv, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an array misaligned");
    const int64_t blocks = (n + kMomentBlock - 1) / kMomentBlock;
    std::vector<Range> codes, full;
    add_range(codes, m, n);
    add_range(codes, v, n);
    add_range(codes, ms, blocks * 4);
    add_range(codes, vs, blocks * 4);
    add_range(full, fm, n * 4);
    add_range(full, fv, n * 4);
    sort_ranges(codes);
    sort_ranges(full);
    std::vector<Range>& writes = codes_written ? codes : full;
    if (self_overlap(writes) || cross_overlap(codes_written ? full : codes, writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "the arrays overlap");
    return SHARDSTEP_OK;
}

int moments(const uint8_t* m, const float* ms, const uint8_t* v, const float* vs, int64_t n,
            const float* fm, const float* fv, bool encode, void* stream) try {
    if (n < 0 || n > (int64_t{1} << 40))
        return ready_fail(SHARDSTEP_ERR_INVALID, "n out of range");
    if (n == 0) return ready_ok();
    if (int rc = check_moments(m, ms, v, vs, n, fm, fv, encode); rc != SHARDSTEP_OK) return rc;
    const bool vec = aligned(m, 8) && aligned(v, 8) && aligned(fm, 16) && aligned(fv, 16);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        encode ? launch_moments_encode(fm, fv, n, const_cast<uint8_t*>(m), const_cast<float*>(ms),
                                       const_cast<uint8_t*>(v), const_cast<float*>(vs), vec, s)
               : launch_moments_decode(m, ms, v, vs, n, const_cast<float*>(fm),
                                       const_cast<float*>(fv), vec, s);
    if (e != cudaSuccess)
        return ready_fail(SHARDSTEP_ERR_CUDA, "moments launch: %s", cudaGetErrorString(e));
    record_kernel(encode ? "moments_encode" : "moments_decode");
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

// One launch of the norm over tensors [at, ...); blocks is the call's grid.
template <int CAP>
int norm_some(const void* const* grads, const int64_t* numels, int32_t n, int32_t* at, int type,
              int es, NormArgs a, int blocks, cudaStream_t stream) {
    std::unique_ptr<NormTable<CAP>> tab(new NormTable<CAP>);
    int k = 0;
    uint64_t chunks = 0;
    int32_t i = *at;
    for (; i < n && k < CAP; ++i) {
        if (numels[i] == 0) continue;
        const uint64_t c = static_cast<uint64_t>((numels[i] + kNormChunk - 1) / kNormChunk);
        if (chunks + c > kMaxLaunchBlocks) break;
        tab->p[k] = grads[i];
        tab->n[k] = numels[i];
        tab->b0[k] = static_cast<uint32_t>(chunks);
        tab->vec[k] = aligned(grads[i], 16);
        chunks += c;
        ++k;
    }
    while (i < n && numels[i] == 0) ++i;
    *at = i;
    tab->b0[k] = static_cast<uint32_t>(chunks);
    tab->count = k;
    a.last = i >= n;
    const cudaError_t e = launch_tensors_norm<CAP>(*tab, type, a, blocks, stream);
    if (e != cudaSuccess)
        return ready_fail(SHARDSTEP_ERR_CUDA, "tensors_norm launch: %s", cudaGetErrorString(e));
    record_kernel("tensors_norm<%d tensors, %s>", CAP, dtype_name(type));
    return SHARDSTEP_OK;
}

// ---------------------------------------------------- losses over tokens

int64_t loss_words(int64_t n_tokens, int64_t n_pairs) { return 4 * n_tokens + 2 * n_pairs; }

// Whether every gradient row lies as far past a 16-byte boundary as its logits
// row, so that a row's staged bytes can be stored back in bulk.
bool same_offsets(const shardstep_token_loss_t* a) {
    const uint64_t off = reinterpret_cast<uintptr_t>(a->grad) -
                         reinterpret_cast<uintptr_t>(a->logits);
    const uint64_t step = (static_cast<uint64_t>(a->grad_stride) -
                           static_cast<uint64_t>(a->row_stride)) * elem_size(a->dtype);
    return off % 16 == 0 && step % 16 == 0;
}

// The per-token words of a workspace.
PreferenceArgs loss_words_at(void* workspace, int64_t tokens) {
    float* words = reinterpret_cast<float*>(static_cast<LossWork*>(workspace) + 1);
    PreferenceArgs p{};
    p.row_ref = words;
    p.row_sum = words + tokens;
    p.term = words + 2 * tokens;
    return p;
}

// The checks both losses share; fills the kernel arguments.
int take_tokens(const shardstep_token_loss_t* a, int64_t need, TokenArgs* k,
                std::vector<Range>* reads, std::vector<Range>* writes) {
    const int es = elem_size(a->dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype %d", a->dtype);
    if (a->id_bytes != 4 && a->id_bytes != 8)
        return ready_fail(SHARDSTEP_ERR_INVALID, "id_bytes must be 4 or 8");
    if (a->n_tokens < 0 || a->n_tokens > INT32_MAX)
        return ready_fail(SHARDSTEP_ERR_INVALID, "n_tokens out of range");
    if (a->vocab < 1 || a->vocab > (int64_t{1} << 28))   // a row's bytes fit 31 bits
        return ready_fail(SHARDSTEP_ERR_INVALID, "vocab out of range");
    if (!std::isfinite(a->grad_scale))
        return ready_fail(SHARDSTEP_ERR_INVALID, "grad_scale is not finite");
    if (!(a->norm >= 0.0f) || !std::isfinite(a->norm))
        return ready_fail(SHARDSTEP_ERR_INVALID, "norm must be finite and >= 0");
    if (a->n_tokens == 0) return SHARDSTEP_OK;
    const int64_t limit = (int64_t{1} << 60) / a->n_tokens;
    if (a->row_stride < a->vocab || a->row_stride > limit ||
        (a->grad && (a->grad_stride < a->vocab || a->grad_stride > limit)))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a row stride is out of range");
    if (!a->logits || !a->ids || !a->logps || !a->stats || !a->workspace)
        return ready_fail(SHARDSTEP_ERR_INVALID,
                          "logits / ids / logps / stats / workspace is NULL");
    if (!aligned(a->logits, es) || !aligned(a->ids, a->id_bytes) || !aligned(a->logps, 4) ||
        !aligned(a->stats, 4) || !aligned(a->workspace, 8) || (a->grad && !aligned(a->grad, es)) ||
        (a->weights && !aligned(a->weights, 4)) || (a->ref_logps && !aligned(a->ref_logps, 4)) ||
        (a->loss_scale && !aligned(a->loss_scale, 4)))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an array is misaligned");
    if (a->workspace_bytes < need)
        return ready_fail(SHARDSTEP_ERR_INVALID, "the workspace needs %lld bytes, got %lld",
                          static_cast<long long>(need),
                          static_cast<long long>(a->workspace_bytes));
    const int64_t n = a->n_tokens;
    const bool in_place = a->grad == a->logits;
    if (in_place && a->grad_stride != a->row_stride)
        return ready_fail(SHARDSTEP_ERR_INVALID, "an in-place gradient needs the logits' stride");
    if (!in_place) add_range(*reads, a->logits, ((n - 1) * a->row_stride + a->vocab) * es);
    add_range(*reads, a->ids, n * a->id_bytes);
    add_range(*reads, a->weights, a->weights ? n * 4 : 0);
    add_range(*reads, a->ref_logps, a->ref_logps ? n * 4 : 0);
    add_range(*reads, a->loss_scale, a->loss_scale ? 4 : 0);
    add_range(*writes, a->logps, n * 4);
    add_range(*writes, a->grad, a->grad ? ((n - 1) * a->grad_stride + a->vocab) * es : 0);
    add_range(*writes, a->stats, 16);
    add_range(*writes, a->workspace, need);
    *k = TokenArgs{a->logits,  a->row_stride, a->grad,       a->grad_stride,
                   a->ids,     a->id_bytes == 8, a->weights, a->ref_logps,
                   a->logps,   n,             a->vocab,      a->grad_scale,
                   a->loss_scale, a->norm,    a->stats,      static_cast<LossWork*>(a->workspace)};
    return SHARDSTEP_OK;
}

int check_ranges(std::vector<Range>* reads, std::vector<Range>* writes) {
    sort_ranges(*reads);
    sort_ranges(*writes);
    if (self_overlap(*writes) || cross_overlap(*reads, *writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an output overlaps an input or another output");
    return SHARDSTEP_OK;
}

}  // namespace
}  // namespace shardstep

using namespace shardstep;

extern "C" {

int tensors_adamw_step(const void* const* grads, const shardstep_tensor_t* tensors, int32_t n,
                       int32_t grad_dtype, int32_t param_dtype, int32_t state_bits,
                       const shardstep_adamw_t* hp, int32_t n_groups, const float* grad_coef,
                       const uint32_t* skip, void* stream) {
    return adamw_step(grads, tensors, n, grad_dtype, param_dtype, state_bits, hp, nullptr, false,
                      n_groups, grad_coef, skip, stream);
}

int tensors_state_adamw_step(const void* const* grads, const shardstep_tensor_t* tensors,
                             int32_t n, int32_t grad_dtype, int32_t param_dtype,
                             int32_t state_bits, const shardstep_adamw_state_t* const* states,
                             int32_t n_groups, const float* grad_coef, const uint32_t* skip,
                             void* stream) {
    return adamw_step(grads, tensors, n, grad_dtype, param_dtype, state_bits, nullptr, states, true,
                      n_groups, grad_coef, skip, stream);
}

int tensors_moments_decode(const uint8_t* m, const float* m_scale, const uint8_t* v,
                           const float* v_scale, int64_t n, float* m_out, float* v_out,
                           void* stream) {
    return moments(m, m_scale, v, v_scale, n, m_out, v_out, false, stream);
}

int tensors_moments_encode(const float* m_in, const float* v_in, int64_t n, uint8_t* m,
                           float* m_scale, uint8_t* v, float* v_scale, void* stream) {
    return moments(m, m_scale, v, v_scale, n, m_in, v_in, true, stream);
}

int64_t tensors_norm_workspace_bytes(void) { return static_cast<int64_t>(sizeof(NormWork)); }

int tensors_grad_norm(const void* const* grads, const int64_t* numels, int32_t n, int32_t dtype,
                      float max_norm, const float* loss_scale, float* out, uint32_t* found_inf,
                      void* workspace, void* stream) try {
    const int es = elem_size(dtype);
    if (es == 0) return ready_fail(SHARDSTEP_ERR_INVALID, "unknown dtype %d", dtype);
    if (n < 0) return ready_fail(SHARDSTEP_ERR_INVALID, "n must be >= 0");
    if (!(max_norm > 0.0f)) return ready_fail(SHARDSTEP_ERR_INVALID, "max_norm must be > 0");
    if (!out || !workspace) return ready_fail(SHARDSTEP_ERR_INVALID, "out / workspace is NULL");
    if (!aligned(out, 4) || !aligned(workspace, 8) || (loss_scale && !aligned(loss_scale, 4)) ||
        (found_inf && !aligned(found_inf, 4)))
        return ready_fail(SHARDSTEP_ERR_INVALID, "a word or the workspace is misaligned");
    if (n > 0 && (!grads || !numels))
        return ready_fail(SHARDSTEP_ERR_INVALID, "grads / numels is NULL");
    uint64_t chunks = 0;
    std::vector<Range> reads, writes;
    reads.reserve(n);
    for (int32_t i = 0; i < n; ++i) {
        if (numels[i] < 0 || numels[i] > (int64_t{1} << 40))
            return ready_fail(SHARDSTEP_ERR_INVALID, "numels[%d] out of range", i);
        if (numels[i] == 0) continue;
        if (!grads[i] || !aligned(grads[i], es))
            return ready_fail(SHARDSTEP_ERR_INVALID, "grads[%d] is NULL or misaligned", i);
        chunks += static_cast<uint64_t>((numels[i] + kNormChunk - 1) / kNormChunk);
        add_range(reads, grads[i], numels[i] * es);
    }
    add_range(writes, out, 8);
    add_range(writes, workspace, sizeof(NormWork));
    if (found_inf) add_range(writes, found_inf, 4);
    if (loss_scale) add_range(reads, loss_scale, 4);
    sort_ranges(reads);
    sort_ranges(writes);
    if (self_overlap(writes) || cross_overlap(reads, writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an output overlaps an input or another output");
    NormArgs a{static_cast<NormWork*>(workspace), loss_scale, max_norm, out, found_inf, 1, 0};
    // four resident blocks per SM keep 64 KB or more of loads in flight on each
    const uint64_t most = std::min<uint64_t>(4 * static_cast<uint64_t>(device_sms()),
                                             kNormMaxBlocks);
    const int blocks = static_cast<int>(std::max<uint64_t>(1, std::min(chunks, most)));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t at = 0;
    do {
        const int rc = n - at <= kNormSmall
                           ? norm_some<kNormSmall>(grads, numels, n, &at, dtype, es, a, blocks, s)
                           : norm_some<kNormLarge>(grads, numels, n, &at, dtype, es, a, blocks, s);
        if (rc != SHARDSTEP_OK) return rc;
        a.first = 0;
    } while (at < n);
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

int64_t token_loss_workspace_bytes(int64_t n_tokens, int32_t n_pairs) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || n_pairs < 0) return -1;
    return static_cast<int64_t>(sizeof(LossWork)) + 4 * loss_words(n_tokens, n_pairs);
}

int token_policy_loss(const shardstep_token_loss_t* args, const float* old_logps,
                      const float* advantages, float clip_low, float clip_high, float kl_coef,
                      void* stream) try {
    if (args == nullptr) return ready_fail(SHARDSTEP_ERR_INVALID, "args is NULL");
    if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f) ||
        !std::isfinite(clip_high) || !(kl_coef >= 0.0f) || !std::isfinite(kl_coef))
        return ready_fail(SHARDSTEP_ERR_INVALID, "clip_low, clip_high or kl_coef out of range");
    // in one pass where a row fits an SM's shared memory; else forward, then backward
    const bool one_pass = args->vocab >= 1 && args->vocab <= (int64_t{1} << 28) &&
                          loss_row_fits(args->vocab, args->dtype) && same_offsets(args);
    const bool two_passes = args->grad != nullptr && !one_pass;
    const int64_t need = two_passes ? token_loss_workspace_bytes(args->n_tokens, 0)
                                    : static_cast<int64_t>(sizeof(LossWork));
    TokenArgs k{};
    std::vector<Range> reads, writes;
    if (int rc = take_tokens(args, need, &k, &reads, &writes); rc != SHARDSTEP_OK) return rc;
    if (args->n_tokens == 0) return ready_ok();
    if (!old_logps || !advantages || (kl_coef != 0.0f && !args->ref_logps))
        return ready_fail(SHARDSTEP_ERR_INVALID, "old_logps / advantages / ref_logps is NULL");
    if (!aligned(old_logps, 4) || !aligned(advantages, 4))
        return ready_fail(SHARDSTEP_ERR_INVALID, "old_logps / advantages misaligned");
    add_range(reads, old_logps, args->n_tokens * 4);
    add_range(reads, advantages, args->n_tokens * 4);
    if (int rc = check_ranges(&reads, &writes); rc != SHARDSTEP_OK) return rc;
    const PolicyArgs p{old_logps, advantages, 1.0f - clip_low, 1.0f + clip_high, kl_coef};
    const PreferenceArgs words =
        two_passes ? loss_words_at(args->workspace, k.n) : PreferenceArgs{};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t most = loss_rows_per_launch();
    cudaError_t e = cudaSuccess;
    for (int64_t row = 0; e == cudaSuccess && row < k.n; row += most) {
        const int64_t end = std::min(k.n, row + most);
        if (k.grad != nullptr && one_pass) {
            e = launch_policy_staged(k, p, row, end, args->dtype, s);
            continue;
        }
        e = launch_policy_forward(k, p, words, row, end, args->dtype, s);
        if (e == cudaSuccess && two_passes)
            e = launch_loss_backward(k, words, row, end, args->dtype, same_offsets(args), s);
    }
    if (e != cudaSuccess)
        return ready_fail(SHARDSTEP_ERR_CUDA, "policy loss launch: %s", cudaGetErrorString(e));
    record_kernel(k.grad == nullptr    ? "stream_forward<%s> (TMA-staged)"
                  : one_pass           ? "staged_rows<%s, policy> (TMA-staged)"
                  : same_offsets(args) ? "staged_rows<%s, backward> (TMA-staged)"
                                       : "offset_backward<%s>",
                  dtype_name(args->dtype));
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

int token_preference_loss(const shardstep_token_loss_t* args, const int64_t* seq_lens,
                          int32_t n_pairs, float beta, float label_smoothing, float* log_ratios,
                          void* stream) try {
    if (args == nullptr) return ready_fail(SHARDSTEP_ERR_INVALID, "args is NULL");
    if (n_pairs < 0 || n_pairs > (1 << 29))
        return ready_fail(SHARDSTEP_ERR_INVALID, "n_pairs out of range");
    if (!std::isfinite(beta) || !(label_smoothing >= 0.0f && label_smoothing <= 0.5f))
        return ready_fail(SHARDSTEP_ERR_INVALID, "beta or label_smoothing out of range");
    if (n_pairs > 0 && seq_lens == nullptr)
        return ready_fail(SHARDSTEP_ERR_INVALID, "seq_lens is NULL");
    int64_t tokens = 0;
    for (int64_t s = 0; s < 2 * static_cast<int64_t>(n_pairs); ++s) {
        if (seq_lens[s] < 0 || seq_lens[s] > INT32_MAX)
            return ready_fail(SHARDSTEP_ERR_INVALID, "seq_lens[%lld] out of range",
                              static_cast<long long>(s));
        tokens += seq_lens[s];
    }
    if (tokens != args->n_tokens)
        return ready_fail(SHARDSTEP_ERR_INVALID, "seq_lens add up to %lld of %lld tokens",
                          static_cast<long long>(tokens),
                          static_cast<long long>(args->n_tokens));
    const int64_t need = token_loss_workspace_bytes(tokens, n_pairs);
    TokenArgs k{};
    std::vector<Range> reads, writes;
    if (int rc = take_tokens(args, need, &k, &reads, &writes); rc != SHARDSTEP_OK) return rc;
    if (tokens == 0) return ready_ok();
    if (!args->ref_logps || !log_ratios)
        return ready_fail(SHARDSTEP_ERR_INVALID, "ref_logps / log_ratios is NULL");
    if (!aligned(log_ratios, 4)) return ready_fail(SHARDSTEP_ERR_INVALID, "log_ratios misaligned");
    add_range(writes, log_ratios, 8 * static_cast<int64_t>(n_pairs));
    if (int rc = check_ranges(&reads, &writes); rc != SHARDSTEP_OK) return rc;
    if (k.norm == 0.0f) k.norm = static_cast<float>(n_pairs);
    PreferenceArgs p = loss_words_at(k.ws, tokens);
    p.beta = beta;
    p.smoothing = label_smoothing;
    p.log_ratios = log_ratios;
    p.seq = reinterpret_cast<int32_t*>(p.term + tokens);
    p.coef = p.term + 2 * tokens;
    p.first = 1;
    const bool staged = k.grad != nullptr && same_offsets(args);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    std::unique_ptr<PairTableLarge> t(new PairTableLarge);
    const int64_t most = loss_rows_per_launch();
    int32_t row = 0;
    for (int32_t q = 0; q < n_pairs; q += kPairsPerLaunch) {
        t->pairs = std::min(kPairsPerLaunch, n_pairs - q);
        for (int32_t j = 0; j < 2 * t->pairs; ++j) {
            t->start[j] = row;
            row += static_cast<int32_t>(seq_lens[2 * static_cast<int64_t>(q) + j]);
        }
        t->start[2 * t->pairs] = row;
        p.last = q + t->pairs >= n_pairs;
        // the table's rows in as few launches as they fit; all of its forward
        // passes before the first backward pass, which needs its pairs' slopes
        const int64_t begin = t->start[0], end = row;
        cudaError_t e = cudaSuccess;
        for (int64_t r = begin; e == cudaSuccess && (r < end || r == begin); r += most)
            e = launch_preference_forward(k, p, *t, r, std::min(end, r + most), args->dtype, s);
        if (k.grad != nullptr)
            for (int64_t r = begin; e == cudaSuccess && r < end; r += most)
                e = launch_loss_backward(k, p, r, std::min(end, r + most), args->dtype, staged, s);
        if (e != cudaSuccess)
            return ready_fail(SHARDSTEP_ERR_CUDA, "preference loss launch: %s",
                              cudaGetErrorString(e));
        p.first = 0;
        p.log_ratios += 2 * static_cast<int64_t>(t->pairs);
        p.coef += 2 * static_cast<int64_t>(t->pairs);
    }
    record_kernel(k.grad == nullptr ? "stream_forward<%s> (TMA-staged)"
                  : staged          ? "staged_rows<%s, backward> (TMA-staged)"
                                    : "offset_backward<%s>",
                  dtype_name(args->dtype));
    return ready_ok();
} catch (const std::bad_alloc&) {
    return ready_fail(SHARDSTEP_ERR_CAPACITY, "out of host memory");
}

}  // extern "C"
