// Argument checks that the host sides of the entry points over tensors share
// (tuning_api.cpp, model_api.cpp): alignment, element sizes, overlapping ranges.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <vector>

#include "internal.h"
#include "shardstep.h"

namespace shardstep {

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline int elem_size(int32_t dtype) {
    return dtype == SHARDSTEP_DTYPE_F32                                        ? 4
           : dtype == SHARDSTEP_DTYPE_BF16 || dtype == SHARDSTEP_DTYPE_F16 ? 2
                                                                               : 0;
}
inline const char* dtype_name(int dtype) {
    return dtype == SHARDSTEP_DTYPE_F32 ? "f32" : dtype == SHARDSTEP_DTYPE_F16 ? "f16" : "bf16";
}

struct Range {
    uintptr_t lo, hi;
};
inline void add_range(std::vector<Range>& v, const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0) v.push_back(Range{a, a + static_cast<uintptr_t>(bytes)});
}
inline void sort_ranges(std::vector<Range>& v) {
    const auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
}
// Whether any two of the sorted ranges share a byte.
inline bool self_overlap(const std::vector<Range>& v) {
    for (size_t k = 1; k < v.size(); ++k)
        if (v[k].lo < v[k - 1].hi) return true;
    return false;
}
// Whether a range of `reads` shares a byte with one of `writes` (both sorted;
// the writes disjoint).
inline bool cross_overlap(const std::vector<Range>& reads, const std::vector<Range>& writes) {
    size_t w = 0;
    for (const Range& r : reads) {
        while (w < writes.size() && writes[w].hi <= r.lo) ++w;
        if (w < writes.size() && writes[w].lo < r.hi) return true;
    }
    return false;
}
inline int check_ranges(std::vector<Range>* reads, std::vector<Range>* writes) {
    sort_ranges(*reads);
    sort_ranges(*writes);
    if (self_overlap(*writes) || cross_overlap(*reads, *writes))
        return ready_fail(SHARDSTEP_ERR_INVALID, "an output overlaps an input or another output");
    return SHARDSTEP_OK;
}

// The ranges of a call with a few arrays, without allocations.
struct FewRanges {
    Range r[16];
    int n = 0;
    void add(const void* p, int64_t bytes) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (bytes > 0) r[n++] = Range{a, a + static_cast<uintptr_t>(bytes)};
    }
};
inline int check_ranges(const FewRanges& reads, const FewRanges& writes) {
    for (int w = 0; w < writes.n; ++w) {
        const auto shares = [&](const Range& o) {
            return o.lo < writes.r[w].hi && writes.r[w].lo < o.hi;
        };
        for (int k = 0; k < w; ++k)
            if (shares(writes.r[k]))
                return ready_fail(SHARDSTEP_ERR_INVALID,
                                  "an output overlaps an input or another output");
        for (int k = 0; k < reads.n; ++k)
            if (shares(reads.r[k]))
                return ready_fail(SHARDSTEP_ERR_INVALID,
                                  "an output overlaps an input or another output");
    }
    return SHARDSTEP_OK;
}

}  // namespace shardstep
