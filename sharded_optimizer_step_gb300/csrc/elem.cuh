// Elements of the three floating types as fp32, one or a 16-byte vector at a
// time: what the row kernels (embedding.cu, layer_norm.cu) and the matrix
// kernels' passes over tensors (matrix.cu) share.
#pragma once

#include "common.cuh"

namespace shardstep {

// The storage type of a dtype code, and how many elements 16 bytes hold.
template <int TYPE>
struct Elem {
    using Store = uint16_t;
    static constexpr int kVec = 8;
};
template <>
struct Elem<kGradF32> {
    using Store = float;
    static constexpr int kVec = 4;
};

template <int TYPE>
__device__ __forceinline__ float elem_to_f32(typename Elem<TYPE>::Store v) {
    if constexpr (TYPE == kGradF32) return v;
    else if constexpr (TYPE == kGradF16) return f16_to_f32(v);
    else return bf16_to_f32(v);
}
// Round to nearest even.
template <int TYPE>
__device__ __forceinline__ typename Elem<TYPE>::Store elem_from_f32(float v) {
    if constexpr (TYPE == kGradF32) return v;
    else if constexpr (TYPE == kGradF16) return __half_as_ushort(__float2half_rn(v));
    else return f32_to_bf16(v);
}

template <int TYPE>
__device__ __forceinline__ void unpack16(const uint4& r, float* f) {
    if constexpr (TYPE == kGradF32) {
        unpack4f(r, f);
    } else if constexpr (TYPE == kGradF16) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
        }
    } else {
        unpack8(r, f);
    }
}
template <int TYPE>
__device__ __forceinline__ uint4 pack16(const float* f) {
    if constexpr (TYPE == kGradF32) {
        return pack4f(f);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (TYPE == kGradF16) {
                const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// N consecutive elements at p (N == 1, or 16-byte aligned vectors).
template <int TYPE, int N>
__device__ __forceinline__ void load_elems(const typename Elem<TYPE>::Store* p, float* f) {
    if constexpr (N == 1) {
        f[0] = elem_to_f32<TYPE>(*p);
    } else if constexpr (N < Elem<TYPE>::kVec) {   // four elements of 16 bits
        static_assert(N == 4, "half a vector");
        const uint2 r = *reinterpret_cast<const uint2*>(p);
        f[0] = elem_to_f32<TYPE>(static_cast<uint16_t>(r.x));
        f[1] = elem_to_f32<TYPE>(static_cast<uint16_t>(r.x >> 16));
        f[2] = elem_to_f32<TYPE>(static_cast<uint16_t>(r.y));
        f[3] = elem_to_f32<TYPE>(static_cast<uint16_t>(r.y >> 16));
    } else {
        constexpr int V = Elem<TYPE>::kVec;
        static_assert(N % V == 0, "whole vectors");
#pragma unroll
        for (int k = 0; k < N / V; ++k)
            unpack16<TYPE>(reinterpret_cast<const uint4*>(p)[k], f + k * V);
    }
}
template <int TYPE, int N>
__device__ __forceinline__ void store_elems(typename Elem<TYPE>::Store* p, const float* f) {
    if constexpr (N == 1) {
        *p = elem_from_f32<TYPE>(f[0]);
    } else if constexpr (N < Elem<TYPE>::kVec) {   // four elements of 16 bits
        static_assert(N == 4, "half a vector");
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = elem_from_f32<TYPE>(f[2 * k]) |
                   static_cast<uint32_t>(elem_from_f32<TYPE>(f[2 * k + 1])) << 16;
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
        constexpr int V = Elem<TYPE>::kVec;
#pragma unroll
        for (int k = 0; k < N / V; ++k)
            reinterpret_cast<uint4*>(p)[k] = pack16<TYPE>(f + k * V);
    }
}

// Calls f(std::integral_constant) of a dtype code.
template <int V>
struct Const {
    static constexpr int value = V;
};
template <typename F>
cudaError_t by_type(int type, F&& f) {
    return type == kGradF32 ? f(Const<kGradF32>()) : type == kGradF16 ? f(Const<kGradF16>())
                                                                     : f(Const<kGradBF16>());
}

}  // namespace shardstep
