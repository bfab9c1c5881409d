// Element access shared by the elementwise and scan kernels: V consecutive io
// elements (fp32 or bf16) moved with one access of up to 16 bytes, and the
// softplus both scan directions use.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace ssd {
namespace elem {

// V elements of T as raw 32-bit words; the address is aligned to V * sizeof(T)
// (at most 16 bytes).
template <typename T, int V>
struct Pack {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T));
    static_assert(kBytes == 2 || kBytes == 4 || kBytes == 8 || kBytes == 16, "one access");
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];

    // read-only data: the non-coherent path
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
        }
    }
    // memory that this kernel writes (shared memory)
    __device__ __forceinline__ void load_plain(const T* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short*>(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t u = w[i >> 1];
            return __uint_as_float((i & 1) ? (u & 0xFFFF0000u) : (u << 16));
        } else {
            return __uint_as_float(w[i]);
        }
    }
    // rounds to nearest even where T is bf16
    __device__ __forceinline__ void set(const float* f) {
        if constexpr (sizeof(T) == 2) {
            if constexpr (V == 1) {
                w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kBytes == 16)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else
            *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(w[0]);
    }
};

constexpr float kLog2e = 1.4426950408889634f;

// 2^v (relative error about 2^-22; flushes subnormal results to zero)
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / v to one ulp, for normal v
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// V = 1 or 2 fp32 values that one thread works on together: two of them in one
// 64-bit register pair, where an add, a multiply or a fused multiply-add of both is
// one instruction.
template <int V>
struct Vals;
template <>
struct Vals<1> {
    float f;
    __device__ __forceinline__ float get(int) const { return f; }
    __device__ __forceinline__ static Vals make(float a, float) { return {a}; }
    __device__ __forceinline__ static Vals splat(float a) { return {a}; }
    __device__ __forceinline__ static Vals load(const float* p) { return {*p}; }
    __device__ __forceinline__ void store(float* p) const { *p = f; }
};
template <>
struct Vals<2> {
    unsigned long long u;
    __device__ __forceinline__ float get(int i) const {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(u));
        return i == 0 ? a : b;
    }
    __device__ __forceinline__ static Vals make(float a, float b) {
        Vals r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ static Vals splat(float a) { return make(a, a); }
    // two floats that need not lie on 8 bytes
    __device__ __forceinline__ static Vals load(const float* p) { return make(p[0], p[1]); }
    __device__ __forceinline__ void store(float* p) const { p[0] = get(0), p[1] = get(1); }
};

__device__ __forceinline__ Vals<1> fma(Vals<1> a, Vals<1> b, Vals<1> c) { return {fmaf(a.f, b.f, c.f)}; }
__device__ __forceinline__ Vals<1> mul(Vals<1> a, Vals<1> b) { return {a.f * b.f}; }
__device__ __forceinline__ Vals<1> add(Vals<1> a, Vals<1> b) { return {a.f + b.f}; }
__device__ __forceinline__ Vals<2> fma(Vals<2> a, Vals<2> b, Vals<2> c) {
    Vals<2> r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return r;
}
__device__ __forceinline__ Vals<2> mul(Vals<2> a, Vals<2> b) {
    Vals<2> r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ Vals<2> add(Vals<2> a, Vals<2> b) {
    Vals<2> r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
// f of each value
template <int V, typename F>
__device__ __forceinline__ Vals<V> each(Vals<V> a, F f) {
    if constexpr (V == 1)
        return {f(a.f)};
    else
        return Vals<2>::make(f(a.get(0)), f(a.get(1)));
}
template <int V>
__device__ __forceinline__ Vals<V> exp2_fast(Vals<V> a) {
    return each<V>(a, [](float v) { return exp2_fast(v); });
}
// e^v, v of either sign. Near 1, where a long product of such factors adds up their errors, the
// series 1 + v + v^2/2 + v^3/6 + v^4/24 (exact to 2^-26 for |v| < 1/16) rounds once; exp2_fast's
// error of up to 2^-22 showed in the gradients of slowly decaying states.
template <int V>
__device__ __forceinline__ Vals<V> exp_near(Vals<V> v) {
    using L = Vals<V>;
    const L e = exp2_fast<V>(mul(v, L::splat(kLog2e)));
    L s = fma(v, L::splat(1.f / 24.f), L::splat(1.f / 6.f));
    s = fma(s, v, L::splat(0.5f));
    s = fma(s, v, L::splat(1.f));
    s = fma(s, v, L::splat(1.f));
    if constexpr (V == 1)
        return {fabsf(v.f) < 0.0625f ? s.f : e.f};
    else
        return L::make(fabsf(v.get(0)) < 0.0625f ? s.get(0) : e.get(0), fabsf(v.get(1)) < 0.0625f ? s.get(1) : e.get(1));
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> unpack(const Pack<T, V>& k) {
    return Vals<V>::make(k.get(0), V == 2 ? k.get(V - 1) : 0.f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vals(T* p, Vals<V> a) {
    float f[2] = {a.get(0), V == 2 ? a.get(V - 1) : 0.f};
    Pack<T, V> k;
    k.set(f);
    k.store(p);
}

// softplus(v) = max(v, 0) + log(1 + u), u = e^-|v| in (0, 1]. With w = u / (2 + u)
// in (0, 1/3], log(1 + u) = 2 atanh(w) = w P(w^2): P of degree 4, interpolated at
// the Chebyshev nodes of [0, 1/9], is within 8e-9 of 2 atanh(w) / w, relative also
// where u is tiny (a logarithm of 1 + u would lose u's low bits there). *u_out: u,
// which the derivative (the sigmoid) needs.
template <int V>
__device__ __forceinline__ Vals<V> softplus(Vals<V> v, Vals<V>* u_out) {
    using L = Vals<V>;
    const L u = each<V>(v, [](float x) { return exp2_fast(-kLog2e * fabsf(x)); });
    const L r = each<V>(add(u, L::splat(2.f)), [](float x) { return rcp_fast(x); });
    const L w = mul(u, r), q = mul(w, w);
    L s = L::splat(0.281577796f);
    s = fma(s, q, L::splat(0.279651582f));
    s = fma(s, q, L::splat(0.400245965f));
    s = fma(s, q, L::splat(0.666663229f));
    s = fma(s, q, L::splat(2.f));
    *u_out = u;
    return fma(w, s, each<V>(v, [](float x) { return fmaxf(x, 0.f); }));
}

// d softplus(v) / d v = sigmoid(v), from u = e^-|v|
template <int V>
__device__ __forceinline__ Vals<V> softplus_slope(Vals<V> v, Vals<V> u) {
    const Vals<V> r = each<V>(add(u, Vals<V>::splat(1.f)), [](float x) { return rcp_fast(x); });
    if constexpr (V == 1)
        return {v.f >= 0.f ? r.f : u.f * r.f};
    else
        return mul(Vals<2>::make(v.get(0) >= 0.f ? 1.f : u.get(0), v.get(1) >= 0.f ? 1.f : u.get(1)), r);
}

}  // namespace elem
}  // namespace ssd
