// The residual update between two blocks and its gradient (include/ssd.h,
// ssd_block_norm), per row of dim channels:
//
//   u  = y silu(z)                           (u = y without z)
//   un = u / sqrt(mean(u^2) + eps)           (un = u without post_weight)
//   r' = residual + scale post_weight un
//   rn = r' / sqrt(mean(r'^2) + eps)         out = pre_weight rn
//
// Backward, with the forward's two 1/rms values rho_u, rho saved per row, c =
// scale post_weight and n = dout pre_weight:
//
//   dr = dresidual_out + rho (n - rn mean(n rn))           (the gradient of r' and of residual)
//   e  = c dr     du = rho_u (e - un mean(e un))     dy = du silu(z)   dz = du y silu'(z)
//   dpost_weight = scale sum dr un   dscale = post_weight sum dr un   dpre_weight = sum dout rn
//
// mean(e un) follows from sums that need no dr first (dr is linear in mean(n rn)):
//   sum e un = sum c un dresidual_out + rho (sum c un n - mean(n rn) sum c un rn)
// so the backward reduces once per row. A row stays in registers between its
// reductions: each input is read once and each output written once. Both
// directions are bound by HBM bandwidth. A row takes one or more whole warps (R
// vectors of V elements per thread); with one warp per row nothing waits for
// another warp. The backward's column sums stay in registers over a fixed set of
// rows per CTA, leave as one row per warp group and are added in a fixed order
// by a second kernel.
#include <algorithm>
#include <initializer_list>

#include "elem.cuh"
#include "ptx.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using elem::Pack;

constexpr int kMaxThreads = 1024;
// backward: 64 registers a thread hold four elements of a row, 128 eight and more
constexpr int bwd_threads(int elements) { return elements <= 4 ? 1024 : 512; }
constexpr int64_t kMaxDim = 16384;

// V elements in accesses of at most 16 bytes
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
    constexpr int N = V * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : V;
#pragma unroll
    for (int i = 0; i < V; i += N) {
        Pack<T, N> k;
        k.load(p + i);
#pragma unroll
        for (int j = 0; j < N; ++j) f[i + j] = k.get(j);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    constexpr int N = V * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : V;
#pragma unroll
    for (int i = 0; i < V; i += N) {
        Pack<T, N> k;
        k.set(f + i);
        k.store(p + i);
    }
}
template <int V>
__device__ __forceinline__ void load_weight(const float* p, long long c, float (&f)[V]) {
    if (p) {
        load_vec<float, V>(p + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 1.f;
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + elem::exp2_fast(-elem::kLog2e * z)); }

template <typename T, typename TR>
struct NormParams {
    const T *y, *z, *dout;
    const TR *res, *dres;
    T *out, *dy, *dz;
    TR *res_out, *dres_in;
    const float *post, *scale, *pre;
    float2* rstd;  // per row (rho_u, rho); the forward may leave it NULL
    float* sums;   // backward: [grid * groups, 2, dim]
    long long rows, ys, zs, dos;  // row strides of y, z and dout
    int dim, warps_per_row;
    int lanes;  // direct kernels: lanes per row where a row takes one warp or less (else 32)
    float eps;
    unsigned* status;
    unsigned long long wait_ns;  // limit on a wait for a row's copies
};

// Sums N values over the threads of one row: `lanes` (8, 16 or 32) lanes of each of its warps.
template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* buf, int warps, int lanes, int warp, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (lanes > 16) s[i] += __shfl_xor_sync(0xffffffffu, s[i], 16);
        if (lanes > 8) s[i] += __shfl_xor_sync(0xffffffffu, s[i], 8);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    }
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[warp * N + i] = s[i];
    }
    __syncthreads();
    const int first = warp / warps * warps;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    for (int w = first; w < first + warps; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += buf[w * N + i];
}

template <typename T, typename TR, int V, int R>
__global__ void __launch_bounds__(kMaxThreads) block_norm_fwd(const NormParams<T, TR> p) {
    __shared__ float buf[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = p.warps_per_row * p.lanes;  // threads per row
    const int groups = blockDim.x / stride, group = threadIdx.x / stride, tid = threadIdx.x - group * stride;
    const long long row = static_cast<long long>(blockIdx.x) * groups + group;
    const bool in = row < p.rows;
    const float inv = 1.f / static_cast<float>(p.dim);
    float u[R][V], r[R][V];
    float su[1] = {0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (tid + k * stride) * V;
        const bool live = in && c < p.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) u[k][i] = r[k][i] = 0.f;
        if (live) {
            load_vec<T, V>(p.y + row * p.ys + c, u[k]);
            if (p.z) {
                float z[V];
                load_vec<T, V>(p.z + row * p.zs + c, z);
#pragma unroll
                for (int i = 0; i < V; ++i) u[k][i] *= z[i] * sigmoid(z[i]);
            }
            if (p.res) load_vec<TR, V>(p.res + row * p.dim + c, r[k]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) su[0] = fmaf(u[k][i], u[k][i], su[0]);
    }
    float rho_u = 1.f;
    if (p.post) {
        row_sum<1>(su, buf[0], p.warps_per_row, p.lanes, warp, lane);
        rho_u = rsqrtf(fmaf(su[0], inv, p.eps));
    }
    float sr[1] = {0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (tid + k * stride) * V;
        if (in && c < p.dim) {
            float w[V], s[V];
            load_weight<V>(p.post, c, w);
            load_weight<V>(p.scale, c, s);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                r[k][i] = fmaf(u[k][i] * rho_u, w[i] * s[i], r[k][i]);
                sr[0] = fmaf(r[k][i], r[k][i], sr[0]);
            }
            store_vec<TR, V>(p.res_out + row * p.dim + c, r[k]);
        }
    }
    float rho = 1.f;
    if (p.pre) {
        row_sum<1>(sr, buf[1], p.warps_per_row, p.lanes, warp, lane);
        rho = rsqrtf(fmaf(sr[0], inv, p.eps));
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (tid + k * stride) * V;
            if (in && c < p.dim) {
                float w[V];
                load_weight<V>(p.pre, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] *= r[k][i] * rho;
                store_vec<T, V>(p.out + row * p.dim + c, w);
            }
        }
    }
    if (p.rstd && in && tid == 0) p.rstd[row] = make_float2(rho_u, rho);
}

// One thread's vector of each backward input, as loaded: values are unpacked where
// they are used, twice, which costs less than holding a row's fp32 intermediates.
template <typename T, int V>
struct RawVec {
    static constexpr int N = V * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : V;
    Pack<T, N> k[V / N];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < V / N; ++i) k[i].load(p + i * N);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V / N; ++i) k[i].zero();
    }
    __device__ __forceinline__ float get(int i) const { return k[i / N].get(i % N); }
};

template <typename T, typename TR, int V, int R>
__global__ void __launch_bounds__(bwd_threads(R * V)) block_norm_bwd(const NormParams<T, TR> p) {
    __shared__ float buf[2][32 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = p.warps_per_row * p.lanes;  // threads per row
    const int groups = blockDim.x / stride, group = threadIdx.x / stride, tid = threadIdx.x - group * stride;
    const float inv = 1.f / static_cast<float>(p.dim);
    float sum_post[R][V], sum_pre[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sum_post[k][i] = sum_pre[k][i] = 0.f;
    int turn = 0;
    for (long long row0 = static_cast<long long>(blockIdx.x) * groups; row0 < p.rows;
         row0 += static_cast<long long>(gridDim.x) * groups, turn ^= 1) {
        const long long row = row0 + group;
        const bool in = row < p.rows;
        const float2 rho = in ? __ldg(p.rstd + row) : make_float2(0.f, 0.f);
        RawVec<T, V> y[R], z[R], dn[R];
        RawVec<TR, V> res[R], dres[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (tid + k * stride) * V;
            y[k].zero(), z[k].zero(), dn[k].zero(), res[k].zero(), dres[k].zero();
            if (in && c < p.dim) {
                y[k].load(p.y + row * p.ys + c);
                if (p.z) z[k].load(p.z + row * p.zs + c);
                if (p.dout) dn[k].load(p.dout + row * p.dos + c);
                if (p.res) res[k].load(p.res + row * p.dim + c);
                if (p.dres) dres[k].load(p.dres + row * p.dim + c);
            }
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};  // n rn, c un dres, c un n, c un rn
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (tid + k * stride) * V;
            if (in && c < p.dim) {
                float w[V], sc[V], pre[V];
                load_weight<V>(p.post, c, w);
                load_weight<V>(p.scale, c, sc);
                load_weight<V>(p.pre, c, pre);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float u = y[k].get(i);
                    if (p.z) u *= z[k].get(i) * sigmoid(z[k].get(i));
                    const float c_un = w[i] * sc[i] * (u * rho.x);
                    const float rn = (res[k].get(i) + c_un) * rho.y;
                    const float n = dn[k].get(i) * pre[i];
                    s[0] = fmaf(n, rn, s[0]);
                    s[1] = fmaf(c_un, dres[k].get(i), s[1]);
                    s[2] = fmaf(c_un, n, s[2]);
                    s[3] = fmaf(c_un, rn, s[3]);
                }
            }
        }
        row_sum<4>(s, buf[turn], p.warps_per_row, p.lanes, warp, lane);
        const float m_rn = s[0] * inv;
        const float m_un = p.post ? (s[1] + rho.y * (s[2] - m_rn * s[3])) * inv : 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (tid + k * stride) * V;
            if (in && c < p.dim) {
                float w[V], sc[V], pre[V], dr[V], dy[V], dz[V];
                load_weight<V>(p.post, c, w);
                load_weight<V>(p.scale, c, sc);
                load_weight<V>(p.pre, c, pre);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float yv = y[k].get(i), zv = z[k].get(i), sg = p.z ? sigmoid(zv) : 1.f;
                    const float gate = p.z ? zv * sg : 1.f;
                    const float un = yv * gate * rho.x, cc = w[i] * sc[i];
                    const float rn = fmaf(cc, un, res[k].get(i)) * rho.y;
                    const float dnv = dn[k].get(i);
                    dr[i] = dres[k].get(i);
                    if (p.pre) dr[i] = fmaf(rho.y, dnv * pre[i] - rn * m_rn, dr[i]);
                    sum_post[k][i] = fmaf(dr[i], un, sum_post[k][i]);
                    sum_pre[k][i] = fmaf(dnv, rn, sum_pre[k][i]);
                    const float du = rho.x * (cc * dr[i] - un * m_un);
                    dz[i] = du * yv * (sg * fmaf(zv, 1.f - sg, 1.f));
                    dy[i] = du * gate;
                }
                if (p.dres_in) store_vec<TR, V>(p.dres_in + row * p.dim + c, dr);
                if (p.z) store_vec<T, V>(p.dz + row * p.dim + c, dz);
                store_vec<T, V>(p.dy + row * p.dim + c, dy);
            }
        }
    }
    // one row of sums per group of whole warps: a warp's rows are added first
    if (p.lanes < 32) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (p.lanes <= 8) {
                    sum_post[k][i] += __shfl_xor_sync(0xffffffffu, sum_post[k][i], 8);
                    sum_pre[k][i] += __shfl_xor_sync(0xffffffffu, sum_pre[k][i], 8);
                }
                sum_post[k][i] += __shfl_xor_sync(0xffffffffu, sum_post[k][i], 16);
                sum_pre[k][i] += __shfl_xor_sync(0xffffffffu, sum_pre[k][i], 16);
            }
        if (lane >= p.lanes) return;
    }
    const int parts = (blockDim.x >> 5) / p.warps_per_row;
    float* out = p.sums + (static_cast<long long>(blockIdx.x) * parts + warp / p.warps_per_row) * 2 * p.dim;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int c = (tid + k * stride) * V;
        if (c < p.dim) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                out[c + i] = sum_post[k][i];
                out[p.dim + c + i] = sum_pre[k][i];
            }
        }
    }
}

// ---------------------------------------------------------------- many rows: persistent CTAs
// The direct kernels above keep a row's loads in flight only until its reduction
// starts: 16384 x 2560 (bf16, fp32 residual) ran at 4.1 TB/s forward and 2.9 backward.
// Here a CTA stays on its SM and each of its groups of warps takes every n-th row: a group's first
// lane has the next rows' tensors copied into shared memory (one bulk copy per tensor and row, a
// ring of stages) while the group works, and the weights stay in registers.
// 96 or 128 registers a thread (rows that start anywhere, backward: 16384 x 771 took 100 us with
// 512 threads and 162 with 640, whose registers spill)
constexpr int ring_threads(int V, int R, bool backward) { return V * R > 8 || (backward && V <= 2) ? 512 : 640; }
constexpr int kRingBytes = 208 << 10;
constexpr unsigned long long kDrainNs = 2000000000ull;  // limit on the wait for copies in flight after a wait has run out

struct RingShape {
    int groups, stages;
    int io_bytes, res_bytes;  // room for a row of an io tensor and of a residual one
    int row_bytes;            // of a stage: the inputs of one row, one after another
};

// A row of n bytes that starts anywhere, as the 16-byte granules that hold it: bulk copies
// start on and consist of those. (The bytes around the row lie in granules of its own first and
// last elements, so in the same allocation.)
__device__ __forceinline__ uint32_t granules(const void* row, uint32_t n) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    return (off + n + 15u) & ~15u;
}

// kAny: rows start anywhere; else on 16 bytes.
template <typename T, typename TR, bool kBwd, bool kAny>
struct Ring {
    const NormParams<T, TR>& p;
    const RingShape& g;
    unsigned char* stage0;  // this group's stages
    uint64_t* full;         // one barrier per stage
    __device__ __forceinline__ unsigned char* stage(int i) const { return stage0 + i * g.row_bytes; }
    template <typename E>
    __device__ __forceinline__ static const E* inside(const unsigned char* at, const void* row) {
        return reinterpret_cast<const E*>(kAny ? at + (reinterpret_cast<uintptr_t>(row) & 15u) : at);
    }
    // each tensor's place in a stage, and its row there
    __device__ __forceinline__ int z_at() const { return g.io_bytes; }
    __device__ __forceinline__ int dn_at() const { return z_at() + (p.z ? g.io_bytes : 0); }
    __device__ __forceinline__ int res_at() const { return dn_at() + (kBwd && p.dout ? g.io_bytes : 0); }
    __device__ __forceinline__ int dres_at() const { return res_at() + (p.res ? g.res_bytes : 0); }
    __device__ __forceinline__ const T* y_of(const unsigned char* s, long long row) const {
        return inside<T>(s, p.y + row * p.ys);
    }
    __device__ __forceinline__ const T* z_of(const unsigned char* s, long long row) const {
        return inside<T>(s + z_at(), p.z + row * p.zs);
    }
    __device__ __forceinline__ const T* dn_of(const unsigned char* s, long long row) const {
        return inside<T>(s + dn_at(), p.dout + row * p.dos);
    }
    __device__ __forceinline__ const TR* res_of(const unsigned char* s, long long row) const {
        return inside<TR>(s + res_at(), p.res + row * p.dim);
    }
    __device__ __forceinline__ const TR* dres_of(const unsigned char* s, long long row) const {
        return inside<TR>(s + dres_at(), p.dres + row * p.dim);
    }
    // one lane
    __device__ __forceinline__ void load(int i, long long row) const {
        unsigned char* s = stage(i);
        const uint32_t n = p.dim * sizeof(T), nr = p.dim * sizeof(TR);
        const void* src[5] = {p.y + row * p.ys, p.z ? p.z + row * p.zs : nullptr,
                              kBwd && p.dout ? p.dout + row * p.dos : nullptr, p.res ? p.res + row * p.dim : nullptr,
                              kBwd && p.dres ? p.dres + row * p.dim : nullptr};
        const int at[5] = {0, z_at(), dn_at(), res_at(), dres_at()};
        uint32_t bytes[5], total = 0;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const uint32_t row_n = k < 3 ? n : nr;
            bytes[k] = src[k] ? (kAny ? granules(src[k], row_n) : row_n) : 0u;
            total += bytes[k];
        }
        ptx::mbar_arrive_expect_tx(&full[i], total);
#pragma unroll
        for (int k = 0; k < 5; ++k)
            if (src[k])
                ptx::bulk_load(s + at[k], reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(src[k]) & ~uintptr_t{15}),
                               bytes[k], &full[i]);
    }
};

// V elements of shared memory
template <typename T, int V>
__device__ __forceinline__ void read_vec(const T* s, RawVec<T, V>& r) {
#pragma unroll
    for (int i = 0; i < V / RawVec<T, V>::N; ++i) r.k[i].load_plain(s + i * RawVec<T, V>::N);
}

// Sums N values over a group's warps; everything the group read before is read when it returns.
template <int N>
__device__ __forceinline__ void group_sum(float (&s)[N], float* buf, int warps, int in_group, int lane, int barrier) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    if (warps == 1) {
        __syncwarp();
        return;
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[in_group * N + i] = s[i];
    }
    ptx::named_sync(barrier, 32 * warps);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += buf[w * N + i];
}

// Polls for a phase for at most limit_ns.
__device__ __forceinline__ bool poll(uint64_t* bar, uint32_t phase, unsigned long long limit_ns) {
    if (ptx::mbar_test_wait(bar, phase)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_test_wait(bar, phase))
        if (ptx::globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

// Common to both directions: the group's place, its ring, and the walk over its rows.
// body(row, stage, release): release(), called by the whole group once it has read the stage.
template <typename T, typename TR, bool kBwd, bool kAny, typename Body>
__device__ __forceinline__ void walk_rows(const NormParams<T, TR>& p, const RingShape& g, unsigned char* smem, Body body) {
    __shared__ uint64_t full[16 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / p.warps_per_row, first_warp = group * p.warps_per_row;
    const Ring<T, TR, kBwd, kAny> ring{p, g, smem + static_cast<size_t>(group) * g.stages * g.row_bytes,
                                       full + group * g.stages};
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.groups * g.stages; ++i) ptx::mbar_init(&full[i], 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const uint32_t step = gridDim.x * g.groups, rows = static_cast<uint32_t>(p.rows);  // (sums stay below 2^32)
    const uint32_t row0 = blockIdx.x * g.groups + group;
    const bool loader = warp == first_warp && lane == 0;
    if (loader) {
        for (int i = 0; i < g.stages; ++i)
            if (row0 + i * step < rows) ring.load(i, row0 + i * step);
    }
    int at = 0;
    uint32_t phase = 0;
    for (uint32_t row = row0; row < rows; row += step) {
        if (!__all_sync(0xffffffffu, poll(&full[group * g.stages + at], phase, p.wait_ns))) {
            // A warp whose wait has run out reports it and works on no more rows, but meets the other warps at the
            // barriers of those rows (their waits end too: nothing more is copied once the loader has left). The
            // loader first sees its copies in flight land, so that none is left when the CTA ends.
            if (lane == 0) atomicOr(p.status, 1u);
            for (int i = 0; i < g.stages && loader && row + i * step < rows; ++i) {
                poll(&ring.full[at], phase, kDrainNs);
                if (++at == g.stages) at = 0, phase ^= 1u;
            }
            __syncwarp();
            const int barriers = p.warps_per_row == 1 ? 0 : !kBwd && p.pre ? 2 : 1;  // group_sums of a row
            for (; row < rows; row += step)
                for (int i = 0; i < barriers; ++i) ptx::named_sync(1 + group, 32 * p.warps_per_row);
            return;
        }
        const uint32_t next = row + g.stages * step;
        body(row, ring, ring.stage(at), [&] {
            if (loader && next < rows) ring.load(at, next);
        });
        if (++at == g.stages) at = 0, phase ^= 1u;
    }
}

template <typename T, typename TR, int V, int R>
__global__ void __launch_bounds__(ring_threads(V, R, false), 1) block_norm_fwd_ring(const NormParams<T, TR> p, const RingShape g) {
    extern __shared__ __align__(128) unsigned char smem[];
    // The first sum's two take turns by row: without a pre-norm it is a row's only barrier, and a fast
    // warp writes the next row's part while a slow one still adds up this row's. The second sum has its own.
    __shared__ float bufs[16][3][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / p.warps_per_row, in_group = warp - group * p.warps_per_row;
    const int tid = in_group * 32 + lane, stride = p.warps_per_row * 32;
    const float inv = 1.f / static_cast<float>(p.dim);
    float c[R][V], pre[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int col = (tid + k * stride) * V;
        if (col < p.dim) {
            float s[V];
            load_weight<V>(p.post, col, c[k]);
            load_weight<V>(p.scale, col, s);
            load_weight<V>(p.pre, col, pre[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) c[k][i] *= s[i];
        }
    }
    int turn = 0;
    walk_rows<T, TR, false, (V <= 2)>(p, g, smem, [&](long long row, const auto& ring, const unsigned char* st, auto release) {
        float u[R][V], r[R][V], su[1] = {0.f};
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int col = (tid + k * stride) * V;
            if (col < p.dim) {
                RawVec<T, V> y, z;
                read_vec(ring.y_of(st, row) + col, y);
                if (p.z) read_vec(ring.z_of(st, row) + col, z);
                if (p.res) {
                    RawVec<TR, V> x;
                    read_vec(ring.res_of(st, row) + col, x);
#pragma unroll
                    for (int i = 0; i < V; ++i) r[k][i] = x.get(i);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    u[k][i] = y.get(i);
                    if (p.z) u[k][i] *= z.get(i) * sigmoid(z.get(i));
                    if (!p.res) r[k][i] = 0.f;
                    su[0] = fmaf(u[k][i], u[k][i], su[0]);
                }
            }
        }
        group_sum<1>(su, bufs[group][turn], p.warps_per_row, in_group, lane, 1 + group);
        turn ^= 1;
        release();
        const float rho_u = p.post ? rsqrtf(fmaf(su[0], inv, p.eps)) : 1.f;
        float sr[1] = {0.f};
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int col = (tid + k * stride) * V;
            if (col < p.dim) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    r[k][i] = fmaf(u[k][i] * rho_u, c[k][i], r[k][i]);
                    sr[0] = fmaf(r[k][i], r[k][i], sr[0]);
                }
                store_vec<TR, V>(p.res_out + row * p.dim + col, r[k]);
            }
        }
        float rho = 1.f;
        if (p.pre) {
            group_sum<1>(sr, bufs[group][2], p.warps_per_row, in_group, lane, 1 + group);
            rho = rsqrtf(fmaf(sr[0], inv, p.eps));
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int col = (tid + k * stride) * V;
                if (col < p.dim) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = pre[k][i] * (r[k][i] * rho);
                    store_vec<T, V>(p.out + row * p.dim + col, o);
                }
            }
        }
        if (p.rstd && tid == 0) p.rstd[row] = make_float2(rho_u, rho);
    });
}

template <typename T, typename TR, int V, int R>
__global__ void __launch_bounds__(ring_threads(V, R, true), 1) block_norm_bwd_ring(const NormParams<T, TR> p, const RingShape g) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float bufs[16][2][32 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / p.warps_per_row, in_group = warp - group * p.warps_per_row;
    const int tid = in_group * 32 + lane, stride = p.warps_per_row * 32;
    const float inv = 1.f / static_cast<float>(p.dim);
    float c[R][V], pre[R][V], sum_post[R][V], sum_pre[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int col = (tid + k * stride) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) sum_post[k][i] = sum_pre[k][i] = 0.f;
        if (col < p.dim) {
            float s[V];
            load_weight<V>(p.post, col, c[k]);
            load_weight<V>(p.scale, col, s);
            load_weight<V>(p.pre, col, pre[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) c[k][i] *= s[i];
        }
    }
    int turn = 0;
    walk_rows<T, TR, true, (V <= 2)>(p, g, smem, [&](long long row, const auto& ring, const unsigned char* st, auto release) {
        const float2 rho = __ldg(p.rstd + row);
        RawVec<T, V> y[R], z[R], dn[R];
        RawVec<TR, V> res[R], dres[R];
        float s[4] = {0.f, 0.f, 0.f, 0.f};  // n rn, c un dres, c un n, c un rn
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int col = (tid + k * stride) * V;
            z[k].zero(), dn[k].zero(), res[k].zero(), dres[k].zero();
            if (col < p.dim) {
                read_vec(ring.y_of(st, row) + col, y[k]);
                if (p.z) read_vec(ring.z_of(st, row) + col, z[k]);
                if (p.dout) read_vec(ring.dn_of(st, row) + col, dn[k]);
                if (p.res) read_vec(ring.res_of(st, row) + col, res[k]);
                if (p.dres) read_vec(ring.dres_of(st, row) + col, dres[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float u = y[k].get(i);
                    if (p.z) u *= z[k].get(i) * sigmoid(z[k].get(i));
                    const float c_un = c[k][i] * (u * rho.x);
                    const float rn = (res[k].get(i) + c_un) * rho.y;
                    const float n = dn[k].get(i) * pre[k][i];
                    s[0] = fmaf(n, rn, s[0]);
                    s[1] = fmaf(c_un, dres[k].get(i), s[1]);
                    s[2] = fmaf(c_un, n, s[2]);
                    s[3] = fmaf(c_un, rn, s[3]);
                }
            }
        }
        group_sum<4>(s, bufs[group][turn], p.warps_per_row, in_group, lane, 1 + group);
        turn ^= 1;
        release();
        const float m_rn = s[0] * inv;
        const float m_un = p.post ? (s[1] + rho.y * (s[2] - m_rn * s[3])) * inv : 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int col = (tid + k * stride) * V;
            if (col < p.dim) {
                float dr[V], dy[V], dz[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float yv = y[k].get(i), zv = z[k].get(i), sg = p.z ? sigmoid(zv) : 1.f;
                    const float gate = p.z ? zv * sg : 1.f;
                    const float un = yv * gate * rho.x;
                    const float rn = fmaf(c[k][i], un, res[k].get(i)) * rho.y;
                    const float dnv = dn[k].get(i);
                    dr[i] = dres[k].get(i);
                    if (p.pre) dr[i] = fmaf(rho.y, dnv * pre[k][i] - rn * m_rn, dr[i]);
                    sum_post[k][i] = fmaf(dr[i], un, sum_post[k][i]);
                    sum_pre[k][i] = fmaf(dnv, rn, sum_pre[k][i]);
                    const float du = rho.x * (c[k][i] * dr[i] - un * m_un);
                    dz[i] = du * yv * (sg * fmaf(zv, 1.f - sg, 1.f));
                    dy[i] = du * gate;
                }
                if (p.dres_in) store_vec<TR, V>(p.dres_in + row * p.dim + col, dr);
                if (p.z) store_vec<T, V>(p.dz + row * p.dim + col, dz);
                store_vec<T, V>(p.dy + row * p.dim + col, dy);
            }
        }
    });
    float* out = p.sums + (static_cast<long long>(blockIdx.x) * g.groups + group) * 2 * p.dim;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int col = (tid + k * stride) * V;
        if (col < p.dim) {
            store_vec<float, V>(out + col, sum_post[k]);
            store_vec<float, V>(out + p.dim + col, sum_pre[k]);
        }
    }
}

// The weights' gradients from the groups' column sums, added in a fixed order.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
    block_norm_sums(const float* __restrict__ sums, int parts, int dim, const float* __restrict__ post,
                    const float* __restrict__ scale, float* dpost, float* dscale, float* dpre) {
    __shared__ float part[kSumRows][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + tx;
    float s = 0.f;
    if (col < 2 * dim) {
#pragma unroll 8
        for (int r = ty; r < parts; r += kSumRows) s += sums[static_cast<long long>(r) * 2 * dim + col];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && col < 2 * dim) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) s += part[k][tx];
        if (col < dim) {
            if (dpost) dpost[col] = scale ? s * scale[col] : s;
            if (dscale) dscale[col] = post ? s * post[col] : s;
        } else if (dpre) {
            dpre[col - dim] = s;
        }
    }
}

// ---------------------------------------------------------------- host side
struct NormPlan {
    int V, R, warps_per_row, lanes;
    unsigned threads, grid;
    int parts;  // rows of the backward's sums
};

// The direct kernels' plan. V: 16 bytes of the io type where every row allows it, two elements
// where every row starts on two, else one. R vectors per thread: one of 16 bytes, or
// four elements (loads in flight per thread), more where a CTA would not cover the row (a power
// of two, at most 32 / V). Short rows share a warp. The backward's CTAs stay and
// take every n-th row.
NormPlan norm_plan(int64_t rows, int64_t dim, ssd_dtype io, int align, bool backward, int sms) {
    NormPlan n;
    n.V = align == 16 ? (io == SSD_BF16 ? 8 : 4) : align;
    const int64_t nvec = (dim + n.V - 1) / n.V;
    n.R = align == 16 || nvec <= 32 ? 1 : 4 / n.V;
    while (nvec > static_cast<int64_t>(n.R) * (backward ? bwd_threads(n.R * n.V) : kMaxThreads)) n.R *= 2;
    n.warps_per_row = static_cast<int>((nvec + 32 * n.R - 1) / (32 * n.R));
    n.lanes = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    const int warps = n.warps_per_row >= 8 ? n.warps_per_row : 8 / n.warps_per_row * n.warps_per_row;
    n.threads = 32u * warps;
    const int64_t per = n.threads / (n.warps_per_row * n.lanes);  // rows per CTA
    int64_t ctas = (rows + per - 1) / per;
    if (backward) ctas = std::min<int64_t>(ctas, static_cast<int64_t>(sms) * std::max(1, 32 / warps));
    n.grid = static_cast<unsigned>(ctas);
    n.parts = static_cast<int>(ctas) * (warps / n.warps_per_row);
    return n;
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T, typename TR, int V, int R>
void launch_norm_r(const NormParams<T, TR>& p, const NormPlan& n, bool backward, cudaStream_t stream) {
    const unsigned threads = n.threads;
    if (backward)
        block_norm_bwd<T, TR, V, R><<<n.grid, threads, 0, stream>>>(p);
    else if constexpr (R * V <= 16)  // kMaxDim over kMaxThreads
        block_norm_fwd<T, TR, V, R><<<n.grid, threads, 0, stream>>>(p);
}

template <typename T, typename TR, int V>
ssd_status launch_norm_v(const NormParams<T, TR>& p, const NormPlan& n, bool backward, cudaStream_t stream) {
    // a vector width of V reaches kMaxDim with R = 16384 / (512 V) at most
    switch (n.R) {
#define SSD_NORM_CASE(RR)                                         \
    case RR:                                                      \
        if constexpr (RR * V <= 32) {                             \
            launch_norm_r<T, TR, V, RR>(p, n, backward, stream);  \
            break;                                                \
        } else {                                                  \
            return SSD_ERR_UNSUPPORTED;                           \
        }
        SSD_NORM_CASE(1)
        SSD_NORM_CASE(2)
        SSD_NORM_CASE(4)
        SSD_NORM_CASE(8)
        SSD_NORM_CASE(16)
        SSD_NORM_CASE(32)
#undef SSD_NORM_CASE
        default: return SSD_ERR_UNSUPPORTED;
    }
    note_launches(1);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// The ring's plan. Rows on 16 bytes: one vector per thread (the forward: two over 384
// vectors), up to 640 vectors backward and 1024 forward (16384 x 8192 forward and
// backward: 0.93 ms with the forward on the ring and the backward direct, 1.28 ms both direct; the backward's
// two vectors per thread would spill). Rows that start anywhere: eight elements per thread, up to
// 4096 backward and 5120 forward (both directions together, bf16 with an fp32 residual, against the
// direct kernels: 16384 x 771 149 and 251 us, x 2561 531 and 1078, x 4001 599 and 1486; with four elements per thread
// x 771 217). As many groups as the threads allow, at least two stages each. Other
// rows, rows that share a warp, and too few rows to fill every group's ring on every SM take the
// direct kernels.
template <typename T, typename TR>
bool ring_plan(const NormParams<T, TR>& p, int align, bool backward, NormPlan* n, RingShape* g) {
    constexpr int kWide = 16 / static_cast<int>(sizeof(T));
    n->V = align == 16 ? kWide : align;
    const int nvec = p.dim / n->V;
    if (align == 16) {
        if (nvec <= 16 || nvec > (backward ? 640 : 1024)) return false;
        n->R = nvec <= (backward ? 640 : 384) ? 1 : 2;
    } else {
        if (p.dim <= 128 || p.dim > (backward ? 4096 : 5120)) return false;
        n->R = 8 / n->V;
    }
    const int most = ring_threads(n->V, n->R, backward);
    n->warps_per_row = (nvec + 32 * n->R - 1) / (32 * n->R);
    if (32 * n->warps_per_row > most) return false;
    const int slack = align == 16 ? 0 : 16;  // a row may begin and end inside a granule
    g->io_bytes = static_cast<int>(align_up(p.dim * sizeof(T), 16)) + slack;
    g->res_bytes = static_cast<int>(align_up(p.dim * sizeof(TR), 16)) + slack;
    g->row_bytes = g->io_bytes * (1 + (p.z ? 1 : 0) + (backward && p.dout ? 1 : 0)) +
                   g->res_bytes * ((p.res ? 1 : 0) + (backward && p.dres ? 1 : 0));
    g->groups = std::min(16, most / (32 * n->warps_per_row));
    while (g->groups > 1 && g->groups * 2 * g->row_bytes > kRingBytes) --g->groups;
    g->stages = std::min(4, kRingBytes / (g->groups * g->row_bytes));
    if (g->stages < 2) return false;
    const int sms = device_sms();
    n->lanes = 32;
    n->threads = 32u * n->warps_per_row * g->groups;
    n->grid = static_cast<unsigned>(sms);
    n->parts = sms * g->groups;
    return p.rows >= 2ll * sms * g->groups;
}

template <typename T, typename TR>
ssd_status launch_ring(const NormParams<T, TR>& p, const NormPlan& n, const RingShape& g, bool backward,
                       cudaStream_t stream) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    using Kernel = void (*)(NormParams<T, TR>, RingShape);
    Kernel kernel;
    if (backward)
        kernel = n.V == 1   ? block_norm_bwd_ring<T, TR, 1, 8>
                 : n.V == 2 ? block_norm_bwd_ring<T, TR, 2, 4>
                            : block_norm_bwd_ring<T, TR, V, 1>;
    else if (n.V == 1)
        kernel = block_norm_fwd_ring<T, TR, 1, 8>;
    else if (n.V == 2)
        kernel = block_norm_fwd_ring<T, TR, 2, 4>;
    else
        kernel = n.R == 1 ? block_norm_fwd_ring<T, TR, V, 1> : block_norm_fwd_ring<T, TR, V, 2>;
    const int smem = g.groups * g.stages * g.row_bytes;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return SSD_ERR_CUDA;
    kernel<<<n.grid, n.threads, smem, stream>>>(p, g);
    note_launches(1);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

template <typename T, typename TR>
ssd_status launch_norm(NormParams<T, TR>& p, int align, bool backward, NormPlan* n, cudaStream_t stream) {
    constexpr int kWide = 16 / static_cast<int>(sizeof(T));
    RingShape g;
    if (ring_plan(p, align, backward, n, &g)) {
        p.warps_per_row = n->warps_per_row;
        const ssd_status st = call_context(&p.status, &p.wait_ns);
        if (st != SSD_OK) return st;
        return launch_ring(p, *n, g, backward, stream);
    }
    *n = norm_plan(p.rows, p.dim, sizeof(T) == 2 ? SSD_BF16 : SSD_F32, align, backward, device_sms());
    p.warps_per_row = n->warps_per_row, p.lanes = n->lanes;
    return n->V == 1   ? launch_norm_v<T, TR, 1>(p, *n, backward, stream)
           : n->V == 2 ? launch_norm_v<T, TR, 2>(p, *n, backward, stream)
                       : launch_norm_v<T, TR, kWide>(p, *n, backward, stream);
}

ssd_status check_norm(ssd_dtype io, ssd_dtype res, int64_t rows, int64_t dim) {
    if ((io != SSD_F32 && io != SSD_BF16) || (res != SSD_F32 && res != SSD_BF16)) return SSD_ERR_INVALID_ARG;
    if (rows < 1 || dim < 1) return SSD_ERR_INVALID_ARG;
    if (io == SSD_F32 && res != SSD_F32) return SSD_ERR_UNSUPPORTED;
    if (dim > kMaxDim || rows >= (1ll << 31)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Every tensor starts on its element's boundary (false: unsupported); *align: 16 where every
// row of every tensor starts on 16 bytes, 2 where on two elements, else 1.
bool norm_alignment(ssd_dtype io, ssd_dtype res, int64_t dim, std::initializer_list<int64_t> strides,
                    std::initializer_list<const void*> io_ptrs, std::initializer_list<const void*> res_ptrs,
                    std::initializer_list<const void*> weights, int* align) {
    const int64_t v = io == SSD_BF16 ? 8 : 4;
    bool wide = dim % v == 0, two = dim % 2 == 0, ok = true;
    for (int64_t s : strides) wide = wide && s % v == 0, two = two && s % 2 == 0;
    auto look = [&](const void* q, size_t element) {
        wide = wide && aligned_to(q, 16);
        two = two && aligned_to(q, 2 * element);
        ok = ok && aligned_to(q, element);
    };
    for (const void* q : io_ptrs) look(q, io == SSD_BF16 ? 2 : 4);
    for (const void* q : res_ptrs) look(q, res == SSD_BF16 ? 2 : 4);
    for (const void* q : weights) look(q, 4);
    *align = wide ? 16 : two ? 2 : 1;
    return ok;
}

// Calls f with a value of the io type and one of the residual's type.
template <typename F>
ssd_status with_types(ssd_dtype io, ssd_dtype res, F f) {
    if (io == SSD_F32) return f(float(), float());
    return res == SSD_F32 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_block_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    using namespace ssd;
    if (check_norm(SSD_F32, SSD_F32, rows, dim) != SSD_OK) return 0;
    // the largest grid of any plan: at most 32 warps of one row each per SM
    const int64_t parts = std::min<int64_t>(rows + 8, 32ll * device_sms());
    return align_up(static_cast<size_t>(parts) * 2 * dim * sizeof(float), kWorkspaceAlign);
}

ssd_status ssd_block_norm(ssd_dtype io_dtype, ssd_dtype residual_dtype, int64_t rows, int64_t dim, const void* y,
                          int64_t y_row_stride, const void* residual, const void* z, int64_t z_row_stride,
                          const float* post_weight, const float* scale, const float* pre_weight, float eps,
                          void* residual_out, void* out, float* rstd, void* stream) {
    using namespace ssd;
    const ssd_status st = check_norm(io_dtype, residual_dtype, rows, dim);
    if (st != SSD_OK) return st;
    if (!y || !residual_out || (pre_weight && !out)) return SSD_ERR_INVALID_ARG;
    if (y_row_stride < dim || (z && z_row_stride < dim) || !(eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    int align;
    if (!norm_alignment(io_dtype, residual_dtype, dim, {y_row_stride, z ? z_row_stride : 0}, {y, z, out},
                        {residual, residual_out}, {post_weight, scale, pre_weight}, &align) ||
        !aligned_to(rstd, 8))
        return SSD_ERR_UNSUPPORTED;
    return with_types(io_dtype, residual_dtype, [&](auto t, auto tr) {
        using T = decltype(t);
        using TR = decltype(tr);
        NormParams<T, TR> p{};
        p.y = static_cast<const T*>(y), p.z = static_cast<const T*>(z), p.out = static_cast<T*>(out);
        p.res = static_cast<const TR*>(residual), p.res_out = static_cast<TR*>(residual_out);
        p.post = post_weight, p.scale = scale, p.pre = pre_weight;
        p.rstd = reinterpret_cast<float2*>(rstd);
        p.rows = rows, p.ys = y_row_stride, p.zs = z_row_stride, p.dim = static_cast<int>(dim), p.eps = eps;
        NormPlan n;
        return launch_norm(p, align, false, &n, static_cast<cudaStream_t>(stream));
    });
}

ssd_status ssd_block_norm_bwd(ssd_dtype io_dtype, ssd_dtype residual_dtype, int64_t rows, int64_t dim, const void* dout,
                              int64_t dout_row_stride, const void* dresidual_out, const void* y, int64_t y_row_stride,
                              const void* residual, const void* z, int64_t z_row_stride, const float* post_weight,
                              const float* scale, const float* pre_weight, const float* rstd, void* dy,
                              void* dresidual, void* dz, float* dpost_weight, float* dscale, float* dpre_weight,
                              void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssd;
    const ssd_status st = check_norm(io_dtype, residual_dtype, rows, dim);
    if (st != SSD_OK) return st;
    if (!y || !rstd || !dy || (z && !dz) || (dpost_weight && !post_weight) || (dscale && !scale) ||
        (dpre_weight && !pre_weight) || (pre_weight && !dout) || (!dout && !dresidual_out))
        return SSD_ERR_INVALID_ARG;
    if (y_row_stride < dim || (z && z_row_stride < dim) || (dout && dout_row_stride < dim)) return SSD_ERR_INVALID_ARG;
    int align;
    if (!norm_alignment(io_dtype, residual_dtype, dim,
                        {y_row_stride, z ? z_row_stride : 0, dout ? dout_row_stride : 0}, {y, z, dout, dy, dz},
                        {residual, dresidual_out, dresidual},
                        {post_weight, scale, pre_weight, dpost_weight, dscale, dpre_weight}, &align) ||
        !aligned_to(rstd, 8))
        return SSD_ERR_UNSUPPORTED;
    if (workspace_bytes < ssd_block_norm_bwd_workspace_bytes(rows, dim) || !workspace ||
        !aligned_to(workspace, kWorkspaceAlign))
        return SSD_ERR_WORKSPACE;
    return with_types(io_dtype, residual_dtype, [&](auto t, auto tr) {
        using T = decltype(t);
        using TR = decltype(tr);
        NormParams<T, TR> p{};
        p.y = static_cast<const T*>(y), p.z = static_cast<const T*>(z);
        p.dout = pre_weight ? static_cast<const T*>(dout) : nullptr;
        p.res = static_cast<const TR*>(residual), p.dres = static_cast<const TR*>(dresidual_out);
        p.dy = static_cast<T*>(dy), p.dz = static_cast<T*>(dz), p.dres_in = static_cast<TR*>(dresidual);
        p.post = post_weight, p.scale = scale, p.pre = pre_weight;
        p.rstd = reinterpret_cast<float2*>(const_cast<float*>(rstd));
        p.sums = static_cast<float*>(workspace);
        p.rows = rows, p.ys = y_row_stride, p.zs = z_row_stride, p.dos = dout_row_stride;
        p.dim = static_cast<int>(dim);
        NormPlan n;
        const ssd_status rc = launch_norm(p, align, true, &n, static_cast<cudaStream_t>(stream));
        if (rc != SSD_OK) return rc;
        block_norm_sums<<<static_cast<unsigned>((2 * dim + 31) / 32), 32 * kSumRows, 0,
                          static_cast<cudaStream_t>(stream)>>>(p.sums, n.parts, p.dim,
                                                               post_weight, scale, dpost_weight, dscale, dpre_weight);
        note_launches(1);
        return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    });
}

}  // extern "C"
