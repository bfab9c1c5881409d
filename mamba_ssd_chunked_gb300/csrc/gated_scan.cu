// The per-channel gated linear recurrence (include/ssd.h, ssd_gated_scan):
//
//   delta = softplus(dt + dt_bias)          a = e^{delta A}, 0 where seq_idx changes
//   h_t   = a_t h_{t-1} + delta_t x_t       y_t = h_t + D x_t
//
// and its gradient. With g_t = dL/dh_t = dy_t + a_{t+1} g_{t+1}:
//
//   dx_t = delta_t g_t + D dy_t             ddelta_t = g_t x_t + A a_t g_t h_{t-1}
//   dt'  = ddelta sigmoid(dt + dt_bias)     dA = sum delta a g h_{t-1}   dD = sum dy x
//
// Both directions are scans of affine maps s -> P s + q, which compose
// associatively: (P2, q2) o (P1, q1) = (P2 P1, P2 q1 + q2). One pass over the
// data: a CTA takes a tile of kWarps runs of tokens by 64 channels, a thread one
// run (kRun consecutive tokens) of two channels.
//   1. each thread folds its own tokens into (P, q);
//   2. the CTA's warps (consecutive runs) exchange theirs through shared memory, and
//      the tile's own map is published in global memory;
//   3. the value entering the tile is the group's carry followed by the maps of
//      the earlier tiles of the group (kGroup tiles along time), so a tile never
//      waits for its predecessor's result, only for its predecessors' inputs; the
//      last tile of a group publishes the next group's carry. The maps are
//      always composed in the same order: results do not depend on timing;
//   4. each thread applies what enters its run and writes its outputs.
// Published words start out as 0xFFFFFFFF, a NaN that no fp32 instruction makes, and
// are polled until they differ: a word's arrival is its own flag. The waits are
// bounded (an abort word ends all of them).
//
// The CTAs are persistent and take tiles in time order through a ticket, so
// whatever a tile waits for is running or done. All warps but one compute; that one does
// step 3 for the tile while they do step 1, publishes, and looks up the tile after
// the next, so a tile costs the computing warps one barrier. Inputs come through
// shared memory in two stages: each warp copies its own rows of the next tile
// while it works on this one.
//
// The backward pass runs the same scan over g from the last tile to the first,
// and rebuilds h inside a tile from the state that the forward pass saved at
// the tile's start. Sums over tokens (dA, d dt_bias, dD) leave each tile as one
// row and are added up by a second kernel, always in the same order.
#include <algorithm>
#include <cstddef>
#include <initializer_list>
#include <type_traits>

#include "elem.cuh"
#include "ptx.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using elem::Pack;
using elem::Vals;
using Pair = Vals<2>;  // a thread's two channels

// Computing warps per CTA (consecutive runs of tokens; one more warp guides them) and
// CTAs per SM. Registers hold 16 warps per SM either way. One CTA of 15 + 1 warps
// against two of 7 + 1, bf16, when the choice was made: 1 x 131072 x 4096 forward 701 against 918 us (longer
// tiles: fewer steps along a sequence), 4 x 4096 x 5120 forward 121 against 117 us,
// with the backward 366 against 360 us. The fp32 backward's stages would not fit with 15; with 7 they and
// the exchange take 117 KB (122 off 16 bytes), so only one of its two CTAs is on an SM at a time (tiles go
// by ticket, so the second half of the grid finds what is left).
template <typename T>
constexpr int kWarps = sizeof(T) == 2 ? 15 : 7;
template <typename T>
constexpr int kThreads = 32 * (kWarps<T> + 1);
template <typename T>
constexpr int kCtasPerSm = sizeof(T) == 2 ? 1 : 2;
constexpr int kGroup = 4;       // tiles between carries (a guide polls up to three maps and a carry)
// Tokens per thread: two fp32 values per token in registers in the forward, four in the backward.
template <typename T>
constexpr int kRunFwd = sizeof(T) == 2 ? 16 : 8;
constexpr int kRunBwd = 8;
template <typename T>
constexpr int kState = kRunBwd * kWarps<T>;  // tokens between saved states: the backward's tile

template <typename T>
struct ScanParams {
    const T* x;
    const T* dt;
    const T* dy;  // backward
    long long xs, dts, dys, dxs, ddts;  // row strides
    const float* bias;
    const float* A;
    const float* D;     // nullable
    const float* init;  // forward: state before the first token; backward: gradient of the final state (nullable)
    const int* seq;     // nullable
    T* y;               // forward: y (dense); backward: dx
    T* ddt;
    float* fin;         // forward: final state; backward: gradient of the initial state (nullable)
    float* states;      // [batch, ceil(L / kState<T>), dim]: state entering each kState<T> tokens (forward: nullable)
    float* sums;        // backward: [batch * tiles, 3, dim]
    // exchange between tiles, all words kUnset before the launch (tiles > 1)
    uint32_t* ticket;   // [0] ticket, less one; [1] anything but kUnset: give up waiting
    uint32_t* maps;     // [tiles, batch, pitch, 2]: P of a thread's channels, then q
    uint32_t* carry;    // [groups, batch, pitch]
    unsigned* status;
    unsigned long long wait_ns;
    long long L, dim, pitch;  // pitch: channels between sequences in maps and carry (dim, made even)
    int batch, tiles, tiles_c, chains;  // tiles along time; tiles along the channels; batch * tiles_c
};

constexpr uint32_t kUnset = 0xFFFFFFFFu;
constexpr unsigned long long kOwnWaitNs = 2000000000ull;  // waits within a CTA, beyond those for other CTAs

// N consecutive published words
template <int N>
__device__ __forceinline__ void load_words(const uint32_t* src, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(src)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(src) : "memory");
    else
        w[0] = ptx::ld_relaxed_gpu(src);
}
template <int N>
__device__ __forceinline__ bool all_set(const uint32_t (&w)[N]) {
    bool set = true;
#pragma unroll
    for (int i = 0; i < N; ++i) set = set && w[i] != kUnset;
    return set;
}
template <int N>
__device__ __forceinline__ void publish(uint32_t* dst, const uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3])
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};" ::"l"(dst), "r"(w[0]), "r"(w[1]) : "memory");
    else
        ptx::st_relaxed_gpu(dst, w[0]);
}
// Two values as words and back
__device__ __forceinline__ void to_words(Pair a, uint32_t* w) {
    w[0] = __float_as_uint(a.get(0)), w[1] = __float_as_uint(a.get(1));
}
__device__ __forceinline__ Pair from_words(const uint32_t* w) {
    return Pair::make(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

// A thread's channels of an fp32 vector; `both`: the second one exists too.
template <bool kAny>
__device__ __forceinline__ Pair load_pair(const float* p, bool both) {
    if constexpr (kAny)
        return Pair::make(p[0], both ? p[1] : 0.f);
    else
        return Pair::load(p);
}
template <bool kAny>
__device__ __forceinline__ void store_pair(float* p, Pair v, bool both) {
    if constexpr (kAny) {
        p[0] = v.get(0);
        if (both) p[1] = v.get(1);
    } else {
        v.store(p);
    }
}
// and of an output row
template <typename T, bool kAny>
__device__ __forceinline__ void store_out(T* p, Pair v, bool both) {
    if (!kAny || (both && (reinterpret_cast<uintptr_t>(p) & (2 * sizeof(T) - 1)) == 0)) {
        elem::store_vals<T, 2>(p, v);
    } else {
        elem::store_vals<T, 1>(p, {v.get(0)});
        if (both) elem::store_vals<T, 1>(p + 1, {v.get(1)});
    }
}

struct Map {
    Pair P, q;
};
// `then` after `first`
__device__ __forceinline__ Map compose(Map then, Map first) {
    return {elem::mul(then.P, first.P), elem::fma(then.P, first.q, then.q)};
}
__device__ __forceinline__ Pair apply(Map m, Pair s) {
    return elem::fma(m.P, s, m.q);
}
// Packed sequences (kSeq): where one begins nothing of the one before passes. A zero in the place of
// the decay would not do: zero times an infinity or a NaN of the other sequence is NaN. A run with such a
// token (Slot::cut_runs) maps every s to q, and maps are composed from the last such run on; a published
// tile's P is then -0, which no product of decays is (none of them is negative). The guide looks seq_idx up
// with the tile. 4 x 4096 x 5120 (bf16) in sequences of 300 tokens: forward 135 us (125 unpacked), backward 279 (255);
// 1 x 131072 x 4096: 792 (731) and 1727 (1573).
__device__ __forceinline__ Pair cut_P() { return Pair::splat(-0.f); }
__device__ __forceinline__ bool is_cut(Pair P) { return __float_as_uint(P.get(0)) == 0x80000000u; }  // (both channels alike)
// f(std::true_type) or f(std::false_type); kMay: `yes` may be true
template <bool kMay, typename F>
__device__ __forceinline__ void with(bool yes, F f) {
    if (kMay && yes)
        f(std::true_type{});
    else
        f(std::false_type{});
}
// and with two conditions
template <bool kMay, typename F>
__device__ __forceinline__ void with(bool yes, bool second, F f) {
    with<kMay>(yes, [&](auto a) { with<true>(second, [&](auto b) { f(a, b); }); });
}

// A tile as the computing warps see it, looked up three tiles ahead by the guiding warp.
struct Slot {
    int step, b;     // step counts tiles in scan order; -1: no more tiles
    long long c0;    // first channel
    Pair A[32], bias[32], D[32], state[32];  // (state: backward only)
    // packed sequences: a bit for each token of the tile that begins one, and for each run with such a token
    uint32_t begins[8], cut_runs;
};

// Live at once: the finished tile whose sums are stored, the current one, and three ahead.
constexpr int kSlots = 8;

template <typename T>
struct Exchange {
    Map run[2][kWarps<T>][32];  // the warps' maps
    Pair enter[2][32];       // what enters the tile
    // Every computing warp's run of tile i is there; what enters it is: phase i / 2 of
    // barrier i % 2. (One barrier could complete two phases before a slow warp has seen
    // the first: the guide may let a tile be entered before it has seen the runs.)
    uint64_t runs_ready[2], enter_ready[2];
    Slot slot[kSlots];
    // backward
    Pair f[2][kWarps<T>][32];        // the forward maps' constants (their P is run's)
    Pair sums[2][3][kWarps<T>][32];  // dA, d dt_bias, dD
};

// The last of the runs before `run`, and the first after it, that is among `cuts` (-1: none).
__device__ __forceinline__ int last_before(uint32_t cuts, int run) { return 31 - __clz(cuts & ((1u << run) - 1u)); }
__device__ __forceinline__ int first_after(uint32_t cuts, int run) {
    const int ahead = __ffs(cuts >> run >> 1);
    return ahead == 0 ? -1 : run + ahead;
}

// One thread's channels. A lane past the last channel computes on whatever is there and
// writes nothing.
struct Place {
    int warp, lane, step, b;
    bool live, both;     // its first channel exists, its second too
    long long c, own;    // the first channel; its place in a [batch, dim] tensor
    long long cell;      // and among the published words
};
template <typename T, bool kAny>
__device__ __forceinline__ Place place_in(const ScanParams<T>& p, const Slot& t) {
    Place w;
    w.warp = threadIdx.x >> 5, w.lane = threadIdx.x & 31;
    w.step = t.step, w.b = t.b;
    w.c = t.c0 + w.lane * 2;
    w.live = w.c < p.dim, w.both = kAny ? w.c + 1 < p.dim : w.live;
    w.own = w.b * p.dim + w.c, w.cell = kAny ? w.b * p.pitch + w.c : w.own;
    return w;
}

// ---------------------------------------------------------------- the guiding warp
// Tile `unit`, looked up.
template <typename T, bool kAny, bool kForward, bool kSeq>
struct Lookup {
    static constexpr int kRun = kForward ? kRunFwd<T> : kRunBwd, kTile = kRun * kWarps<T>, kWords = (kTile + 31) / 32;
    int step, b;
    long long c0;
    Pair A, bias, D, state;
    uint32_t begins[kWords], cut_runs;
    __device__ __forceinline__ void fetch(const ScanParams<T>& p, int unit, int lane) {
        step = -1;
        if (unit >= p.chains * p.tiles) return;
        step = unit / p.chains;
        const int chain = unit - step * p.chains;
        b = chain / p.tiles_c;
        c0 = static_cast<long long>(chain - b * p.tiles_c) * 64;
        const long long c = c0 + lane * 2;
        const bool both = c + 1 < p.dim;
        A = bias = D = state = Pair::splat(0.f);
        if (c < p.dim) {
            A = load_pair<kAny>(p.A + c, both);
            bias = load_pair<kAny>(p.bias + c, both);
            if (p.D) D = load_pair<kAny>(p.D + c, both);
            if (!kForward)
                state = load_pair<kAny>(p.states + (static_cast<long long>(b) * p.tiles + (p.tiles - 1 - step)) * p.dim + c, both);
        }
        if constexpr (kSeq) {
            const long long t0 = static_cast<long long>(kForward ? step : p.tiles - 1 - step) * kTile;
            const int* seq = p.seq + b * p.L + t0;
            int here[kWords], last[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const int i = k * 32 + lane;
                here[k] = last[k] = 0;
                if (i < kTile && t0 + i > 0 && t0 + i < p.L) here[k] = __ldg(seq + i), last[k] = __ldg(seq + i - 1);
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) begins[k] = __ballot_sync(0xffffffffu, here[k] != last[k]);
            cut_runs = 0u;
#pragma unroll
            for (int k = 0; k < kWarps<T>; ++k)
                if (begins[k * kRun / 32] >> k * kRun % 32 & ((1u << kRun) - 1u)) cut_runs |= 1u << k;
        }
    }
    __device__ __forceinline__ void store(Slot& t, int lane) const {
        if (lane == 0) t.step = step, t.b = b, t.c0 = c0;
        t.A[lane] = A, t.bias[lane] = bias, t.D[lane] = D;
        if (!kForward) t.state[lane] = state;
        if constexpr (kSeq) {
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < kWords; ++k) t.begins[k] = begins[k];
                t.cut_runs = cut_runs;
            }
        }
    }
};

// What enters a tile in scan order: the group's carry (or the scan's initial value),
// then the group's earlier maps.
template <typename T, bool kAny>
struct Incoming {
    uint32_t carry[2], m[kGroup - 1][4];
    const uint32_t *from, *src;
    long long stride;
    int group, n;
    bool live;
    __device__ __forceinline__ void start(const ScanParams<T>& p, const Place& w) {
        const long long cells = static_cast<long long>(p.batch) * p.pitch;
        group = w.step / kGroup, n = w.step % kGroup, live = w.live;
        src = p.maps + (static_cast<long long>(group) * kGroup * cells + w.cell) * 2;
        from = p.carry + group * cells + w.cell;
        stride = cells * 2;
        carry[0] = kUnset;
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k) m[k][0] = kUnset;
        read();
    }
    // loads what has not arrived yet
    __device__ __forceinline__ void read() {
        if (!live) return;
        if (group > 0 && (carry[0] == kUnset || !all_set(carry))) load_words(from, carry);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (k < n && (m[k][0] == kUnset || !all_set(m[k]))) load_words(src + k * stride, m[k]);
    }
    __device__ __forceinline__ bool there() const {
        bool yes = !live || group == 0 || all_set(carry);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (live && k < n) yes = yes && all_set(m[k]);
        return yes;
    }
    template <bool kSeq>
    __device__ __forceinline__ Pair value(const ScanParams<T>& p, const Place& w) const {
        Pair s = Pair::splat(0.f);
        if (!live) return s;
        if (group > 0)
            s = from_words(carry);
        else if (p.init)
            s = load_pair<kAny>(p.init + w.own, w.both);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (k < n) {
                const Map map{from_words(m[k]), from_words(m[k] + 2)};
                s = kSeq && is_cut(map.P) ? map.q : apply(map, s);
            }
        return s;
    }
};

// Publishes the tile's map for the later tiles of its group, or the next group's carry.
template <typename T, bool kForward, bool kSeq>
__device__ __forceinline__ void publish_tile(const ScanParams<T>& p, const Map (*run)[32], uint32_t cuts, Pair enter,
                                             const Place& w) {
    if (w.step + 1 >= p.tiles || !w.live) return;  // nobody reads it
    auto nth = [](int k) { return kForward ? k : kWarps<T> - 1 - k; };  // in scan order
    // what the runs before the last with a cut do does not count
    const int from = !kSeq || cuts == 0u ? 0 : nth(kForward ? 31 - __clz(cuts) : __ffs(cuts) - 1);
    Map m = run[nth(from)][w.lane];
#pragma unroll
    for (int k = 1; k < kWarps<T>; ++k)
        if (!kSeq || k > from) m = compose(run[nth(k)][w.lane], m);
    if (kSeq && cuts != 0u) m.P = cut_P();
    const long long cells = static_cast<long long>(p.batch) * p.pitch;
    if (w.step % kGroup == kGroup - 1) {
        uint32_t o[2];
        to_words(kSeq && cuts != 0u ? m.q : apply(m, enter), o);
        publish(p.carry + (w.step / kGroup + 1) * cells + w.cell, o);
    } else {
        uint32_t o[4];
        to_words(m.P, o), to_words(m.q, o + 2);
        publish(p.maps + (w.step * cells + w.cell) * 2, o);
    }
}

// One row of a finished backward tile's sums.
template <typename T, bool kAny>
__device__ __forceinline__ void store_sums(const ScanParams<T>& p, const Exchange<T>& ex, const Place& w, int turn) {
    if (!w.live) return;
    float* out = p.sums + (static_cast<long long>(w.b) * p.tiles + (p.tiles - 1 - w.step)) * 3 * p.dim + w.c;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        Pair s = ex.sums[turn][i][0][w.lane];
#pragma unroll
        for (int o = 1; o < kWarps<T>; ++o) s = elem::add(s, ex.sums[turn][i][o][w.lane]);
        store_pair<kAny>(out + i * p.dim, s, w.both);
    }
}

template <typename T, bool kAny, bool kForward, bool kSeq>
__device__ __forceinline__ void guide(const ScanParams<T>& p, Exchange<T>& ex) {
    const int lane = threadIdx.x & 31;
    // The next ticket; a sequence of one tile has nothing to take in order.
    int nth = 0;
    auto ask = [&] {
        if (p.tiles == 1) return nth++ == 0 ? static_cast<int>(blockIdx.x) : p.chains;
        return lane == 0 ? static_cast<int>(atomicAdd(p.ticket, 1u) + 1u) : 0;
    };
    Lookup<T, kAny, kForward, kSeq> next;
    Incoming<T, kAny> in;
    for (int k = 0; k < 3; ++k) {
        next.fetch(p, __shfl_sync(0xffffffffu, ask(), 0), lane);
        next.store(ex.slot[k], lane);
        __syncthreads();
    }
    unsigned i = 0;
    for (; ex.slot[i % kSlots].step >= 0; ++i) {
        const Place w = place_in<T, kAny>(p, ex.slot[i % kSlots]);
        const uint32_t cuts = kSeq ? ex.slot[i % kSlots].cut_runs : 0u;
        const int ticket = ask();  // in flight until the tile is done
        in.start(p, w);
        // The map goes out as soon as the runs are there, whatever this tile still waits
        // for; only a group's last tile publishes a carry, which needs what enters.
        const bool last = w.step % kGroup == kGroup - 1;
        bool runs = false, entered = false;
        Pair enter = Pair::splat(0.f);
        uint64_t since = 0;
        unsigned spins = 0;
        while (!runs || !entered) {
            for (int k = 0; k < 8 && !runs; ++k) {
                runs = ptx::mbar_test_wait(&ex.runs_ready[i & 1], i >> 1 & 1);
                runs = __any_sync(0xffffffffu, runs);
                if (runs && !last) publish_tile<T, kForward, kSeq>(p, ex.run[i & 1], cuts, enter, w);
            }
            if (!entered && __all_sync(0xffffffffu, in.there())) {
                enter = in.template value<kSeq>(p, w);
                ex.enter[i & 1][lane] = enter;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&ex.enter_ready[i & 1]);
                entered = true;
            }
            if (runs && entered) break;
            // the limit, and now and then whether another wait has given up
            const uint64_t now = ptx::globaltimer_ns();
            if (since == 0) since = now;
            bool give_up = p.tiles > 1 && !entered && (++spins & 15u) == 0 && ptx::ld_relaxed_gpu(p.ticket + 1) != kUnset;
            if (!entered && now - since > p.wait_ns) {
                if (p.tiles > 1) ptx::st_relaxed_gpu(p.ticket + 1, 0u);
                atomicOr(p.status, 1u);
                give_up = true;
            }
            if (__any_sync(0xffffffffu, give_up)) in.n = in.group = 0;  // nothing more to wait for
            if (__any_sync(0xffffffffu, now - since > p.wait_ns + kOwnWaitNs)) {  // the computing warps have gone
                if (lane == 0) atomicOr(p.status, 1u);
                return;
            }
            if (!entered) in.read();
        }
        if (last) publish_tile<T, kForward, kSeq>(p, ex.run[i & 1], cuts, enter, w);
        next.fetch(p, __shfl_sync(0xffffffffu, ticket, 0), lane);
        next.store(ex.slot[(i + 3) % kSlots], lane);
        if (!kForward && i > 0) store_sums<T, kAny>(p, ex, place_in<T, kAny>(p, ex.slot[(i - 1) % kSlots]), (i - 1) & 1);
    }
    if (!kForward && i > 0) {
        __syncthreads();
        store_sums<T, kAny>(p, ex, place_in<T, kAny>(p, ex.slot[(i - 1) % kSlots]), (i - 1) & 1);
    }
}

// ---------------------------------------------------------------- the computing warps
// This warp's run is in shared memory; waits for the other warps' and for what enters the tile.
// The guide's own wait ends after p.wait_ns, so these end; false (never seen): leave.
template <typename T>
__device__ __forceinline__ bool wait_enter(const ScanParams<T>& p, Exchange<T>& ex, int nth) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&ex.runs_ready[nth & 1]);
    const uint32_t phase = nth >> 1 & 1;
    const bool ok = ptx::mbar_wait(&ex.runs_ready[nth & 1], phase, p.wait_ns + kOwnWaitNs) &&
                    ptx::mbar_wait(&ex.enter_ready[nth & 1], phase, p.wait_ns + kOwnWaitNs);
    if (!ok) atomicOr(p.status, 1u);
    return __all_sync(0xffffffffu, ok);
}

// Elements of a 16-byte granule, and from one row of a stage to the next. Copies start on and
// consist of granules: a row that starts anywhere arrives as the granules that hold it, one more
// than its 64 elements fill, and begins row_shift elements into its slot. 4 x 4096 x 5121 (bf16),
// forward and forward + backward: 184 and 532 us; in words of 4 bytes 222 and 652; in elements, one channel
// per thread, 437 and 1214; x 5120, whose rows all start on 16 bytes, 125 and 380.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));
template <typename T, bool kAny>
constexpr int kPitch = kAny ? 64 + kVec<T> : 64;
template <typename T, bool kAny>
__device__ __forceinline__ unsigned row_shift(const T* row) {
    return kAny ? static_cast<unsigned>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (kVec<T> - 1) : 0;
}

// This warp's rows of one input of a tile into shared memory, n tokens from src on. Channels
// past dim hold anything. (A granule that is half outside a row lies in the same allocation:
// allocations start and end on 16 bytes.)
template <typename T, bool kAny, int kRun>
__device__ __forceinline__ void copy_rows(T* dst, const T* src, long long stride, int n, long long c0, long long dim,
                                          int lane) {
    constexpr int kRow = 64 / kVec<T>, kRows = 32 / kRow;
    const int end = static_cast<int>(min(dim - c0, 64ll));  // of a row's elements
    auto granule = [&](int r, int i) {
        const T* row = src + r * stride;
        const int at = i * kVec<T> - static_cast<int>(row_shift<T, kAny>(row));
        if (r < n && at < end) ptx::cp_async<16>(ptx::smem_u32(dst + r * kPitch<T, kAny> + i * kVec<T>), row + at);
    };
#pragma unroll
    for (int r = 0; r < kRun; r += kRows) granule(r + lane / kRow, lane % kRow);
    if (kAny && lane < kRun) granule(lane, kRow);
}

// One input's rows in shared memory as this thread reads them.
template <typename T, bool kAny>
struct Rows {
    const T* at;
    unsigned shift, step;  // (of a row's start only the low bits count)
    // stage: the run's rows; row: its first row in global memory
    __device__ __forceinline__ Rows(const T* stage, const T* row, long long stride, int lane)
        : at(stage + 2 * lane), shift(row_shift<T, kAny>(row)), step(static_cast<unsigned>(stride)) {}
    __device__ __forceinline__ Pair operator()(int r) const {
        const T* p = at + r * kPitch<T, kAny>;
        if constexpr (kAny) {
            p += (shift + r * step) & (kVec<T> - 1);
            Pack<T, 1> a, b;
            a.load_plain(p), b.load_plain(p + 1);
            return Pair::make(elem::unpack<T, 1>(a).f, elem::unpack<T, 1>(b).f);
        } else {
            Pack<T, 2> k;
            k.load_plain(p);
            return elem::unpack<T, 2>(k);
        }
    }
};

// load(slot, stage) copies this warp's inputs of a tile, body(slot, nth) works on the CTA's nth tile
// and says whether to go on.
template <typename T, bool kForward, typename Load, typename Body>
__device__ __forceinline__ void walk_tiles(Exchange<T>& ex, Load load, Body body) {
    __syncthreads();  // the first slot
    if (ex.slot[0].step >= 0) load(ex.slot[0], 0);
    ptx::cp_async_commit();
    __syncthreads();  // the second and the third
    __syncthreads();
    unsigned i = 0;
    for (; ex.slot[i % kSlots].step >= 0; ++i) {
        __syncwarp();  // every lane has read the stage that is filled now
        const Slot& next = ex.slot[(i + 1) % kSlots];
        if (next.step >= 0) load(next, (i + 1) & 1);
        ptx::cp_async_commit();
        ptx::cp_async_wait<1>();
        __syncwarp();  // a warp reads what its own lanes copied
        if (!body(ex.slot[i % kSlots], i)) return;
    }
    if (!kForward && i > 0) __syncthreads();  // the last tile's sums
}

// Bits r < kRun set where a sequence begins with token r of this warp's run.
template <int kRun, bool kSeq>
__device__ __forceinline__ uint32_t begins_in(const Slot& t, int warp) {
    return kSeq ? t.begins[warp * kRun / 32] >> warp * kRun % 32 & ((1u << kRun) - 1u) : 0u;
}

// The decay e^(delta A), from delta and A_in = decay_A(A). The forward and the decode step of bf16 io take the
// hardware's 2^x as it is, with A in units of log 2 (final states are 4e-7 off, far inside y's rounding; exp_near
// costs the forward 13 % of its time); fp32 io and the gradients, whose states and sums over tokens keep such
// errors, do not (4000 fp32 decode steps with decays down to 1 - 1/2000: 1e-5 off by 2^x, 1.4e-6 so).
template <typename T, int V>
__device__ __forceinline__ Vals<V> decay_A(Vals<V> A) {
    return sizeof(T) == 2 ? elem::mul(A, Vals<V>::splat(elem::kLog2e)) : A;
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> decay(Vals<V> A_in, Vals<V> delta) {
    if constexpr (sizeof(T) == 2)
        return elem::exp2_fast<V>(elem::mul(A_in, delta));
    else
        return elem::exp_near<V>(elem::mul(A_in, delta));
}

// kWhole: every token of the tile exists.
template <typename T, bool kAny, bool kSeq, bool kWhole>
__device__ __forceinline__ bool forward_tile(const ScanParams<T>& p, Exchange<T>& ex, const Slot& t, const T* sx,
                                             const T* sd, int nth) {
    using L = Pair;
    constexpr int kRun = kRunFwd<T>;
    const int turn = nth & 1;
    const Place w = place_in<T, kAny>(p, t);
    const long long t0 = static_cast<long long>(w.step) * (kRun * kWarps<T>) + w.warp * kRun;
    const long long row0 = w.b * p.L + t0;
    const int n = kWhole ? kRun : static_cast<int>(min(max(p.L - t0, 0ll), static_cast<long long>(kRun)));
    const Rows<T, kAny> x(sx, p.x + row0 * p.xs + t.c0, p.xs, w.lane), dt(sd, p.dt + row0 * p.dts + t.c0, p.dts, w.lane);
    // per token: decay and input; then the run's map token by token: h_t from a zero state, decay product P_t
    L h[kRun], P[kRun];
    {
        const L A = decay_A<T, 2>(t.A[w.lane]), bias = t.bias[w.lane];
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            P[r] = L::splat(1.f), h[r] = L::splat(0.f);
            if (kWhole || r < n) {
                L u;
                const L delta = elem::softplus<2>(elem::add(dt(r), bias), &u);
                P[r] = decay<T, 2>(A, delta);
                h[r] = elem::mul(delta, x(r));
            }
        }
    }
    const uint32_t cut = begins_in<kRun, kSeq>(t, w.warp);
    auto begun = [&](int r) { return (cut & ((2u << r) - 1u)) != 0u; };  // a sequence, by token r of the run
    with<kSeq>(cut != 0u, [&](auto some) {
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            if (r > 0 && !(some.value && (cut >> r & 1u))) h[r] = elem::fma(P[r], h[r - 1], h[r]);
            if (r > 0) P[r] = elem::mul(P[r], P[r - 1]);  // (past a cut: not used)
        }
    });
    const Map(*run)[32] = ex.run[turn];
    ex.run[turn][w.warp][w.lane] = {P[kRun - 1], h[kRun - 1]};
    if (!wait_enter(p, ex, nth)) return false;
    if (!w.live) return true;
    const int last = kSeq ? last_before(t.cut_runs, w.warp) : -1;
    L s = last >= 0 ? run[last][w.lane].q : ex.enter[turn][w.lane];
    for (int k = last + 1; k < w.warp; ++k) s = apply(run[k][w.lane], s);
    // the state entering token t0 + keep_at is saved (kState<T> may end inside a run)
    int keep_at = -1;
    float* keep = nullptr;
    if (p.states) {
        const long long nth = (t0 + kState<T> - 1) / kState<T>, per = (p.L + kState<T> - 1) / kState<T>;
        if (nth < per) keep_at = static_cast<int>(nth * kState<T> - t0);
        keep = p.states + (w.b * per + nth) * p.dim + w.c;
        if (keep_at == 0) store_pair<kAny>(keep, s, w.both);
    }
    const L D = t.D[w.lane];
    with<kSeq>(cut != 0u, p.D != nullptr, [&](auto some, auto skip) {  // (zero times an infinite x is no skip)
        T* py = p.y + row0 * p.dim + w.c;
#pragma unroll
        for (int r = 0; r < kRun; ++r, py += p.dim) {
            if (kWhole || r < n) {
                const L ht = some.value && begun(r) ? h[r] : elem::fma(P[r], s, h[r]);
                store_out<T, kAny>(py, skip.value ? elem::fma(D, x(r), ht) : ht, w.both);
                if (r + 1 < kRun && r + 1 == keep_at) store_pair<kAny>(keep, ht, w.both);
                if ((!kWhole || r == kRun - 1) && p.fin && t0 + r == p.L - 1) store_pair<kAny>(p.fin + w.own, ht, w.both);
            }
        }
    });
    return true;
}

template <typename T, bool kAny>
__host__ __device__ constexpr int stage_bytes(int run, int inputs) {
    return inputs * run * kWarps<T> * kPitch<T, kAny> * static_cast<int>(sizeof(T));
}

template <typename T, bool kAny, bool kSeq>
__global__ void __launch_bounds__(kThreads<T>, kCtasPerSm<T>) gated_scan_fwd(const ScanParams<T> p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kRun = kRunFwd<T>, kTile = kRun * kWarps<T>, kElems = kTile * kPitch<T, kAny>;
    Exchange<T>& ex = *reinterpret_cast<Exchange<T>*>(smem + 2 * stage_bytes<T, kAny>(kRun, 2));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k) {
            ptx::mbar_init(&ex.runs_ready[k], kWarps<T>);
            ptx::mbar_init(&ex.enter_ready[k], 1);
        }
        ptx::fence_mbar_init();
    }
    if (warp == kWarps<T>) {
        guide<T, kAny, true, kSeq>(p, ex);
        return;
    }
    T* mine = reinterpret_cast<T*>(smem) + warp * kRun * kPitch<T, kAny>;  // this warp's rows
    walk_tiles<T, true>(
        ex,
        [&](const Slot& t, int stage) {
            const long long t0 = static_cast<long long>(t.step) * kTile + warp * kRun, row0 = t.b * p.L + t0;
            const int n = static_cast<int>(min(max(p.L - t0, 0ll), static_cast<long long>(kRun)));
            T* to = mine + stage * 2 * kElems;
            copy_rows<T, kAny, kRun>(to, p.x + row0 * p.xs + t.c0, p.xs, n, t.c0, p.dim, lane);
            copy_rows<T, kAny, kRun>(to + kElems, p.dt + row0 * p.dts + t.c0, p.dts, n, t.c0, p.dim, lane);
        },
        [&](const Slot& t, int nth) {
            const T* sx = mine + (nth & 1) * 2 * kElems;
            if (static_cast<long long>(t.step + 1) * kTile <= p.L)
                return forward_tile<T, kAny, kSeq, true>(p, ex, t, sx, sx + kElems, nth);
            else
                return forward_tile<T, kAny, kSeq, false>(p, ex, t, sx, sx + kElems, nth);
        });
}

template <typename T, bool kAny, bool kSeq, bool kWhole>
__device__ __forceinline__ bool backward_tile(const ScanParams<T>& p, Exchange<T>& ex, const Slot& t, const T* sx,
                                              const T* sd, const T* sg, int nth) {
    using L = Pair;
    constexpr int kRun = kRunBwd;
    const int turn = nth & 1;
    const Place w = place_in<T, kAny>(p, t);
    const int tile = p.tiles - 1 - w.step;  // the scan over g runs back in time
    const long long t0 = static_cast<long long>(tile) * kState<T> + w.warp * kRun;
    const long long row0 = w.b * p.L + t0;
    const int n = kWhole ? kRun : static_cast<int>(min(max(p.L - t0, 0ll), static_cast<long long>(kRun)));
    const L A = t.A[w.lane];
    const Rows<T, kAny> x(sx, p.x + row0 * p.xs + t.c0, p.xs, w.lane), dt(sd, p.dt + row0 * p.dts + t.c0, p.dts, w.lane),
        dy(sg, p.dy + row0 * p.dys + t.c0, p.dys, w.lane);
    L a[kRun], delta[kRun], slope[kRun];
    {
        const L bias = t.bias[w.lane];
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            a[r] = L::splat(1.f), delta[r] = slope[r] = L::splat(0.f);
            if (kWhole || r < n) {
                L u;
                const L v = elem::add(dt(r), bias);
                delta[r] = elem::softplus<2>(v, &u);
                slope[r] = elem::softplus_slope<2>(v, u);
                a[r] = elem::exp_near<2>(elem::mul(A, delta[r]));
            }
        }
    }
    const uint32_t cut = begins_in<kRun, kSeq>(t, w.warp);
    auto begins = [&](int r) { return (cut >> r & 1u) != 0u; };  // a sequence, with token r of the run
    // the run's two maps: the state's (P, f) forward in time, g's (P, q) backward
    with<kSeq>(cut != 0u, [&](auto some) {
        L f = L::splat(0.f), P = L::splat(1.f), q = L::splat(0.f);
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            if (kWhole || r < n) {
                const L in = elem::mul(delta[r], x(r));
                f = some.value && begins(r) ? in : elem::fma(a[r], f, in);
                P = elem::mul(P, a[r]);
            }
        }
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r)
            if (kWhole || r < n) q = some.value && begins(r) ? L::splat(0.f) : elem::mul(a[r], elem::add(q, dy(r)));
        ex.run[turn][w.warp][w.lane] = {P, q};
        ex.f[turn][w.warp][w.lane] = f;
    });
    if (!wait_enter(p, ex, nth)) return false;
    const Map(*run)[32] = ex.run[turn];
    // h entering the run, then h before each of its tokens (zero before a sequence's first)
    const int last = kSeq ? last_before(t.cut_runs, w.warp) : -1;
    L h = last >= 0 ? ex.f[turn][last][w.lane] : t.state[w.lane];
    for (int k = last + 1; k < w.warp; ++k) h = elem::fma(run[k][w.lane].P, h, ex.f[turn][k][w.lane]);
    L before[kRun];
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
        if (kSeq && begins(r)) h = L::splat(0.f);
        before[r] = h;
        if (kWhole || r < n) h = elem::fma(a[r], h, elem::mul(delta[r], x(r)));
    }
    // what enters the run from the tokens after it
    const int next = kSeq ? first_after(t.cut_runs, w.warp) : -1;
    L k = next >= 0 ? run[next][w.lane].q : ex.enter[turn][w.lane];
    for (int o = (next >= 0 ? next : kWarps<T>) - 1; o > w.warp; --o) k = apply(run[o][w.lane], k);
    const L D = t.D[w.lane];
    L sA = L::splat(0.f), sb = sA, sD = sA;
    with<kSeq>(cut != 0u, p.D != nullptr, [&](auto some, auto skip) {
        T *px = p.y + (row0 + kRun - 1) * p.dxs + w.c, *pd = p.ddt + (row0 + kRun - 1) * p.ddts + w.c;
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r, px -= p.dxs, pd -= p.ddts) {
            if (!kWhole && r >= n) continue;
            const L dyv = dy(r), xv = x(r);
            const L g = elem::add(dyv, k);
            k = some.value && begins(r) ? L::splat(0.f) : elem::mul(a[r], g);
            const L gh = elem::mul(k, before[r]);  // dL / d(delta A)
            const L dd = elem::mul(elem::fma(A, gh, elem::mul(g, xv)), slope[r]);
            if (w.live) {
                store_out<T, kAny>(px, skip.value ? elem::fma(g, delta[r], elem::mul(D, dyv)) : elem::mul(g, delta[r]), w.both);
                store_out<T, kAny>(pd, dd, w.both);
            }
            sA = elem::fma(gh, delta[r], sA);
            sb = elem::add(sb, dd);
            sD = elem::fma(dyv, xv, sD);
        }
    });
    if (p.fin && w.live && tile == 0 && w.warp == 0) store_pair<kAny>(p.fin + w.own, k, w.both);
    ex.sums[turn][0][w.warp][w.lane] = sA;
    ex.sums[turn][1][w.warp][w.lane] = sb;
    ex.sums[turn][2][w.warp][w.lane] = sD;
    return true;
}

template <typename T, bool kAny, bool kSeq>
__global__ void __launch_bounds__(kThreads<T>, kCtasPerSm<T>) gated_scan_bwd(const ScanParams<T> p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kRun = kRunBwd, kElems = kState<T> * kPitch<T, kAny>;
    Exchange<T>& ex = *reinterpret_cast<Exchange<T>*>(smem + 2 * stage_bytes<T, kAny>(kRun, 3));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k) {
            ptx::mbar_init(&ex.runs_ready[k], kWarps<T>);
            ptx::mbar_init(&ex.enter_ready[k], 1);
        }
        ptx::fence_mbar_init();
    }
    if (warp == kWarps<T>) {
        guide<T, kAny, false, kSeq>(p, ex);
        return;
    }
    T* mine = reinterpret_cast<T*>(smem) + warp * kRun * kPitch<T, kAny>;
    walk_tiles<T, false>(
        ex,
        [&](const Slot& t, int stage) {
            const long long t0 = static_cast<long long>(p.tiles - 1 - t.step) * kState<T> + warp * kRun, row0 = t.b * p.L + t0;
            const int n = static_cast<int>(min(max(p.L - t0, 0ll), static_cast<long long>(kRun)));
            T* to = mine + stage * 3 * kElems;
            copy_rows<T, kAny, kRun>(to, p.x + row0 * p.xs + t.c0, p.xs, n, t.c0, p.dim, lane);
            copy_rows<T, kAny, kRun>(to + kElems, p.dt + row0 * p.dts + t.c0, p.dts, n, t.c0, p.dim, lane);
            copy_rows<T, kAny, kRun>(to + 2 * kElems, p.dy + row0 * p.dys + t.c0, p.dys, n, t.c0, p.dim, lane);
        },
        [&](const Slot& t, int nth) {
            const T* sx = mine + (nth & 1) * 3 * kElems;
            if (static_cast<long long>(p.tiles - t.step) * kState<T> <= p.L)
                return backward_tile<T, kAny, kSeq, true>(p, ex, t, sx, sx + kElems, sx + 2 * kElems, nth);
            else
                return backward_tile<T, kAny, kSeq, false>(p, ex, t, sx, sx + kElems, sx + 2 * kElems, nth);
        });
}

// dA, d dt_bias, dD: the tiles' rows added up, rows r, r + 16, ... by one thread
// and the 16 partial sums in a fixed order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows)
    gated_scan_sums(const float* __restrict__ sums, long long rows, long long dim, float* dA, float* dbias, float* dD) {
    __shared__ float part[kSumRows][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long col = static_cast<long long>(blockIdx.x) * 32 + tx, cols = 3 * dim;
    float s = 0.f;
    if (col < cols) {
#pragma unroll 4
        for (long long r = ty; r < rows; r += kSumRows) s += sums[r * cols + col];
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && col < cols) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) s += part[k][tx];
        const long long which = col / dim, cc = col - which * dim;
        float* out = which == 0 ? dA : which == 1 ? dbias : dD;
        if (out) out[cc] = s;
    }
}

// One decode token: V channels of one sequence per thread, the state in place.
template <typename T, int V>
__global__ void __launch_bounds__(128)
    gated_scan_step(const T* __restrict__ x, const T* __restrict__ dt, long long xs, long long dts,
                    const float* __restrict__ bias, const float* __restrict__ A, const float* __restrict__ D,
                    float* __restrict__ state, T* __restrict__ y, long long dim) {
    const long long c = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) * V;
    if (c >= dim) return;
    const long long b = blockIdx.y;
    using L = Vals<V>;
    Pack<T, V> xv, dv;
    xv.load(x + b * xs + c);
    dv.load(dt + b * dts + c);
    L u;
    const L delta = elem::softplus<V>(elem::add(elem::unpack<T, V>(dv), L::load(bias + c)), &u);
    const L a = decay<T, V>(decay_A<T, V>(L::load(A + c)), delta);
    const L h = elem::fma(a, L::load(state + b * dim + c), elem::mul(delta, elem::unpack<T, V>(xv)));
    h.store(state + b * dim + c);
    elem::store_vals<T, V>(y + b * dim + c, D ? elem::fma(L::load(D + c), elem::unpack<T, V>(xv), h) : h);
}

// ---------------------------------------------------------------- host side
template <typename T>
long long tiles_of(long long L, bool backward) {
    const long long tile = backward ? kState<T> : kRunFwd<T> * kWarps<T>;
    return (L + tile - 1) / tile;
}

// Workspace of one call: exchange area (only with more than one tile), then the
// backward's sums.
struct ScanLayout {
    long long tiles;
    size_t unset = 0;  // bytes to set to kUnset before the launch: ticket, abort word, carries, maps
    size_t carry = 0, maps = 0, sums, total;
};
long long pitch_of(const ssd_scan_dims& d) { return d.dim + (d.dim & 1); }
ScanLayout scan_layout(const ssd_scan_dims& d, ssd_dtype io, bool backward) {
    ScanLayout l;
    l.tiles = io == SSD_BF16 ? tiles_of<__nv_bfloat16>(d.seqlen, backward) : tiles_of<float>(d.seqlen, backward);
    const size_t tiles = l.tiles, groups = (tiles + kGroup - 1) / kGroup, cells = d.batch * pitch_of(d);
    size_t at = 0;
    if (tiles > 1) {
        l.carry = 256;
        l.maps = align_up(l.carry + 4 * groups * cells, kWorkspaceAlign);
        l.unset = l.maps + 8 * tiles * cells;
        at = align_up(l.unset, kWorkspaceAlign);
    }
    l.sums = at;
    if (backward) at = align_up(at + 12 * tiles * d.batch * d.dim, kWorkspaceAlign);
    l.total = at;
    return l;
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

ssd_status check_scan(const ssd_scan_dims* d, ssd_dtype io) {
    if (!d || (io != SSD_F32 && io != SSD_BF16)) return SSD_ERR_INVALID_ARG;
    if (d->batch < 1 || d->seqlen < 1 || d->dim < 1) return SSD_ERR_INVALID_ARG;
    // 32-bit tile and ticket counts, and products that stay far inside 64 bits
    if (d->batch >= (1ll << 24) || d->dim >= (1ll << 24) || d->seqlen >= (1ll << 40)) return SSD_ERR_UNSUPPORTED;
    const long long chains = d->batch * ((d->dim + 31) / 32);
    if (chains >= (1ll << 30) || tiles_of<float>(d->seqlen, true) >= (1ll << 30) / chains) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

template <typename T, bool kAny, bool kSeq>
ssd_status launch_scan(ScanParams<T>& p, const ssd_scan_dims& d, bool backward, const ScanLayout& l, void* ws,
                       float* dA, float* dbias, float* dD, cudaStream_t stream) {
    p.L = d.seqlen;
    p.dim = d.dim;
    p.pitch = pitch_of(d);
    p.batch = static_cast<int>(d.batch);
    p.tiles = static_cast<int>(l.tiles);
    p.tiles_c = static_cast<int>((d.dim + 63) / 64);
    p.chains = p.batch * p.tiles_c;
    char* base = static_cast<char*>(ws);
    p.ticket = reinterpret_cast<uint32_t*>(base);
    p.carry = reinterpret_cast<uint32_t*>(base + l.carry);
    p.maps = reinterpret_cast<uint32_t*>(base + l.maps);
    p.sums = reinterpret_cast<float*>(base + l.sums);
    const ssd_status st = call_context(&p.status, &p.wait_ns);
    if (st != SSD_OK) return st;
    if (l.unset && cudaMemsetAsync(ws, 0xFF, l.unset, stream) != cudaSuccess) return SSD_ERR_CUDA;
    const int run = backward ? kRunBwd : kRunFwd<T>;
    using Ex = Exchange<T>;
    const int smem = 2 * stage_bytes<T, kAny>(run, backward ? 3 : 2) +
                     static_cast<int>(backward ? sizeof(Ex) : offsetof(Ex, f));
    auto* kernel = backward ? gated_scan_bwd<T, kAny, kSeq> : gated_scan_fwd<T, kAny, kSeq>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return SSD_ERR_CUDA;
    // one tile per CTA where a sequence is one tile (nothing to take in order); else persistent CTAs
    const long long units = static_cast<long long>(p.chains) * p.tiles;
    const unsigned grid = static_cast<unsigned>(p.tiles == 1 ? units : std::min<long long>(units, kCtasPerSm<T> * device_sms()));
    kernel<<<grid, kThreads<T>, smem, stream>>>(p);
    note_launches(1);
    if (backward) {
        gated_scan_sums<<<static_cast<unsigned>((3 * d.dim + 31) / 32), 32 * kSumRows, 0, stream>>>(
            p.sums, d.batch * static_cast<long long>(p.tiles), d.dim, dA, dbias, dD);
        note_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Whether every row of every io tensor starts on 16 bytes, and whether sequences are packed.
template <typename T>
ssd_status dispatch_scan(ScanParams<T>& p, const ssd_scan_dims& d, bool backward, void* ws, size_t ws_bytes, float* dA,
                         float* dbias, float* dD, cudaStream_t stream) {
    const ScanLayout l = scan_layout(d, sizeof(T) == 2 ? SSD_BF16 : SSD_F32, backward);
    if (ws_bytes < l.total || (l.total > 0 && (!ws || !aligned_to(ws, kWorkspaceAlign)))) return SSD_ERR_WORKSPACE;
    auto whole = [](long long n) { return n % kVec<T> == 0; };
    bool wide = whole(d.dim) && whole(p.xs) && whole(p.dts);
    for (const void* q : {static_cast<const void*>(p.x), static_cast<const void*>(p.dt),
                          static_cast<const void*>(p.dy), static_cast<const void*>(p.y),
                          static_cast<const void*>(p.ddt)})
        wide = wide && aligned_to(q, 16);
    if (backward) wide = wide && whole(p.dys) && whole(p.dxs) && whole(p.ddts);
    auto* launch = p.seq ? (wide ? launch_scan<T, false, true> : launch_scan<T, true, true>)
                         : (wide ? launch_scan<T, false, false> : launch_scan<T, true, false>);
    return launch(p, d, backward, l, ws, dA, dbias, dD, stream);
}

bool scan_aligned(ssd_dtype io, std::initializer_list<const void*> io_ptrs, std::initializer_list<const void*> f32_ptrs) {
    for (const void* q : io_ptrs)
        if (!aligned_to(q, io == SSD_BF16 ? 2 : 4)) return false;
    for (const void* q : f32_ptrs)
        if (!aligned_to(q, 4)) return false;
    return true;
}

}  // namespace
}  // namespace ssd

extern "C" {

int64_t ssd_gated_scan_chunks(ssd_dtype io_dtype, int64_t seqlen) {
    using namespace ssd;
    if (seqlen < 1) return 0;
    return io_dtype == SSD_BF16 ? tiles_of<__nv_bfloat16>(seqlen, true) : tiles_of<float>(seqlen, true);
}

size_t ssd_gated_scan_workspace_bytes(const ssd_scan_dims* dims, ssd_dtype io_dtype, int backward) {
    using namespace ssd;
    if (check_scan(dims, io_dtype) != SSD_OK) return 0;
    return scan_layout(*dims, io_dtype, backward != 0).total;
}

ssd_status ssd_gated_scan(const ssd_scan_dims* dims, ssd_dtype io_dtype, const void* x, int64_t x_row_stride,
                          const void* dt, int64_t dt_row_stride, const float* dt_bias, const float* A, const float* D,
                          const float* init_state, const int32_t* seq_idx, void* y, float* final_state,
                          float* chunk_states, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssd;
    const ssd_status st = check_scan(dims, io_dtype);
    if (st != SSD_OK) return st;
    if (!x || !dt || !dt_bias || !A || !y) return SSD_ERR_INVALID_ARG;
    if (x_row_stride < dims->dim || dt_row_stride < dims->dim) return SSD_ERR_INVALID_ARG;
    if (!scan_aligned(io_dtype, {x, dt, y}, {dt_bias, A, D, init_state, seq_idx, final_state, chunk_states}))
        return SSD_ERR_UNSUPPORTED;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        ScanParams<T> p{};
        p.x = static_cast<const T*>(x), p.dt = static_cast<const T*>(dt), p.y = static_cast<T*>(y);
        p.xs = x_row_stride, p.dts = dt_row_stride;
        p.bias = dt_bias, p.A = A, p.D = D, p.init = init_state, p.seq = seq_idx;
        p.fin = final_state, p.states = chunk_states;
        return dispatch_scan<T>(p, *dims, false, workspace, workspace_bytes, nullptr, nullptr, nullptr,
                                static_cast<cudaStream_t>(stream));
    };
    return io_dtype == SSD_BF16 ? go(__nv_bfloat16()) : go(float());
}

ssd_status ssd_gated_scan_bwd(const ssd_scan_dims* dims, ssd_dtype io_dtype, const void* dy, int64_t dy_row_stride,
                              const void* x, int64_t x_row_stride, const void* dt, int64_t dt_row_stride,
                              const float* dt_bias, const float* A, const float* D, const int32_t* seq_idx,
                              const float* chunk_states, const float* dfinal_state, void* dx, int64_t dx_row_stride,
                              void* ddt, int64_t ddt_row_stride, float* ddt_bias, float* dA, float* dD,
                              float* dinit_state, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssd;
    const ssd_status st = check_scan(dims, io_dtype);
    if (st != SSD_OK) return st;
    if (!dy || !x || !dt || !dt_bias || !A || !chunk_states || !dx || !ddt || !ddt_bias || !dA)
        return SSD_ERR_INVALID_ARG;
    for (int64_t s : {dy_row_stride, x_row_stride, dt_row_stride, dx_row_stride, ddt_row_stride})
        if (s < dims->dim) return SSD_ERR_INVALID_ARG;
    if (!scan_aligned(io_dtype, {dy, x, dt, dx, ddt},
                      {dt_bias, A, D, seq_idx, chunk_states, dfinal_state, ddt_bias, dA, dD, dinit_state}))
        return SSD_ERR_UNSUPPORTED;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        ScanParams<T> p{};
        p.x = static_cast<const T*>(x), p.dt = static_cast<const T*>(dt), p.dy = static_cast<const T*>(dy);
        p.y = static_cast<T*>(dx), p.ddt = static_cast<T*>(ddt);
        p.xs = x_row_stride, p.dts = dt_row_stride, p.dys = dy_row_stride;
        p.dxs = dx_row_stride, p.ddts = ddt_row_stride;
        p.bias = dt_bias, p.A = A, p.D = D, p.init = dfinal_state, p.seq = seq_idx;
        p.fin = dinit_state, p.states = const_cast<float*>(chunk_states);
        return dispatch_scan<T>(p, *dims, true, workspace, workspace_bytes, dA, ddt_bias, dD,
                                static_cast<cudaStream_t>(stream));
    };
    return io_dtype == SSD_BF16 ? go(__nv_bfloat16()) : go(float());
}

ssd_status ssd_gated_scan_step(const ssd_scan_dims* dims, ssd_dtype io_dtype, const void* x, int64_t x_row_stride,
                               const void* dt, int64_t dt_row_stride, const float* dt_bias, const float* A,
                               const float* D, float* state, void* y, void* stream) {
    using namespace ssd;
    const ssd_status st = check_scan(dims, io_dtype);
    if (st != SSD_OK) return st;
    if (dims->seqlen != 1 || !x || !dt || !dt_bias || !A || !state || !y) return SSD_ERR_INVALID_ARG;
    if (x_row_stride < dims->dim || dt_row_stride < dims->dim) return SSD_ERR_INVALID_ARG;
    if (dims->batch >= 65536) return SSD_ERR_UNSUPPORTED;
    if (!scan_aligned(io_dtype, {x, dt, y}, {dt_bias, A, D, state})) return SSD_ERR_UNSUPPORTED;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        const bool two = dims->dim % 2 == 0 && x_row_stride % 2 == 0 && dt_row_stride % 2 == 0 &&
                         aligned_to(x, 2 * sizeof(T)) && aligned_to(dt, 2 * sizeof(T)) && aligned_to(y, 2 * sizeof(T));
        const int V = two ? 2 : 1;
        const dim3 grid(static_cast<unsigned>((dims->dim + 128 * V - 1) / (128 * V)),
                        static_cast<unsigned>(dims->batch));
        auto* kernel = two ? gated_scan_step<T, 2> : gated_scan_step<T, 1>;
        kernel<<<grid, 128, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const T*>(x), static_cast<const T*>(dt), x_row_stride, dt_row_stride, dt_bias, A, D, state,
            static_cast<T*>(y), dims->dim);
        note_launches(1);
        return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    };
    return io_dtype == SSD_BF16 ? go(__nv_bfloat16()) : go(float());
}

}  // extern "C"
