// Softmax cross entropy of a vocabulary projection and its gradient
// (include/ssd.h, ssd_linear_cross_entropy), without keeping the logits:
//
//   logits = hidden weight^T      lse_n = log sum_v e^{logits_nv}
//   loss_n = lse_n - logits_{n, target_n}
//   dl_nv = dloss_n (e^{logits_nv - lse_n} - [v = target_n])
//   dhidden = dl weight           dweight = dl^T hidden
//
// Four matrix products, all on the fifth-generation tensor cores. The forward
// reduces each tile of logits to a (maximum, sum) pair per row while it is still
// in tensor memory; a second kernel joins the pairs in a fixed order. The
// backward goes over the vocabulary in pieces: it rebuilds a piece's logits, turns
// them into dl in the product's epilogue (bf16, the operand type of the next two
// products), and one launch then takes both gradients of the piece. dweight's
// rows are final; dhidden is accumulated in fp32 over the pieces (each tile of it
// owned by one CTA pair, so the order is fixed) and rounded once at the end. dl is held
// relative to the first row's dloss, which multiplies both gradients in fp32: where all rows weigh
// the same (a mean), what is rounded is p - [target], near -1 for most rows' targets,
// while dloss's own rounding would be one common error of all of them. Where
// dhidden has fewer tiles than there are CTA pairs its sum over the vocabulary is
// split, each part with an accumulator of its own.
//
// One persistent kernel, a CTA pair (two SMs) per 256 x 256 output tile: each CTA
// holds 128 rows of A and 128 of B's 256, so every operand byte in shared memory
// serves both. Roles per CTA: warp 0 issues the TMA loads, warp 1 of the pair's
// first CTA the MMAs, warps 4 to 11 run the epilogue from one of two accumulators
// (256 columns of tensor memory each) while the MMAs fill the other.
//
// The epilogues' outputs go through shared memory and leave as TMA stores (dl,
// dweight) or TMA additions (dhidden's accumulators, later parts of a tile), so a warp does not wait
// for global memory.
//
// fp32 operands are written as sums of three bf16 terms (24 bits): a = a0 + a1 + a2.
// Six of the nine products are kept (a0 b0, a0 b1, a1 b0, a1 b1, a0 b2, a2 b0; the
// others are below 2^-24 of a0 b0) and run through the same kernel as one
// product of six times the depth, the largest term last; the gradients' sums leave the
// accumulators every 512 of depth and add up in fp32. The forward of few fp32 rows
// reads the weight as it is (ce_few_stats).
#include <algorithm>
#include <initializer_list>

#include "elem.cuh"
#include "ptx.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kTileM = 256, kTileN = 256;  // per CTA pair
constexpr int kHalf = 128;                 // rows of A, and of B, per CTA
constexpr int kBK = 64;                    // depth of a stage: one 128-byte swizzle row
constexpr int kStages = 5;                 // (4 to 6 measured alike)
constexpr uint32_t kOperand = kHalf * kBK * 2;  // bytes of one CTA's part of an operand's stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kEpiWarps = 8;               // two per quarter of the rows, 128 columns each
constexpr int kEpiCols = kTileN / 2;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kOutTile = 32 * 128;    // an epilogue warp's output tile: 32 rows of 128 bytes; two per warp
constexpr uint32_t kSmem = kStages * kStage + kEpiWarps * 2 * kOutTile + 1024;
constexpr int kMaxSegs = 6;

enum Mode { kStats = 0, kDlogits = 1, kGrads = 2 };

// One product A B^T over depth blocks of kBK; an operand is stored with the depth
// contiguous (K-major) or with its rows contiguous (MN-major).
struct Product {
    int a_mn, b_mn;    // 1: MN-major
    int a_row, b_row;  // first row of the operand that tile row / column 0 maps to
    int a_dep, b_dep;  // the operands' depth coordinates of depth 0
    int tiles_m, tiles_n, splits;
    int blocks;        // depth blocks
    int m_fast;        // 1: consecutive tiles go along m
};

struct CeParams {
    Product prod[2];
    int jobs[2];  // tiles of each product; prod[1] only in kGrads
    int lead;     // see nth_tile
    int late;     // its operands are not written by the kernels before it: only the epilogue waits for them
    int segs;     // 1 (bf16), or the six products of three-term operands
    int seg_a[kMaxSegs], seg_b[kMaxSegs];
    long long rows, vocab, dim;
    int v0, v1;  // the piece's vocabulary range (v0: a whole number of tiles)
    const long long* target;
    long long ignore;
    // kStats
    float2* stats;  // [2 tiles_n, rows]: per half tile
    float* picked;  // [rows]: the targets' logits (kDlogits: summed in fp32)
    // kDlogits
    const float* lse;
    const float* dloss;  // (and kGrads)
    int planes;
    // kGrads: prod[0] is dhidden, prod[1] dweight
    int flush;  // depth blocks after which an accumulator is added to the output and starts again (kNoFlush: at the end)
    long long acc_ld;
    int first;  // the first piece stores, later ones add
    void* dweight;
    int dw_f32, dw_vec;  // dw_vec: rows start on 16 bytes (else stored element by element)
    unsigned* status;
};

constexpr int kSegBlocks = 4;  // see the loads
constexpr int kNoFlush = 1 << 30;
// Limit on a wait for this pair's own copies, products and epilogues.
constexpr unsigned long long kWaitNs = 2000000000ull;

// Operands of the two products; outputs: dl [planes, rows, piece] (kDlogits) or the
// accumulators [splits, rows, acc_ld] (kGrads), and dweight.
struct Maps {
    CUtensorMap a0, b0, a1, b1, out, dw;
};

// ---------------------------------------------------------------- CTA pair primitives
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// a box into this CTA's shared memory; the bytes count on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int c0, int c2,
                                              int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(0), "r"(c2), "r"(c3), "r"(bar_cluster)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(dst)), "r"(cols)
                 : "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}

struct Control {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    volatile uint32_t abort;
};

// Waits for a phase; false (for good) once any wait of this CTA has run out of time.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Control* c, const CeParams& p) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (c->abort) return false;
        if (ptx::globaltimer_ns() - t0 > kWaitNs) {
            c->abort = 1u;
            atomicOr(p.status, 1u);
            return false;
        }
    }
    return true;
}

// The i-th tile of a pair, or a number past the last. The first product's tiles go round the
// pairs. Where they end inside a round, the pairs without one in it take `lead` of the
// second product's tiles first (about what that tile costs), then those go round too.
__device__ __forceinline__ int nth_tile(const CeParams& p, int pair, int pairs, int i) {
    const int mine = (p.jobs[0] - pair + pairs - 1) / pairs;
    if (i < mine) return pair + i * pairs;
    i -= mine;
    const int extra = p.jobs[0] % pairs, others = pairs - extra;
    int j = p.lead * others + pair;
    if (pair < extra)
        j += i * pairs;
    else if (i < p.lead)
        j = i * others + pair - extra;
    else
        j += (i - p.lead) * pairs;
    return j < p.jobs[1] ? p.jobs[0] + j : p.jobs[0] + p.jobs[1];
}

struct Tile {
    int which, m, n, split, b0, b1;  // product, tile coordinates, depth blocks [b0, b1)
};
__device__ __forceinline__ Tile tile_at(const CeParams& p, int t) {
    Tile r;
    r.which = t >= p.jobs[0];
    if (r.which) t -= p.jobs[0];
    const Product& q = p.prod[r.which];
    const int per = q.tiles_m * q.tiles_n;
    r.split = t / per;
    t -= r.split * per;
    if (q.m_fast)
        r.n = t / q.tiles_m, r.m = t - r.n * q.tiles_m;
    else
        r.m = t / q.tiles_n, r.n = t - r.m * q.tiles_n;
    r.b0 = static_cast<int>(static_cast<long long>(q.blocks) * r.split / q.splits);
    r.b1 = static_cast<int>(static_cast<long long>(q.blocks) * (r.split + 1) / q.splits);
    return r;
}

// One operand's part of a stage, 128 rows by kBK of depth, as two boxes of 64 rows at
// (x, y) and (x + dx, y + dy); the next depth block lies (sx, sy) further. The
// issuing loop keeps no more than this: one lane's address arithmetic per box was
// what bounded the products (1.38 ms for the logits of 8192 x 2560 x 50280).
struct Boxes {
    const CUtensorMap* map;
    int x, y, dx, dy, sx, sy;
    __device__ __forceinline__ Boxes(const CUtensorMap* m, int mn, int row, int depth)
        : map(m), x(mn ? row : depth), y(mn ? depth : row), dx(mn ? 64 : 0), dy(mn ? 0 : 64), sx(mn ? 0 : kBK),
          sy(mn ? kBK : 0) {}
    __device__ __forceinline__ void load(uint32_t dst, uint32_t bar, int plane) const {
        tma_load_pair(dst, map, bar, x, y, plane);
        tma_load_pair(dst + kOperand / 2, map, bar, x + dx, y + dy, plane);
    }
    __device__ __forceinline__ void next() { x += sx, y += sy; }
};

// ---------------------------------------------------------------- epilogues (one thread: one row, 128 columns)
// An epilogue warp's tile of the accumulator: 32 rows, one per lane, from row0 (of the
// output) on, columns [col0, col0 + 128) of the tile's 256.
struct EpiTile {
    const CeParams& p;
    const Tile& t;
    uint32_t taddr;  // tensor memory, at its rows and columns
    long long row0, row;
    int half, lane;
    uint32_t out;    // this warp's output tiles in shared memory
    uint32_t* turn;  // which of the two is next

    // 32 columns of this thread's row, by the whole warp
    __device__ __forceinline__ void load(int c, uint32_t (&r)[32]) const {
        __syncwarp();
        ptx::tmem_ld32(taddr + c, r);
        ptx::tmem_wait_ld(r);
    }
    // An output tile that no earlier store still reads.
    __device__ __forceinline__ uint32_t begin_out() const {
        if (lane == 0) ptx::bulk_wait_group_read<1>();
        __syncwarp();
        const uint32_t at = out + (*turn & 1u) * kOutTile;
        ++*turn;
        return at;
    }
    // 16 bytes of this lane's row
    __device__ __forceinline__ void put(uint32_t at, int chunk, uint4 v) const {
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + ptx::swz128(lane, chunk)), "r"(v.x), "r"(v.y),
                     "r"(v.z), "r"(v.w)
                     : "memory");
    }
    // The tile to the output at column c0; rows and columns outside the tensor are dropped.
    __device__ __forceinline__ void end_out(uint32_t at, const CUtensorMap* map, int c0, long long outer, bool add) const {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (add)
                tma_add(map, at, c0, static_cast<int>(row0), static_cast<int>(outer));
            else
                tma_store(map, at, c0, static_cast<int>(row0), static_cast<int>(outer));
            ptx::bulk_commit_group();
        }
    }
    __device__ static __forceinline__ void tma_store(const CUtensorMap* map, uint32_t at, int c0, int c2, int c3) {
        asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(at), "r"(c0), "r"(0), "r"(c2), "r"(c3)
                     : "memory");
    }
    __device__ static __forceinline__ void tma_add(const CUtensorMap* map, uint32_t at, int c0, int c2, int c3) {
        asm volatile("cp.reduce.async.bulk.tensor.4d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::
                         "l"(reinterpret_cast<uint64_t>(map)),
                     "r"(at), "r"(c0), "r"(0), "r"(c2), "r"(c3)
                     : "memory");
    }
};
// n clamped to [-1, 64]: an index or a count within 64 columns
__device__ __forceinline__ int within64(long long n) { return n < 0 ? -1 : n > 64 ? 64 : static_cast<int>(n); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What exponents are taken relative to: the maximum, or nothing while there is none (no class so far, or
// only logits of minus infinity: they count zero; of NaN: the sum is NaN).
__device__ __forceinline__ float relative_to(float m) { return m == -__builtin_inff() ? 0.f : m; }

__device__ __forceinline__ void epilogue_stats(const EpiTile& e) {
    const CeParams& p = e.p;
    const long long col0 = p.v0 + static_cast<long long>(e.t.n) * kTileN + e.half * kEpiCols;
    const long long target = e.row < p.rows ? p.target[e.row] : -1;
    float m = -__builtin_inff(), s = 0.f;
#pragma unroll 1
    for (int c = 0; c < kEpiCols; c += 32) {
        uint32_t r[32];
        e.load(c, r);
        const int left = within64(p.v1 - (col0 + c));
        if (left <= 0) continue;
        if (left < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i >= left) r[i] = 0xFF800000u;  // -inf: not a column
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = __uint_as_float(r[i]);
#pragma unroll
        for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(r[i]));
        const float m2 = fmaxf(fmaxf(m, fmaxf(top[0], top[1])), fmaxf(top[2], top[3]));
        const float base = relative_to(m2);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) part[i & 3] += elem::exp2_fast((__uint_as_float(r[i]) - base) * elem::kLog2e);
        s = fmaf(s, elem::exp2_fast((m - base) * elem::kLog2e), (part[0] + part[1]) + (part[2] + part[3]));
        m = m2;
        const int at = within64(target - (col0 + c));
        if (at >= 0 && at < 32) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i == at) v = __uint_as_float(r[i]);
            p.picked[e.row] = v;
        }
    }
    if (e.row < p.rows) p.stats[(2ll * (p.v0 / kTileN + e.t.n) + e.half) * p.rows + e.row] = make_float2(m, s);
}

// What dl is held relative to: the first row's dloss, where it is of a magnitude that
// quotients by it stay finite.
__device__ __forceinline__ float reference_dloss(const float* dloss) {
    const float g = dloss[0], a = fabsf(g);
    return a >= 0x1p-40f && a <= 0x1p40f ? g : 1.f;
}

__device__ __forceinline__ void epilogue_dlogits(const EpiTile& e, const CUtensorMap* map) {
    const CeParams& p = e.p;
    const bool in = e.row < p.rows;
    const long long target = in ? p.target[e.row] : p.ignore;
    const bool kept = target != p.ignore;
    const float lse = in ? p.lse[e.row] : 0.f;
    float g = kept ? p.dloss[e.row] / reference_dloss(p.dloss) : 0.f;
    if (kept && (target < 0 || target >= p.vocab)) g = __uint_as_float(0x7FC00000u);  // not a class: NaN
    const int col0 = e.t.n * kTileN + e.half * kEpiCols;  // within the piece
#pragma unroll 1
    for (int c = 0; c < kEpiCols; c += 64) {
        const long long v = static_cast<long long>(p.v0) + col0 + c;
        const int left = within64(p.v1 - v), at = within64(target - v);
        float d[64];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            e.load(c + 32 * h, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) d[32 * h + i] = g * elem::exp2_fast((__uint_as_float(r[i]) - lse) * elem::kLog2e);
        }
        if (at >= 0 && at < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i == at) d[i] = g * expm1f(p.picked[e.row] - lse);
        }
        if (left < 64 || !kept) {  // entries past the vocabulary; rows without a loss, whatever their logits are
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= left || !kept) d[i] = 0.f;
        }
        for (int plane = 0; plane < p.planes && e.row0 < p.rows; ++plane) {
            const uint32_t o = e.begin_out();
#pragma unroll
            for (int i = 0; i < 64; i += 8)
                e.put(o, i / 8, make_uint4(pack2(d[i], d[i + 1]), pack2(d[i + 2], d[i + 3]), pack2(d[i + 4], d[i + 5]),
                                           pack2(d[i + 6], d[i + 7])));
            e.end_out(o, map, col0 + c, plane, false);
            if (plane + 1 < p.planes) {  // what this term leaves
#pragma unroll
                for (int i = 0; i < 64; ++i) d[i] -= __bfloat162float(__float2bfloat16_rn(d[i]));
            }
        }
    }
}

// 32 fp32 columns per output tile, times scale
__device__ __forceinline__ void epilogue_f32(const EpiTile& e, const CUtensorMap* map, long long rows, long long cols,
                                             long long outer, bool add, float scale) {
    const int col0 = e.t.n * kTileN + e.half * kEpiCols;
#pragma unroll 1
    for (int c = 0; c < kEpiCols; c += 32) {
        uint32_t r[32];
        e.load(c, r);
        if (e.row0 >= rows || col0 + c >= cols) continue;
        const uint32_t o = e.begin_out();
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * scale);
#pragma unroll
        for (int i = 0; i < 32; i += 4) e.put(o, i / 4, make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]));
        e.end_out(o, map, col0 + c, outer, add);
    }
}

// 64 bf16 columns per output tile, times scale
__device__ __forceinline__ void epilogue_bf16(const EpiTile& e, const CUtensorMap* map, long long rows, long long cols,
                                              float scale) {
    const int col0 = e.t.n * kTileN + e.half * kEpiCols;
#pragma unroll 1
    for (int c = 0; c < kEpiCols; c += 64) {
        uint32_t w[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            e.load(c + 32 * h, r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) w[16 * h + i / 2] = pack2(__uint_as_float(r[i]) * scale, __uint_as_float(r[i + 1]) * scale);
        }
        if (e.row0 >= rows || col0 + c >= cols) continue;
        const uint32_t o = e.begin_out();
#pragma unroll
        for (int i = 0; i < 8; ++i) e.put(o, i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
        e.end_out(o, map, col0 + c, 0, false);
    }
}

// Rows that start anywhere: 32 by 32 values through shared memory, stored a row at a time.
__device__ __forceinline__ void epilogue_elements(const EpiTile& e, bool add, float scale) {
    const CeParams& p = e.p;
    const long long col0 = static_cast<long long>(e.t.n) * kTileN + e.half * kEpiCols;
    if (e.lane == 0) ptx::bulk_wait_group_read0();  // no earlier store reads this warp's tiles
#pragma unroll 1
    for (int c = 0; c < kEpiCols; c += 32) {
        uint32_t r[32];
        e.load(c, r);
        const int left = within64(p.dim - (col0 + c));
        if (e.row0 >= p.v1 || left <= 0) continue;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) e.put(e.out, i / 4, make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]));
        __syncwarp();
        const long long off = e.row0 * p.dim + col0 + c + e.lane;
        const int rows = static_cast<int>(min(32ll, static_cast<long long>(p.v1) - e.row0));
        if (e.lane >= left) continue;
        auto value = [&](int k) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(v)
                         : "r"(e.out + ptx::swz128(k, e.lane >> 2) + (e.lane & 3) * 4)
                         : "memory");
            return v * scale;
        };
        if (!add) {
#pragma unroll 8
            for (int k = 0; k < rows; ++k) {
                if (p.dw_f32)
                    static_cast<float*>(p.dweight)[off + k * p.dim] = value(k);
                else
                    static_cast<__nv_bfloat16*>(p.dweight)[off + k * p.dim] = __float2bfloat16_rn(value(k));
            }
        } else {  // (fp32) sixteen rows' loads in flight
            float* to = static_cast<float*>(p.dweight) + off;
#pragma unroll 1
            for (int k0 = 0; k0 < rows; k0 += 16, to += 16 * p.dim) {
                float old[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) old[k] = k0 + k < rows ? to[k * p.dim] : 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (k0 + k < rows) to[k * p.dim] = old[k] + value(k0 + k);
            }
        }
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    ce_gemm(const __grid_constant__ Maps maps, const __grid_constant__ CeParams p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;  // the same offset in both CTAs
    __shared__ Control ctl;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform)
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int total = p.jobs[0] + p.jobs[1];
    const int flush = MODE == kGrads ? p.flush : kNoFlush;

    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&ctl.full[i], 1);
            ptx::mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ctl.acc_full[i], 1);
            ptx::mbar_init(&ctl.acc_empty[i], 2 * kEpiWarps);
        }
        ptx::mbar_init(&ctl.drain, 1);
        ctl.abort = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 2) tmem_alloc_pair(&ctl.tmem, 512);
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    if (!p.late) ptx::griddep_wait();

    if (warp == 0) {
        // ---- loads: this CTA's 128 rows of A and of B; the bytes of both CTAs count on the first one's
        // barrier. The warp walks the loop, one elected lane issues. Six products: the smaller five go
        // kSegBlocks of depth at a time, so that a plane that two of them read comes from L2 the second time
        // (51 x 2752 x 56015 forward 539 to 499 us). The largest comes last: the accumulator truncates by its size.
        const bool leader = elect_one();
        const uint32_t full0 = map_rank(ptx::smem_u32(&ctl.full[0]), 0);
        uint32_t st = 0, phase = 1;
        bool ok = true;
        for (int i = 0, t; ok && (t = nth_tile(p, pair, pairs, i)) < total; ++i) {
            const Tile w = tile_at(p, t);
            const Product& q = p.prod[w.which];
            const int half = static_cast<int>(rank) * kHalf;
            // depth [from, to) of the products [s0, s1)
            auto stretch = [&](int from, int to, int s0, int s1) {
                for (int s = s0; s < s1 && ok; ++s) {
                    const int pa = p.seg_a[s], pb = p.seg_b[s];
                    Boxes a(w.which ? &maps.a1 : &maps.a0, q.a_mn, q.a_row + w.m * kTileM + half, q.a_dep + from * kBK);
                    Boxes b(w.which ? &maps.b1 : &maps.b0, q.b_mn, q.b_row + w.n * kTileN + half, q.b_dep + from * kBK);
                    for (int k = from; k < to; ++k) {
                        if (!(ok = wait_bar(&ctl.empty[st], phase, &ctl, p))) break;
                        if (leader) {
                            const uint32_t dst = sbase + st * kStage, bar = full0 + st * 8;
                            if (rank == 0) ptx::mbar_arrive_expect_tx(&ctl.full[st], 2 * kStage);
                            a.load(dst, bar, pa);
                            b.load(dst + kOperand, bar, pb);
                        }
                        __syncwarp();
                        a.next(), b.next();
                        if (++st == kStages) st = 0, phase ^= 1;
                    }
                }
            };
            for (int b0 = w.b0; b0 < w.b1 && ok; b0 += flush) {
                const int b1 = min(w.b1 - b0, flush) + b0;
                for (int k = b0; p.segs > 1 && k < b1 && ok; k += kSegBlocks)
                    stretch(k, min(k + kSegBlocks, b1), 0, p.segs - 1);
                stretch(b0, b1, p.segs - 1, p.segs);
            }
        }
        if (!ok) {  // the copies in flight land before the shared memory is given up
            const uint64_t t0 = ptx::globaltimer_ns();
            while (ptx::globaltimer_ns() - t0 < 1000000ull) {
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- MMAs of the pair. The whole warp walks the loop and one elected lane issues: the
        // descriptors then stay in uniform registers (a loop inside one lane's branch moves them
        // there for every MMA, which made the issue and not the tensor pipe the limit).
        const bool leader = elect_one();
        uint32_t st = 0, phase = 0;
        int n_tile = 0;
        bool ok = true;
        for (int i = 0, t; ok && (t = nth_tile(p, pair, pairs, i)) < total; ++i) {
            const Tile w = tile_at(p, t);
            const Product& q = p.prod[w.which];
            const uint32_t idesc = ptx::idesc_bf16_f32(kTileM, kTileN, q.a_mn, q.b_mn);
            // 16 of depth: 32 bytes along a K-major row, two 8-row groups of an MN-major tile
            const uint32_t step_a = q.a_mn ? 2048u >> 4 : 32u >> 4, step_b = q.b_mn ? 2048u >> 4 : 32u >> 4;
            const uint64_t a0 = ptx::desc_sw128(sbase, q.a_mn ? kOperand / 2 : 16u, 1024);
            const uint64_t b0 = ptx::desc_sw128(sbase + kOperand, q.b_mn ? kOperand / 2 : 16u, 1024);
            for (int at = w.b0; at < w.b1 && ok; at += flush, ++n_tile) {
                const int ac = n_tile & 1;
                if (!(ok = wait_bar(&ctl.acc_empty[ac], ((n_tile >> 1) & 1) ^ 1, &ctl, p))) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem + ac * kTileN;
                const int blocks = min(w.b1 - at, flush) * p.segs;
                for (int k = 0; k < blocks; ++k) {
                    if (!(ok = wait_bar(&ctl.full[st], phase, &ctl, p))) break;
                    ptx::tc_fence_after();
                    if (leader) {
                        const uint64_t a = a0 + st * (kStage >> 4), b = b0 + st * (kStage >> 4);
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j) mma_pair(d, a + j * step_a, b + j * step_b, idesc, (k | j) != 0);
                        commit_pair(&ctl.empty[st]);
                    }
                    __syncwarp();
                    if (++st == kStages) st = 0, phase ^= 1;
                }
                if (ok && leader) commit_pair(&ctl.acc_full[ac]);
                __syncwarp();
            }
        }
        if (!ok && leader) {  // no MMA is in flight when the tensor memory is freed
            commit_pair(&ctl.drain);
            ptx::mbar_wait(&ctl.drain, 0, 10000000ull);
        }
    } else if (warp >= 4) {
        // ---- epilogue: thread = row of this CTA's half of the tile, 128 of its columns
        if (p.late) ptx::griddep_wait();
        const int sub = warp & 3, half = (warp - 4) >> 2;
        const float scale = MODE == kGrads ? reference_dloss(p.dloss) : 1.f;
        uint32_t turn = 0;
        int n_tile = 0;
        bool ok = true;
        for (int i = 0, t; ok && (t = nth_tile(p, pair, pairs, i)) < total; ++i) {
            const Tile w = tile_at(p, t);
            const long long base = MODE == kGrads && w.which ? p.v0 : 0;  // dweight's rows are the piece's
            const long long row0 = base + static_cast<long long>(w.m) * kTileM + rank * kHalf + sub * 32;
            for (int at = w.b0; at < w.b1; at += flush, ++n_tile) {
                const int ac = n_tile & 1;
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.acc_full[ac], (n_tile >> 1) & 1, &ctl, p));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t taddr = tmem + ac * kTileN + half * kEpiCols + (static_cast<uint32_t>(sub * 32) << 16);
                const EpiTile e{p, w, taddr, row0, row0 + lane, half, lane,
                                sbase + kStages * kStage + static_cast<uint32_t>(warp - 4) * 2 * kOutTile, &turn};
                if constexpr (MODE == kStats) epilogue_stats(e);
                if constexpr (MODE == kDlogits) epilogue_dlogits(e, &maps.out);
                if constexpr (MODE == kGrads) {
                    const bool more = at > w.b0;  // the tile's first part has been stored, by this warp
                    if (more && lane == 0) ptx::bulk_wait_group0();
                    __syncwarp();
                    if (w.which == 0)
                        epilogue_f32(e, &maps.out, p.rows, p.acc_ld, w.split, more || !p.first, scale);
                    else if (!p.dw_vec)
                        epilogue_elements(e, more, scale);
                    else if (p.dw_f32)
                        epilogue_f32(e, &maps.dw, p.v1, p.dim, 0, more, scale);
                    else
                        epilogue_bf16(e, &maps.dw, p.v1, p.dim, scale);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_remote(map_rank(ptx::smem_u32(&ctl.acc_empty[ac]), 0));
            }
        }
        if (lane == 0) ptx::bulk_wait_group0();  // the last output tiles have left
    }
    __syncwarp();
    if (p.late) ptx::griddep_wait();
    ptx::tc_fence_before();
    cluster_sync();
    ptx::tc_fence_after();
    if (warp == 2) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------- around the products
// The fp32 product of one row of hidden and its target's row of weight, by one warp.
template <typename T>
__device__ __forceinline__ float dot_row(const T* a, const T* b, long long dim, bool vec, int lane) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    float s[2] = {0.f, 0.f};
    if (vec) {
#pragma unroll 4
        for (long long c = lane * V; c < dim; c += 32 * V) {
            elem::Pack<T, V> x, y;
            x.load(a + c), y.load(b + c);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i & 1] = fmaf(x.get(i), y.get(i), s[i & 1]);
        }
    } else {
#pragma unroll 2
        for (long long c = lane * V; c < dim; c += 32 * V) {  // the same sums in the same order
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < dim) s[i & 1] = fmaf(static_cast<float>(a[c + i]), static_cast<float>(b[c + i]), s[i & 1]);
        }
    }
    float v = s[0] + s[1];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// lse and loss of eight rows per CTA: 32 threads per row take every 32nd pair of
// statistics, and a warp joins the row's. The tensor cores' sum of the target's logit is off by about
// one ulp per 16 of depth; a trained row's loss is that error, so the target's
// term is replaced by the logit summed in fp32, in the loss and in the lse.
constexpr int kLseRows = 8, kLseGroups = 32;
template <typename T>
__global__ void __launch_bounds__(kLseRows * kLseGroups)
    ce_lse(const float2* stats, const float* picked, const long long* __restrict__ target,
           const T* __restrict__ hidden, long long stride, const T* __restrict__ weight, long long dim, int vec,
           long long ignore, long long rows, long long vocab, int parts, float* loss, float* lse) {
    __shared__ float sm[kLseGroups][kLseRows + 1], ss[kLseGroups][kLseRows + 1];
    const long long row0 = static_cast<long long>(blockIdx.x) * kLseRows;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long mine = row0 + ty;  // the row that this warp joins
    const long long t = mine < rows ? target[mine] : ignore;
    const bool real = t != ignore && t >= 0 && t < vocab;
    float logit = 0.f;
    if (real) logit = dot_row(hidden + mine * stride, weight + t * dim, dim, vec != 0, tx);
    ptx::griddep_wait();  // stats and picked
    {
        const int r = threadIdx.x % kLseRows, group = threadIdx.x / kLseRows;
        const long long row = row0 + r;
        float m = -__builtin_inff(), s = 0.f;
        if (row < rows) {
#pragma unroll 4
            for (int t = group; t < parts; t += kLseGroups) {
                const float2 v = stats[t * rows + row];
                const float m2 = fmaxf(m, v.x), base = relative_to(m2);  // (half a tile past the vocabulary has no maximum)
                s = s * elem::exp2_fast((m - base) * elem::kLog2e) + v.y * elem::exp2_fast((v.x - base) * elem::kLog2e);
                m = m2;
            }
        }
        sm[group][r] = m;
        ss[group][r] = s;
    }
    __syncthreads();
    if (mine >= rows) return;
    const float m = sm[tx][ty];
    float s = ss[tx][ty];
    float top = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    s = m == -__builtin_inff() ? s : s * elem::exp2_fast((m - top) * elem::kLog2e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (real) s += expf(picked[mine] - top) * expm1f(logit - picked[mine]);
    if (tx == 0) {
        const float l = top + logf(s);
        lse[mine] = l;
        loss[mine] = t == ignore ? 0.f : real ? l - logit : __uint_as_float(0x7FC00000u);
    }
}

// The targets' logits in fp32, a warp per row, for the backward: a trained row's p - 1 at its
// target is the difference of that logit and the lse, which the forward took from this sum. (The
// tensor cores' sum is off by an ulp per 16 of depth: bf16 rows of 4096 with 1 - p = 2e-3 and 3e-5 had gradients 4 %
// and 260 % off by it, 0.2 % and 3 % so.)
template <typename T>
__global__ void __launch_bounds__(256)
    ce_targets(const T* __restrict__ hidden, long long stride, const T* __restrict__ weight, long long dim, int vec,
               const long long* __restrict__ target, long long ignore, long long rows, long long vocab, float* picked) {
    ptx::griddep_launch_dependents();
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const long long t = row < rows ? target[row] : ignore;
    if (t != ignore && t >= 0 && t < vocab) {
        const float v = dot_row(hidden + row * stride, weight + t * dim, dim, vec != 0, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) picked[row] = v;
    }
    ptx::griddep_wait();
}

// ---------------------------------------------------------------- few rows of fp32: statistics without packing
// Splitting the weight into bf16 planes and reading those costs 22 bytes per element, the
// weight itself 4. With few rows that is the bound, and fp32 FMAs are fast enough: here a CTA takes kFewV
// classes by all (at most RP) rows, with chunks of kFewK of depth in shared memory (a ring of copies) and the chunk's
// depth split over four pairs of warps, whose sums are added in a fixed order. A thread keeps 4 classes by
// RP / 4 rows, two partial sums each (even and odd depth: packed FMAs without a shuffle). Forward of rows x 3968
// x 19388, here and with packed planes: 8 rows 71 and 262 us, 23 134 and 263; 32 x 2560 x 50280 254 and 432 us, bound by
// the FMAs (33 TFLOP/s; 8 by 8 per thread measured the same). 64 rows as two passes: 451 and 435.
constexpr int kFewV = 64, kFewK = 64, kFewStages = 4, kFewPitch = kFewK + 4;  // (the pitch spreads rows over the banks)
constexpr int few_smem(int RP) { return 4 * kFewStages * (kFewV + RP) * kFewPitch; }
template <int RP, bool kVec>
__global__ void __launch_bounds__(256, 2)
    ce_few_stats(const float* __restrict__ hidden, long long stride, const float* __restrict__ weight, long long dim,
                 const long long* __restrict__ target, long long rows, long long vocab, float2* stats, float* picked) {
    extern __shared__ __align__(16) float sm[];
    constexpr int N = kVec ? 4 : 1, kLanes = kFewK / N, kPass = 256 / kLanes, kStageFloats = (kFewV + RP) * kFewPitch;
    ptx::griddep_launch_dependents();
    const long long v0 = static_cast<long long>(blockIdx.x) * kFewV;
    const int at_row = threadIdx.x / kLanes, at_col = threadIdx.x % kLanes * N;
    const int chunks = static_cast<int>((dim + kFewK - 1) / kFewK);
    auto load = [&](int chunk) {
        float* to = sm + chunk % kFewStages * kStageFloats + at_col;
        const long long k = static_cast<long long>(chunk) * kFewK + at_col;
        auto put = [&](int row, bool there, const float* src) {
            float* dst = to + row * kFewPitch;
            if (there && k < dim) {
                ptx::cp_async<4 * N>(ptx::smem_u32(dst), src + k);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) dst[i] = 0.f;
            }
        };
#pragma unroll
        for (int i = at_row; i < kFewV; i += kPass) put(i, v0 + i < vocab, weight + (v0 + i) * dim);
#pragma unroll
        for (int i = at_row; i < RP; i += kPass) put(kFewV + i, i < rows, hidden + i * stride);
    };
    using Pair = elem::Vals<2>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp >> 1;
    const int cls = (warp & 1) * 32 + (lane & 7), row = lane >> 3;  // this thread's first class and row
    Pair acc[4][RP / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RP / 4; ++j) acc[i][j] = Pair::splat(0.f);
    for (int c = 0; c < kFewStages - 1; ++c) {
        if (c < chunks) load(c);
        ptx::cp_async_commit();
    }
    for (int c = 0; c < chunks; ++c) {
        ptx::cp_async_wait<kFewStages - 2>();
        __syncthreads();  // chunk c is there, and chunk c - 1's stage is free
        if (c + kFewStages - 1 < chunks) load(c + kFewStages - 1);
        ptx::cp_async_commit();
        const float* st = sm + c % kFewStages * kStageFloats + part * (kFewK / 4);
#pragma unroll
        for (int k = 0; k < kFewK / 4; k += 4) {
            ulonglong2 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const ulonglong2*>(st + (cls + 8 * i) * kFewPitch + k);
#pragma unroll
            for (int j = 0; j < RP / 4; ++j) {
                const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(st + (kFewV + row + 4 * j) * kFewPitch + k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i][j] = elem::fma(Pair{w[i].y}, Pair{h.y}, elem::fma(Pair{w[i].x}, Pair{h.x}, acc[i][j]));
            }
        }
    }
    ptx::cp_async_wait<0>();
    __syncthreads();
    constexpr int kTo = kFewV + 1;  // [part][row][class]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RP / 4; ++j)
            sm[(part * RP + row + 4 * j) * kTo + cls + 8 * i] = acc[i][j].get(0) + acc[i][j].get(1);
    __syncthreads();
    constexpr int kPer = 256 / RP, kCols = kFewV / kPer;  // threads per row, and its classes of each
    const int mine = threadIdx.x / kPer, first = threadIdx.x % kPer;
    const long long t = mine < rows ? target[mine] : -1;
    float v[kCols], m = -__builtin_inff(), s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        const float* at = sm + mine * kTo + first + i * kPer;
        v[i] = (at[0] + at[RP * kTo]) + (at[2 * RP * kTo] + at[3 * RP * kTo]);
        const long long col = v0 + first + i * kPer;
        if (col >= vocab) v[i] = -__builtin_inff();  // not a class
        if (col == t && col < vocab) picked[mine] = v[i];
        m = fmaxf(m, v[i]);
    }
#pragma unroll
    for (int off = kPer / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
    for (int i = 0; i < kCols; ++i) s += elem::exp2_fast((v[i] - relative_to(m)) * elem::kLog2e);
#pragma unroll
    for (int off = kPer / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (first == 0 && mine < rows) stats[blockIdx.x * rows + mine] = make_float2(m, s);
}

// An operand as one (bf16) or three (fp32) bf16 planes of rows padded to 8 elements, eight
// of them per thread. Rows without a loss (target == ignore; target may be NULL) become zero.
template <typename T>
__global__ void __launch_bounds__(256)
    ce_pack(const T* __restrict__ src, long long stride, long long rows, long long dim, long long ld, int planes, int vec,
            const long long* __restrict__ target, long long ignore, __nv_bfloat16* __restrict__ dst) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const int per = static_cast<int>(ld / 8);
    const long long n = rows * per;
    ptx::griddep_launch_dependents();
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * 256) {
        const long long r = i / per;
        const int c = static_cast<int>(i - r * per) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
        if (!target || target[r] != ignore) {
            if (vec) {
#pragma unroll
                for (int k = 0; k < 8; k += N) {
                    elem::Pack<T, N> x;
                    x.load(src + r * stride + c + k);
#pragma unroll
                    for (int j = 0; j < N; ++j) v[k + j] = x.get(j);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < dim) v[k] = static_cast<float>(src[r * stride + c + k]);
            }
        }
        for (int p = 0; p < planes; ++p) {
            elem::Pack<__nv_bfloat16, 8> x;
            x.set(v);
            x.store(dst + p * rows * ld + r * ld + c);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] -= x.get(k);
        }
    }
    ptx::griddep_wait();
}

// dhidden from its accumulators, eight elements per thread.
template <typename T>
__global__ void __launch_bounds__(256)
    ce_finish(const float* acc, int splits, long long rows, long long dim, long long ld, int vec,
              T* __restrict__ out) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const int per = static_cast<int>(ld / 8);
    const long long n = rows * per;
    ptx::griddep_wait();
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * 256) {
        const long long r = i / per;
        const int c = static_cast<int>(i - r * per) * 8;
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = 0.f;
#pragma unroll 4
        for (int z = 0; z < splits; ++z) {
            const float4* a = reinterpret_cast<const float4*>(acc + (z * rows + r) * ld + c);
            const float4 x = a[0], y = a[1];
            s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
            s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
        }
        if (vec) {
#pragma unroll
            for (int k = 0; k < 8; k += N) {
                elem::Pack<T, N> x;
                x.set(s + k);
                x.store(out + r * dim + c + k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c + k < dim) {
                    elem::Pack<T, 1> x;
                    x.set(s + k);
                    x.store(out + r * dim + c + k);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- host side
constexpr long long kPieceBytes = 256ll << 20;  // dl of one piece, at most (one tile's width at least)
constexpr long long kWeightBytes = 64ll << 20;  // of a weight that is packed in pieces, likewise

long long up(long long v, long long m) { return (v + m - 1) / m * m; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kFewRows = 32;
// The accumulators truncate, one ulp per 16 of depth, which fp32 gradients over thousands of
// rows or classes would show; a part of 512 keeps that under the rounding of ordinary fp32 sums (dweight of 3175 x 159 x 36028:
// 3.9e-6 off in one part, under 1e-6 so; forward + backward 982 us both, 1500 x 1024 x 32000 1404 and 1480).
constexpr int kFlush = 8;
int pair_count() { return std::max(1, device_sms() / 2); }

// How the products read the weight: as it is; as a copy; or, where only its first element's
// address is in the way (bf16, dim a multiple of 8), as copies of one piece of the vocabulary after another, so
// that the workspace need not hold a copy of a weight that nearly always lies right.
enum Weight { kInPlace, kPacked, kPieces };

// Everything that follows from the sizes. Operands are packed where TMA cannot read
// them in place: fp32, or rows that do not start on 16 bytes.
struct CePlan {
    bool few;      // the forward of few fp32 rows: no packing, statistics of kFewV classes
    Weight form;
    long long ld;  // packed rows
    int planes, segs, piece, splits;  // (piece of the forward: the whole vocabulary but in kPieces)
    size_t hidden, weight, stats, picked, dl, acc, total;
};
CePlan ce_plan(long long rows, long long dim, long long vocab, ssd_dtype io, bool backward, bool pack_h, Weight form,
               int pairs) {
    CePlan c{};
    c.ld = up(dim, 8);
    c.planes = io == SSD_F32 ? 3 : 1;
    c.segs = io == SSD_F32 ? kMaxSegs : 1;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at = align_up(at + bytes, 1024);
        return r;
    };
    c.few = !backward && io == SSD_F32 && rows <= kFewRows;
    if (c.few) pack_h = false, form = kInPlace;
    c.form = form;
    const long long all = up(vocab, kTileN) / kTileN;  // tiles
    long long most = all;                              // and of one piece
    if (form == kPieces) most = std::min(all, std::max<long long>(1, kWeightBytes / (2 * c.ld * kTileN)));
    c.hidden = take(pack_h ? 2 * c.planes * rows * c.ld : 0);
    c.weight = take(form == kInPlace ? 0 : 2 * c.planes * std::min(vocab, most * kTileN) * c.ld);
    if (!backward) {
        c.piece = static_cast<int>(most * kTileN);
        c.stats = take(8 * (c.few ? up(vocab, kFewV) / kFewV : 2 * (up(vocab, kTileN) / kTileN)) * rows);
        c.picked = take(4 * rows);
    } else {
        most = std::min(most, std::max<long long>(1, kPieceBytes / (2ll * c.planes * rows * kTileN)));
        const long long pieces = (all + most - 1) / most;
        c.piece = static_cast<int>((all + pieces - 1) / pieces * kTileN);  // even pieces
        const long long tiles = up(rows, kTileM) / kTileM * (up(dim, kTileN) / kTileN);
        c.splits = static_cast<int>(std::max<long long>(1, std::min<long long>((c.planes > 1 ? 2 : 1) * pairs / tiles, c.piece / kBK / 4)));
        c.picked = take(4 * rows);
        c.dl = take(2ll * c.planes * rows * c.piece);
        c.acc = take(4ll * c.splits * rows * c.ld);
    }
    c.total = at;
    return c;
}

struct CeCall {
    long long rows, dim, vocab;
    ssd_dtype io;
    const void* hidden;
    long long hs;
    const void* weight;
    const long long* target;
    long long ignore;
    char* ws;
    cudaStream_t stream;
};

// Rows that start on 16 bytes and are a whole number of them.
bool whole16(const void* p, long long stride, const CeCall& c) {
    const long long v = c.io == SSD_BF16 ? 8 : 4;
    return c.dim % v == 0 && stride % v == 0 && aligned_to(p, 16);
}

// One thread per eight elements of the padded rows, a few waves of CTAs at most.
unsigned rows_grid(long long rows, long long ld) {
    return static_cast<unsigned>(std::min<long long>((rows * (ld / 8) + 255) / 256, 16ll * device_sms()));
}

// A call's kernels form a chain of programmatic launches: each starts while the one before it
// drains and waits on the device for what it reads, and every one waits for the one before it
// before it ends, so that a kernel's end means the end of all earlier ones. The
// first starts as usual (`after`: it is not the first; nor does one that overwrites what an earlier one reads). Forward +
// backward launched one after another and so: 301 x 771 x 8191 (fp32, ten kernels) 200 and 172 us, 512 x 768 x 32000 (bf16,
// then six) 118 and 115.
template <typename... P, typename... A>
void launch(bool after, void (*kernel)(P...), unsigned grid, unsigned block, int smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem), cfg.stream = stream;
    cfg.attrs = &attr, cfg.numAttrs = after ? 1u : 0u;
    cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);  // (an error stays for cudaGetLastError)
    note_launches(1);
}

template <typename T>
void pack(bool after, const void* src, long long stride, long long rows, bool drop, const CeCall& c, const CePlan& pl,
          void* dst) {
    const bool vec = c.dim % 8 == 0 && whole16(src, stride, c);
    launch(after, ce_pack<T>, rows_grid(rows, pl.ld), 256, 0, c.stream, static_cast<const T*>(src), stride, rows, c.dim,
           pl.ld, pl.planes, vec, drop ? c.target : nullptr, c.ignore, static_cast<__nv_bfloat16*>(dst));
}

// The operands as TMA reads them: in place or packed. The backward always packs
// hidden, with zeros in the rows without a loss: whatever they hold (a padding row may be
// infinite or NaN) stays out of dweight.
struct Operands {
    const void *h, *w;
    long long h_ld, w_ld;
};
bool in_place(const void* p, long long stride, const CeCall& c) {
    return c.io == SSD_BF16 && c.dim % 8 == 0 && stride == c.dim && aligned_to(p, 16);
}
Weight weight_form(const CeCall& c) {
    return in_place(c.weight, c.dim, c) ? kInPlace : c.io == SSD_BF16 && c.dim % 8 == 0 ? kPieces : kPacked;
}
// Rows [v0, v1) of the weight into the workspace, once nothing reads what is there (kPieces).
const void* pack_piece(const CeCall& c, const CePlan& pl, long long v0, long long v1) {
    void* dst = c.ws + pl.weight;
    pack<__nv_bfloat16>(false, static_cast<const __nv_bfloat16*>(c.weight) + v0 * c.dim, c.dim, v1 - v0, false, c, pl, dst);
    return dst;
}
Operands lay_out(const CeCall& c, const CePlan& pl, bool pack_h, bool drop) {
    const bool pack_w = pl.form == kPacked;
    Operands o{c.hidden, c.weight, c.dim, c.dim};
    auto one = [&](bool after, const void* src, long long stride, long long rows, bool zero, size_t at) -> const void* {
        void* dst = c.ws + at;
        if (c.io == SSD_BF16)
            pack<__nv_bfloat16>(after, src, stride, rows, zero, c, pl, dst);
        else
            pack<float>(after, src, stride, rows, zero, c, pl, dst);
        return dst;
    };
    if (pack_h) o.h = one(false, c.hidden, c.hs, c.rows, drop, pl.hidden), o.h_ld = pl.ld;
    if (pack_w) o.w = one(pack_h, c.weight, c.dim, c.vocab, false, pl.weight), o.w_ld = pl.ld;
    return o;
}

template <int MODE>
ssd_status launch_gemm(bool after, const Maps& maps, const CeParams& p, int pairs, cudaStream_t stream) {
    if (cudaFuncSetAttribute(ce_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return SSD_ERR_CUDA;
    const int jobs = p.jobs[0] + p.jobs[1];
    launch(after, ce_gemm<MODE>, 2u * std::min(pairs, jobs), kThreads, kSmem, stream, maps, p);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status base_params(const CeCall& c, const CePlan& pl, CeParams* p) {
    *p = CeParams{};
    p->rows = c.rows, p->vocab = c.vocab, p->dim = c.dim;
    p->target = c.target, p->ignore = c.ignore;
    p->segs = pl.segs, p->planes = pl.planes;
    // smallest products first
    static const int sa[kMaxSegs] = {2, 0, 1, 1, 0, 0}, sb[kMaxSegs] = {0, 2, 1, 0, 1, 0};
    for (int i = 0; i < pl.segs; ++i) {
        p->seg_a[i] = pl.segs == 1 ? 0 : sa[i];
        p->seg_b[i] = pl.segs == 1 ? 0 : sb[i];
    }
    unsigned long long unused;
    return call_context(&p->status, &unused);
}

ssd_status check_ce(ssd_dtype io, int64_t rows, int64_t dim, int64_t vocab) {
    if (io != SSD_F32 && io != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (rows < 1 || dim < 1 || vocab < 1) return SSD_ERR_INVALID_ARG;
    // TMA coordinates and tile counts are 32-bit
    if (rows >= (1ll << 30) || vocab >= (1ll << 30) || dim >= (1ll << 24)) return SSD_ERR_UNSUPPORTED;
    if (up(rows, kTileM) / kTileM * (up(vocab, kTileN) / kTileN) >= (1ll << 30)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd_status tile_stats(const CeCall& c, const CePlan& pl, bool pack_h, int pairs) {
    CeParams p;
    ssd_status st = base_params(c, pl, &p);
    if (st != SSD_OK) return st;
    const Operands o = lay_out(c, pl, pack_h, false);
    const bool pieces = pl.form == kPieces;
    p.stats = reinterpret_cast<float2*>(c.ws + pl.stats);
    p.picked = reinterpret_cast<float*>(c.ws + pl.picked);
    for (long long v0 = 0; v0 < c.vocab; v0 += pl.piece) {
        const long long v1 = std::min<long long>(c.vocab, v0 + pl.piece);
        const void* w = pieces ? pack_piece(c, pl, v0, v1) : o.w;
        Maps m{};
        if (!make_map_bf16(&m.a0, o.h, o.h_ld, 1, c.rows, pl.planes, 64) ||
            !make_map_bf16(&m.b0, w, o.w_ld, 1, v1 - v0, pl.planes, 64))
            return SSD_ERR_CUDA;
        m.a1 = m.a0, m.b1 = m.b0;
        p.v0 = static_cast<int>(v0), p.v1 = static_cast<int>(v1);
        Product& q = p.prod[0];
        q.tiles_m = static_cast<int>(up(c.rows, kTileM) / kTileM);
        q.tiles_n = static_cast<int>(up(v1 - v0, kTileN) / kTileN);
        q.splits = 1, q.blocks = static_cast<int>(up(pl.ld, kBK) / kBK), q.m_fast = 1;
        p.jobs[0] = q.tiles_m * q.tiles_n;
        st = launch_gemm<kStats>(pack_h || pl.form != kInPlace, m, p, pairs, c.stream);
        if (st != SSD_OK) return st;
    }
    return SSD_OK;
}

template <int RP>
ssd_status few_stats(const CeCall& c, const CePlan& pl, bool vec) {
    auto* kernel = vec ? ce_few_stats<RP, true> : ce_few_stats<RP, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(RP)) != cudaSuccess)
        return SSD_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(up(c.vocab, kFewV) / kFewV);
    launch(false, kernel, grid, 256, few_smem(RP), c.stream, static_cast<const float*>(c.hidden), c.hs,
           static_cast<const float*>(c.weight), c.dim, c.target, c.rows, c.vocab,
           reinterpret_cast<float2*>(c.ws + pl.stats), reinterpret_cast<float*>(c.ws + pl.picked));
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Statistics of all logits, then loss and lse from them.
ssd_status ce_forward(const CeCall& c, const CePlan& pl, bool pack_h, float* loss, float* lse, int pairs) {
    const bool vec = whole16(c.hidden, c.hs, c) && whole16(c.weight, c.dim, c);
    int parts;
    ssd_status st;
    if (pl.few) {
        parts = static_cast<int>(up(c.vocab, kFewV) / kFewV);
        st = c.rows <= 8 ? few_stats<8>(c, pl, vec) : c.rows <= 16 ? few_stats<16>(c, pl, vec) : few_stats<32>(c, pl, vec);
    } else {
        parts = static_cast<int>(2 * (up(c.vocab, kTileN) / kTileN));
        st = tile_stats(c, pl, pack_h, pairs);
    }
    if (st != SSD_OK) return st;
    const unsigned grid = static_cast<unsigned>((c.rows + kLseRows - 1) / kLseRows);
    auto join = [&](auto tag) {
        using T = decltype(tag);
        launch(true, ce_lse<T>, grid, kLseRows * kLseGroups, 0, c.stream, reinterpret_cast<const float2*>(c.ws + pl.stats),
               reinterpret_cast<const float*>(c.ws + pl.picked), c.target, static_cast<const T*>(c.hidden), c.hs,
               static_cast<const T*>(c.weight), c.dim, vec, c.ignore, c.rows, c.vocab, parts, loss, lse);
    };
    if (c.io == SSD_BF16)
        join(__nv_bfloat16());
    else
        join(float());
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ce_backward(const CeCall& c, const CePlan& pl, const float* dloss, const float* lse, void* dhidden, void* dweight,
                       int pairs) {
    CeParams p;
    ssd_status st = base_params(c, pl, &p);
    if (st != SSD_OK) return st;
    const Operands o = lay_out(c, pl, true, true);
    const bool pieces = pl.form == kPieces;
    p.lse = lse, p.dloss = dloss, p.acc_ld = pl.ld;
    void* dl = c.ws + pl.dl;
    float* acc = reinterpret_cast<float*>(c.ws + pl.acc);
    p.dweight = dweight, p.dw_f32 = c.io == SSD_F32;
    p.dw_vec = c.dim % (p.dw_f32 ? 4 : 8) == 0 && aligned_to(dweight, 16);
    Maps logits{}, grads{};
    // The logits come from hidden itself where they can (a row without a loss has none that count):
    // their products then run beside the packing and the targets' logits.
    const bool beside = in_place(c.hidden, c.hs, c) && pl.form == kInPlace;
    if (!make_map_bf16(&logits.a0, beside ? c.hidden : o.h, beside ? c.dim : o.h_ld, 1, c.rows, pl.planes, 64) ||
        !make_map_bf16(&logits.out, dl, pl.piece, 1, c.rows, pl.planes, 32) ||
        !make_map_bf16(&grads.a0, dl, pl.piece, 1, c.rows, pl.planes, 64) ||
        !make_map_bf16(&grads.a1, dl, pl.piece, 1, c.rows, pl.planes, 64) ||
        !make_map_bf16(&grads.b1, o.h, o.h_ld, 1, c.rows, pl.planes, 64) ||
        !make_map_f32(&grads.out, acc, pl.ld, 1, c.rows, pl.splits, 32))
        return SSD_ERR_CUDA;
    if (p.dw_vec && !(p.dw_f32 ? make_map_f32(&grads.dw, dweight, c.dim, 1, c.vocab, 1, 32)
                               : make_map_bf16(&grads.dw, dweight, c.dim, 1, c.vocab, 1, 32)))
        return SSD_ERR_CUDA;
    logits.a1 = logits.a0;
    p.picked = reinterpret_cast<float*>(c.ws + pl.picked);
    auto targets = [&](auto tag) {
        using T = decltype(tag);
        launch(true, ce_targets<T>, static_cast<unsigned>((c.rows + 7) / 8), 256, 0, c.stream,
               static_cast<const T*>(c.hidden), c.hs, static_cast<const T*>(c.weight), c.dim,
               whole16(c.hidden, c.hs, c) && whole16(c.weight, c.dim, c), c.target, c.ignore, c.rows, c.vocab, p.picked);
    };
    if (c.io == SSD_BF16)
        targets(__nv_bfloat16());
    else
        targets(float());
    const int tiles_r = static_cast<int>(up(c.rows, kTileM) / kTileM);
    const int tiles_d = static_cast<int>(up(c.dim, kTileN) / kTileN);
    for (long long v0 = 0; v0 < c.vocab; v0 += pl.piece) {
        const long long v1 = std::min<long long>(c.vocab, v0 + pl.piece);
        const int tiles_v = static_cast<int>(up(v1 - v0, kTileN) / kTileN);
        p.v0 = static_cast<int>(v0), p.v1 = static_cast<int>(v1), p.first = v0 == 0;
        if (v0 == 0 || pieces) {
            const void* w = pieces ? pack_piece(c, pl, v0, v1) : o.w;
            if (!make_map_bf16(&logits.b0, w, o.w_ld, 1, pieces ? v1 - v0 : c.vocab, pl.planes, 64)) return SSD_ERR_CUDA;
            grads.b0 = logits.b1 = logits.b0;
        }
        const int w_row = pieces ? 0 : p.v0;
        CeParams a = p;
        Product& q = a.prod[0];
        q = Product{};
        q.b_row = w_row;
        q.tiles_m = tiles_r, q.tiles_n = tiles_v, q.splits = 1;
        q.blocks = static_cast<int>(up(pl.ld, kBK) / kBK), q.m_fast = 1;
        a.jobs[0] = tiles_r * tiles_v;
        a.late = v0 == 0 && beside;
        st = launch_gemm<kDlogits>(true, logits, a, pairs, c.stream);
        if (st != SSD_OK) return st;
        CeParams b = p;
        Product& dh = b.prod[0];  // [rows, dim] = dl [rows, piece] weight [piece, dim]
        dh.b_mn = 1, dh.b_dep = w_row;
        dh.tiles_m = tiles_r, dh.tiles_n = tiles_d, dh.splits = pl.splits;
        dh.blocks = tiles_v * (kTileN / kBK);
        b.jobs[0] = tiles_r * tiles_d * pl.splits;
        Product& dw = b.prod[1];  // [piece, dim] = dl^T [piece, rows] hidden [rows, dim]
        dw.a_mn = dw.b_mn = 1;
        dw.tiles_m = tiles_v, dw.tiles_n = tiles_d, dw.splits = 1;
        dw.blocks = static_cast<int>(up(c.rows, kBK) / kBK);
        b.jobs[1] = tiles_v * tiles_d;
        // a tile costs its products, but no less than its way out: about eight 64-deep ones (1 row,
        // 1600 x 58577, forward + backward: 363 us by the products alone, 229 so)
        auto cost = [&](int blocks) { return std::max(blocks * p.segs, 8); };
        b.flush = pl.planes > 1 ? kFlush : kNoFlush;
        b.lead = (cost(dh.blocks / dh.splits) + cost(dw.blocks) / 2) / cost(dw.blocks);
        st = launch_gemm<kGrads>(true, grads, b, pairs, c.stream);
        if (st != SSD_OK) return st;
    }
    const unsigned grid = rows_grid(c.rows, pl.ld);
    const bool vec = c.dim % 8 == 0 && aligned_to(dhidden, 16);
    if (c.io == SSD_BF16)
        launch(true, ce_finish<__nv_bfloat16>, grid, 256, 0, c.stream, acc, pl.splits, c.rows, c.dim, pl.ld, vec,
               static_cast<__nv_bfloat16*>(dhidden));
    else
        launch(true, ce_finish<float>, grid, 256, 0, c.stream, acc, pl.splits, c.rows, c.dim, pl.ld, vec,
               static_cast<float*>(dhidden));
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

bool ce_aligned(ssd_dtype io, std::initializer_list<const void*> io_ptrs, std::initializer_list<const void*> f32_ptrs,
                const void* target) {
    for (const void* q : io_ptrs)
        if (!aligned_to(q, io == SSD_BF16 ? 2 : 4)) return false;
    for (const void* q : f32_ptrs)
        if (!aligned_to(q, 4)) return false;
    return aligned_to(target, 8);
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_linear_cross_entropy_workspace_bytes(ssd_dtype io_dtype, int64_t rows, int64_t dim, int64_t vocab, int backward) {
    using namespace ssd;
    if (check_ce(io_dtype, rows, dim, vocab) != SSD_OK) return 0;
    const int pairs = pair_count();
    auto bytes = [&](Weight form) { return ce_plan(rows, dim, vocab, io_dtype, backward != 0, true, form, pairs).total; };
    if (io_dtype == SSD_F32 || dim % 8 != 0) return bytes(kPacked);
    return std::max(bytes(kInPlace), bytes(kPieces));  // wherever the weight starts
}

ssd_status ssd_linear_cross_entropy(ssd_dtype io_dtype, int64_t rows, int64_t dim, int64_t vocab, const void* hidden,
                                    int64_t hidden_row_stride, const void* weight, const int64_t* target,
                                    int64_t ignore_index, float* loss, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    using namespace ssd;
    const ssd_status st = check_ce(io_dtype, rows, dim, vocab);
    if (st != SSD_OK) return st;
    if (!hidden || !weight || !target || !loss || !lse || hidden_row_stride < dim) return SSD_ERR_INVALID_ARG;
    if (!ce_aligned(io_dtype, {hidden, weight}, {loss, lse}, target)) return SSD_ERR_UNSUPPORTED;
    const CeCall c{rows, dim, vocab, io_dtype, hidden, hidden_row_stride, weight,
                   reinterpret_cast<const long long*>(target), ignore_index, static_cast<char*>(workspace),
                   static_cast<cudaStream_t>(stream)};
    const bool pack_h = !in_place(hidden, hidden_row_stride, c);
    const int pairs = pair_count();
    const CePlan pl = ce_plan(rows, dim, vocab, io_dtype, false, pack_h, weight_form(c), pairs);
    if (!workspace || !aligned_to(workspace, kWorkspaceAlign) || workspace_bytes < pl.total) return SSD_ERR_WORKSPACE;
    return ce_forward(c, pl, pack_h, loss, lse, pairs);
}

ssd_status ssd_linear_cross_entropy_bwd(ssd_dtype io_dtype, int64_t rows, int64_t dim, int64_t vocab, const float* dloss,
                                        const void* hidden, int64_t hidden_row_stride, const void* weight,
                                        const int64_t* target, int64_t ignore_index, const float* lse, void* dhidden,
                                        void* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssd;
    const ssd_status st = check_ce(io_dtype, rows, dim, vocab);
    if (st != SSD_OK) return st;
    if (!dloss || !hidden || !weight || !target || !lse || !dhidden || !dweight || hidden_row_stride < dim)
        return SSD_ERR_INVALID_ARG;
    if (!ce_aligned(io_dtype, {hidden, weight, dhidden, dweight}, {dloss, lse}, target)) return SSD_ERR_UNSUPPORTED;
    const CeCall c{rows, dim, vocab, io_dtype, hidden, hidden_row_stride, weight,
                   reinterpret_cast<const long long*>(target), ignore_index, static_cast<char*>(workspace),
                   static_cast<cudaStream_t>(stream)};
    const int pairs = pair_count();
    const CePlan pl = ce_plan(rows, dim, vocab, io_dtype, true, true, weight_form(c), pairs);
    if (!workspace || !aligned_to(workspace, kWorkspaceAlign) || workspace_bytes < pl.total) return SSD_ERR_WORKSPACE;
    return ce_backward(c, pl, dloss, lse, dhidden, dweight, pairs);
}

}  // extern "C"
