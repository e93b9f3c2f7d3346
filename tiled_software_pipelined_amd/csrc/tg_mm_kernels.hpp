// Kernels on the 16-bit product tiles, one for each fused end, and the table
// that the host picks from.
#pragma once

#include <climits>

#include "tg_mm.hpp"

namespace tg {

struct MmGrid {
    int32_t tiles_m, tiles_n;
};

// How a launch's tiles are dealt to the compute units.  `slots` workgroups are on
// the machine at once: the first `full` tiles fill it whole times, and the rest
// are shared out along k, `splits` workgroups a tile of `per` slices each, whose
// sums are joined by a kernel of its own.  Sharing costs that launch and the
// sums' way through memory: about 9 us and 2.5 TB/s, against (1 - 1 / splits) of a
// tile's slices at `slice` ns each (64 tiles of 44 slices: shared out 18.7 us,
// not 16.1; of 172 slices 35 against 79).  Host and device come to the same answer
// (whole numbers).
struct MmSchedule {
    int32_t full, rest, splits, per;
    __host__ __device__ __forceinline__ int total() const { return full + rest * splits; }
};
// more parts than 16 pay nowhere: 60x768x50257 in 16 takes 24 us and 6 for the
// join, in 64 27 and 15
constexpr int MM_SPLITS = 16, MM_LEAST_SLICES = 8;
__host__ __device__ __forceinline__ MmSchedule mm_schedule(int tiles, int slices, int slots, int slice, int tile_kb, bool may_split) {
    MmSchedule s{tiles, 0, 1, slices};
    const int rest = tiles % slots;
    if (!may_split || rest == 0 || 2 * rest > slots || slices < MM_LEAST_SLICES) return s;
    int64_t least = (int64_t)slices * slice;
    for (int n = 2; n <= MM_SPLITS && n * rest <= slots && slices >= 4 * n; ++n) {
        const int per = (slices + n - 1) / n;
        if ((n - 1) * per >= slices) continue;  // a part would be empty
        const int64_t t = (int64_t)per * slice + 9000 + n * rest * tile_kb * 2 / 5;
        if (t < least) {
            least = t;
            s = MmSchedule{tiles - rest, rest, n, per};
        }
    }
    return s;
}

// ---- products that are only stored -------------------------------------------
// One C = alpha (a b^T [+ a' b'^T]); up to three of them share a launch.
struct MmJob {
    MmOperands op[2];
    int32_t pairs;
    MmGrid grid;
    void* C;        // result, row stride ldc elements
    int64_t ldc;
    float* sum;     // not NULL: float sums (M x N) instead
    int32_t add;    // sum: add to what is there
    // C's rows are whole cache lines: they go past the caches, which keep the
    // operands (32000x4096x2048 across k 467 -> 444 us)
    int32_t stream;
};
struct MmStoreArgs {
    MmJob job[3];
    int32_t jobs;
    const float* alpha;  // NULL: one
    const float* row_alpha;  // not NULL: that of each row, in alpha's place
    // A number of rows that only the device knows (NULL: as the operands say): the
    // first job's M, or its K (rows_are_k; then rounded up to 64, operands being
    // zero between), up to what the operands say.
    const int32_t* rows;
    int32_t rows_are_k;
    const int32_t* map;  // not NULL: row m of the result is row map[m] of C
    float* split;        // not NULL: room for the sums of tiles that are shared out
};

// ---- gated feed-forward: gate and up projections ---------------------------------
struct MmGateArgs {
    MmOperands op;
    MmGrid grid;
    // M x N, row stride ld; anything may be written between N and ld.  h: act(g) u; the
    // others: Kept24 of g and u, NULL where they are not kept
    void *h, *gate, *up, *low;
    int64_t ld;
    int32_t act;
};
// ---- its backward: dh = dy Wd, then du = dh act(g) and dg = dh act'(g) u ---------
struct MmDhArgs {
    MmOperands op;
    MmGrid grid;
    const void *gate, *up, *low;  // Kept24 of g and u
    // M x N, row stride ld, as the others; NULL where they are not wanted.  h: act(g) u
    // again, rounded.  Anything may be written between N and ld
    void *dg, *du, *h;
    int64_t ld;
    int32_t act;
};

// g and u in 24 bits each, for the backward pass: a sign, float's 8 bits of exponent
// and 15 behind the point (off by 2^-16), the upper halves of eight g, those of
// eight u, and a byte more of each.  act(g) and act'(g) u are made from them in
// float and rounded with dh, as du and dg.  In 16 bits themselves, in as many bytes
// with h, they would add a rounding (gradients off by 2.9e-3 of their norm in
// bfloat16, 2.3e-3 so) and those of closed gates would have no digits in float16
// (silu(-18) off by 9 %, silu(-21) zero), though a scaled loss's dh makes numbers of
// them that it holds.  It costs 2 % of a training step of 4096x4096x11008.
struct Kept24 {
    i32x4 g, u, low;
    __device__ static __forceinline__ uint32_t rounded(float v) {
        // a NaN's bits could be carried over into a number's
        return v != v ? 0x7fc00000u : __builtin_bit_cast(uint32_t, v) + 0x80u;
    }
    __device__ __forceinline__ void set(const float (&gs)[8], const float (&us)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t g0 = rounded(gs[2 * i]), g1 = rounded(gs[2 * i + 1]), u0 = rounded(us[2 * i]), u1 = rounded(us[2 * i + 1]);
            g[i] = (int)__builtin_amdgcn_perm(g1, g0, 0x07060302u);
            u[i] = (int)__builtin_amdgcn_perm(u1, u0, 0x07060302u);
            // the bytes below: of g0, u0, g1, u1
            low[i] = (int)__builtin_amdgcn_perm(__builtin_amdgcn_perm(u1, g1, 0x0c0c0501u), __builtin_amdgcn_perm(u0, g0, 0x0c0c0501u), 0x05040100u);
        }
    }
    __device__ __forceinline__ void get(float (&gs)[8], float (&us)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gs[2 * i] = __builtin_bit_cast(float, __builtin_amdgcn_perm((uint32_t)g[i], (uint32_t)low[i], 0x0504000cu));
            gs[2 * i + 1] = __builtin_bit_cast(float, __builtin_amdgcn_perm((uint32_t)g[i], (uint32_t)low[i], 0x0706020cu));
            us[2 * i] = __builtin_bit_cast(float, __builtin_amdgcn_perm((uint32_t)u[i], (uint32_t)low[i], 0x0504010cu));
            us[2 * i + 1] = __builtin_bit_cast(float, __builtin_amdgcn_perm((uint32_t)u[i], (uint32_t)low[i], 0x0706030cu));
        }
    }
};

// ---- cross entropy ---------------------------------------------------------------
// Rows of x are those that count, gathered; how many only the device knows.
struct MmStatsArgs {
    MmOperands op;
    MmGrid grid;
    const int32_t* rows;
    const int32_t* map;     // their places in target
    const int64_t* target;
    float2* part;  // (max, sum of 2^((z - max) log2 e)) of each wave's columns: part[piece M + row]
    float* hit;    // the target's logit of a row, where it has one
    uint16_t* powers;  // KEEP: 2^((z - max) log2 e) of every logit, as power_code has it, M x N
    int64_t ldp;       // their row stride; anything may be written between
};
// A kept power, which is at most one, in 16 bits without a sign.  For bfloat16: 7
// bits of an exponent and 9 behind the point, over float's normal numbers up to
// one, as far as bfloat16 itself reaches; off by 2^-10, a quarter of what rounding
// dz adds (elements of dz off by 1.71e-3; 1.66e-3 from logits made again, 2.35e-3
// from powers kept as bfloat16 numbers).  For float16: 5 and 11, off by 2^-12, half
// of what rounding dz adds; evenly spaced by 2^-41 below 2^-30, finer than float16's
// dz.  Times SCALE, a float's own bits are the code with more behind it; SHIFT
// brings the code to the upper half.  A NaN becomes some number: its row's sum has
// it.
template <class T>
struct Power {
    static constexpr int SHIFT = 2;
    static constexpr float SCALE = 1.0f, BACK = 1.0f;
};
template <>
struct Power<_Float16> {
    static constexpr int SHIFT = 4;
    static constexpr float SCALE = 0x1p-96f, BACK = 0x1p96f;
};
template <class T>
__device__ __forceinline__ uint32_t power_code(float power) {
    return (__builtin_bit_cast(uint32_t, power * Power<T>::SCALE) << Power<T>::SHIFT) + 0x8000u;
}
// SCALE times the power of a code that stands in the lower half.
template <class T>
__device__ __forceinline__ float power_of(uint32_t code) {
    return __builtin_bit_cast(float, (code & 0xffffu) << (16 - Power<T>::SHIFT));
}
struct MmDzArgs {
    MmOperands op;   // b: rows v0 .. of W
    MmGrid grid;
    const int32_t* rows;
    const int32_t* map;
    const int64_t* target;
    int64_t v0;
    const float2* lse;  // (max, log2 of the sum above it) of each row
    const float* coef;  // likewise
    void* dz;           // M x N, row stride ldz elements; anything may be written between
    int64_t ldz;
};

// Activations and their derivatives, by the C ABI's numbers.
enum MmAct { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3 };

__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(-1.44269504f * x); }

// a = act(g), d = act'(g), 8 at a time (the choice of activation is outside).
template <bool D>
__device__ __forceinline__ void activate8(int act, const float (&g)[8], float (&a)[8], float (&d)[8]) {
    switch (act) {
        case ACT_SILU:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // exp past float's range makes s zero
                const float s = __builtin_amdgcn_rcpf(1.0f + exp_neg(g[e]));
                a[e] = g[e] * s;
                if (D) d[e] = s * (1.0f + g[e] * (1.0f - s));
            }
            break;
        case ACT_GELU:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = 0.5f * erfcf(-0.70710678f * g[e]);  // erfc: small tails keep their digits
                a[e] = g[e] * p;
                if (D) d[e] = p + g[e] * 0.39894228f * exp_neg(0.5f * g[e] * g[e]);
            }
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (1 + tanh t) / 2 = 1 / (1 + exp(-2 t)).  Past 30 it is 0 or 1 and the
                // powers of g would only overflow
                const float c = g[e] != g[e] ? g[e] : fminf(fmaxf(g[e], -30.0f), 30.0f), c2 = c * c;
                const float s = __builtin_amdgcn_rcpf(1.0f + exp_neg(1.59576912f * c * (1.0f + 0.044715f * c2)));
                a[e] = g[e] * s;
                if (D) d[e] = s * (1.0f + (1.0f - s) * 1.59576912f * c * (1.0f + 0.134145f * c2));
            }
            break;
        default:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = g[e] > 0.0f ? g[e] : g[e] != g[e] ? g[e] : 0.0f;
                if (D) d[e] = g[e] > 0.0f ? 1.0f : 0.0f;
            }
    }
}

// Where a workgroup's tile is, and its wave's block.
template <class G>
struct MmPlace {
    int m0, n0, wm0, wn0, wave, lane;
    __device__ __forceinline__ MmPlace(const MmGrid& g, int tile) {
        wave = wave_id();
        lane = lane_id();
        int tm, tn;
        grouped_tile(tile, g.tiles_m, g.tiles_n, 4, tm, tn);
        m0 = tm * G::BM;
        n0 = tn * G::TILE_N;
        wm0 = (wave / G::WAVES_N) * G::WTM;
        wn0 = (wave % G::WAVES_N) * G::WTN;
    }
    // first row and column of C of the wave's block, the same for the whole wave
    __device__ __forceinline__ int row0() const { return m0 + wm0; }
    __device__ __forceinline__ int col0() const { return n0 + (wn0 / G::WTN) * G::WAVE_N; }
};

// The tiles of a launch's jobs, with what only the device knows.
struct MmTilesOf {
    int M, most_k, tiles, slices;  // M: of a lone job
    MmGrid grid;                   // likewise
};
template <int BM>
__device__ __forceinline__ MmTilesOf mm_tiles(const MmStoreArgs& g) {
    MmTilesOf t;
    t.grid = g.job[0].grid;
    t.M = g.job[0].op[0].M;
    t.most_k = INT_MAX;
    if (g.rows) {
        const int rows = *g.rows;
        if (g.rows_are_k) {
            t.most_k = (rows + 63) / 64 * 64;
        } else {
            t.M = rows;
            t.grid.tiles_m = (rows + BM - 1) / BM;
        }
    }
    t.tiles = t.grid.tiles_m * t.grid.tiles_n;
    for (int i = 1; i < g.jobs; ++i) t.tiles += g.job[i].grid.tiles_m * g.job[i].grid.tiles_n;
    t.slices = 0;
    for (int p = 0; p < g.job[0].pairs; ++p) t.slices += (min(g.job[0].op[p].K, t.most_k) + 63) / 64;
    return t;
}
// The job of a tile; `tile` becomes its number there.
__device__ __forceinline__ int mm_job_of(const MmStoreArgs& g, int& tile) {
    int which = 0;
    for (; which + 1 < g.jobs; ++which) {
        const int n = g.job[which].grid.tiles_m * g.job[which].grid.tiles_n;
        if (tile < n) break;
        tile -= n;
    }
    return which;
}

// Where a wave's results stand in a row-major M x N matrix: for 8 of them, at(p, u)
// is their address and count(u) how many lie inside.
template <class G>
struct MmOut {
    int m1, n1, M, N, r0, c0;
    int64_t ld;
    uint32_t lane_at;  // elements from the wave's first of its rows
    __device__ __forceinline__ MmOut(const MmPlace<G>& place, int M_, int N_, int64_t ld_)
        : m1(place.row0()), n1(place.col0()), M(M_), N(N_), r0(G::lane_row(place.lane)), c0(G::lane_col(place.lane)), ld(ld_),
          lane_at((uint32_t)(r0 * ld_ + c0)) {}
    __device__ __forceinline__ bool inside() const { return G::inside(m1, n1, M, N); }
    template <class T>
    __device__ __forceinline__ T* at(T* p, int u) const { return p + ((int64_t)(m1 + u) * ld + n1) + lane_at; }
    __device__ __forceinline__ int row(int u) const { return m1 + u + r0; }
    __device__ __forceinline__ int col() const { return n1 + c0; }
    __device__ __forceinline__ int count(int u) const { return row(u) < M ? N - col() : 0; }
};

// SUM: for jobs with float sums (job.sum), which are not shared out.
template <class G, bool SUM>
__global__ __launch_bounds__(G::NT) void mm_store_kernel(MmStoreArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    TG_LDS char* smem = (TG_LDS char*)smem_raw;
    MmTilesOf all = mm_tiles<G::BM>(g);
    const MmSchedule plan = mm_schedule(all.tiles, all.slices, G::SLOTS, G::SLICE_NS, G::TILE_KB, g.split != nullptr);
    int tile = blockIdx.x, split = 0, t0 = 0, t1 = all.slices;
    if (tile >= plan.total()) return;
    float* shared = nullptr;
    if (tile < plan.full) {
        tile = xcd_rank(tile, plan.full);
    } else {
        // parts in the order of their k: workgroups of one XCD share operands
        const int r = xcd_rank(tile - plan.full, plan.rest * plan.splits);
        split = r / plan.rest;
        tile = r - split * plan.rest;
        shared = g.split + (int64_t)(tile * plan.splits + split) * (G::BM * G::BN);
        tile += plan.full;
        t0 = split * plan.per;
        t1 = min(t0 + plan.per, all.slices);
    }
    const int which = mm_job_of(g, tile);
    if (g.jobs > 1) {
        all.M = g.job[which].op[0].M;
        all.grid = g.job[which].grid;
    }
    const MmJob& job = g.job[which];
    const MmPlace<G> at(all.grid, tile);
    typename G::Acc acc;
    G::clear(acc);
    for (int p = 0; p < job.pairs; ++p) {
        MmOperands op = job.op[p];
        op.M = all.M;
        op.K = min(op.K, all.most_k);
        const int slices = (op.K + 63) / 64;
        if (t0 < slices && t1 > 0)
            G::product(op, at.m0, at.n0, max(t0, 0), min(t1, slices), smem, acc, at.wm0, at.wn0, at.lane, at.wave);
        t0 -= slices;
        t1 -= slices;
    }
    const int M = all.M, N = job.op[0].N;
    typedef float(&F8)[8];
    if constexpr (SUM) {
        const MmOut<G> out(at, M, N, N);
        float* sum = job.sum;
        const bool add = job.add != 0;
        struct Before {
            f32x4 v[2];
        };
        auto way = [&](auto inside) {
            G::template each_row<Before>(acc, smem, at.lane, at.wave, [&](int u, Before& b) {
                if (inside.value && add) __builtin_memcpy(&b, out.at(sum, u), 32);
            }, [&](int u, F8 v, F8, Before& b) {
                float* dst = out.at(sum, u);
                if (inside.value) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = add ? v[e] + b.v[e >> 2][e & 3] : v[e];
                    __builtin_memcpy(dst, v, 32);
                } else {
                    const int count = out.count(u);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < count) dst[e] = add ? dst[e] + v[e] : v[e];
                }
            });
        };
        if (out.inside()) way(Yes{});
        else way(No{});
    } else if (shared) {
        float* mine = shared + (at.wm0 + G::lane_row(at.lane)) * G::BN + at.wn0 + G::lane_col(at.lane);
        G::each_row(acc, smem, at.lane, at.wave, [&](int u, F8 v, F8) { __builtin_memcpy(mine + u * G::BN, v, 32); });
    } else {
        typedef typename G::T T;
        const float alpha = g.alpha ? *g.alpha : 1.0f;
        T* C = static_cast<T*>(job.C);
        const MmOut<G> out(at, M, N, job.ldc);
        const bool stream = job.stream != 0;
        struct Row {
            int to;
            float alpha;
        };
        auto way = [&](auto inside) {
            G::template each_row<Row>(acc, smem, at.lane, at.wave, [&](int u, Row& row) {
                row.to = inside.value ? out.row(u) : min(out.row(u), M - 1);
                row.alpha = g.row_alpha ? g.row_alpha[row.to] : alpha;
                if (g.map) row.to = g.map[row.to];
            }, [&](int u, F8 v, F8, Row& row) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= row.alpha;
                T* dst = C + (int64_t)row.to * out.ld + out.col();
                if (inside.value) {
                    if (stream) stream8(dst, v);
                    else store8(dst, v);
                } else {
                    store8(dst, v, out.count(u));
                }
            });
        };
        if (out.inside()) way(Yes{});
        else way(No{});
    }
}

// C = alpha sum of the parts of the tiles that mm_store_kernel shared out, in an
// order that does not depend on who ended first.  A workgroup takes 512 results of
// a tile: each wave adds a quarter of the parts.
constexpr int MM_JOIN = 512;
template <class T, int BM, int BN, int SLOTS>
__device__ __forceinline__ void mm_join(const MmStoreArgs& g, int slice, int tile_kb) {
    constexpr int PER = BM * BN / MM_JOIN;
    __shared__ f32x4 held[3][2][64];
    const MmTilesOf all = mm_tiles<BM>(g);
    const MmSchedule plan = mm_schedule(all.tiles, all.slices, SLOTS, slice, tile_kb, true);
    int tile = blockIdx.x / PER;
    if (tile >= plan.rest) return;
    const int lane = lane_id(), wave = wave_id();
    const int e = (blockIdx.x % PER) * MM_JOIN + lane * 8;
    const float* p = g.split + (int64_t)tile * plan.splits * (BM * BN) + e;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int per = (plan.splits + 3) / 4, end = min((wave + 1) * per, plan.splits);
#pragma unroll 4
    for (int s = wave * per; s < end; ++s) {
        float x[8];
        __builtin_memcpy(x, p + (int64_t)s * (BM * BN), 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += x[i];
    }
    if (wave > 0) {
        held[wave - 1][0][lane] = f32x4{v[0], v[1], v[2], v[3]};
        held[wave - 1][1][lane] = f32x4{v[4], v[5], v[6], v[7]};
    }
    __syncthreads();
    if (wave > 0) return;
    tile += plan.full;
    const int which = mm_job_of(g, tile);
    const MmJob& job = g.job[which];
    const MmGrid grid = g.jobs > 1 ? job.grid : all.grid;
    int tm, tn;
    grouped_tile(tile, grid.tiles_m, grid.tiles_n, 4, tm, tn);
    const int m = tm * BM + e / BN, n = tn * BN + e % BN, M = g.jobs > 1 ? job.op[0].M : all.M, N = job.op[0].N;
    if (m >= M || n >= N) return;
    const float alpha = g.row_alpha ? g.row_alpha[m] : g.alpha ? *g.alpha : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = (v[i] + held[0][i >> 2][lane][i & 3] + held[1][i >> 2][lane][i & 3] + held[2][i >> 2][lane][i & 3]) * alpha;
    T* dst = static_cast<T*>(job.C) + (int64_t)(g.map ? g.map[m] : m) * job.ldc + n;
    if (n + 8 <= N) store8(dst, v);
    else store8(dst, v, N - n);
}
template <class G>
__global__ __launch_bounds__(256) void mm_join_kernel(MmStoreArgs g) {
    mm_join<typename G::T, G::BM, G::BN, G::SLOTS>(g, G::SLICE_NS, G::TILE_KB);
}

// A float sum (job.sum) in the result's type and place, 4 columns a thread.
template <class T>
__global__ __launch_bounds__(256) void mm_round_kernel(MmStoreArgs g) {
    const MmJob& job = g.job[0];
    const int64_t N = job.op[0].N, quads = (N + 3) / 4, q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= (g.rows ? *g.rows : job.op[0].M) * quads) return;
    const int64_t m = q / quads, n = (q - m * quads) * 4;
    const int count = (int)min(N - n, (int64_t)4);
    const float* p = job.sum + m * N + n;
    float v[4] = {0, 0, 0, 0};
    if (count == 4) {
        __builtin_memcpy(v, p, 16);
    } else {
        for (int e = 0; e < 3; ++e)
            if (e < count) v[e] = p[e];
    }
    const float alpha = g.row_alpha ? g.row_alpha[m] : g.alpha ? *g.alpha : 1.0f;
    T o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (T)(v[e] * alpha);
    T* dst = static_cast<T*>(job.C) + (g.map ? g.map[m] : m) * job.ldc + n;
    if (count == 4) {
        __builtin_memcpy(dst, o, 8);
    } else {
        for (int e = 0; e < 3; ++e)
            if (e < count) dst[e] = o[e];
    }
}

template <class G>
__global__ __launch_bounds__(G::NT) void mm_gate_kernel(MmGateArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    TG_LDS char* smem = (TG_LDS char*)smem_raw;
    typedef typename G::T T;
    const MmPlace<G> at(g.grid, xcd_rank(blockIdx.x, gridDim.x));
    typename G::Acc acc;
    G::clear(acc);
    G::product(g.op, at.m0, at.n0, 0, (g.op.K + 63) / 64, smem, acc, at.wm0, at.wn0, at.lane, at.wave);
    const MmOut<G> out(at, g.op.M, (int)g.ld, g.ld);  // rows whole up to their stride: no edge inside them
    typedef float(&F8)[8];
    auto way = [&](auto inside) {
        G::each_row(acc, smem, at.lane, at.wave, [&](int u, F8 v, F8 w) {
            auto put = [&](void* p, F8 x) {
                if (inside.value || out.count(u) > 0) store8(out.at(static_cast<T*>(p), u), x);
            };
            float a[8], d[8];
            if (g.low) {  // for the backward pass: past the caches
                Kept24 k;
                k.set(v, w);
                auto keep = [&](void* p, i32x4 x) {
                    if (inside.value || out.count(u) > 0) __builtin_nontemporal_store(x, reinterpret_cast<i32x4*>(out.at(static_cast<T*>(p), u)));
                };
                keep(g.gate, k.g);
                keep(g.up, k.u);
                keep(g.low, k.low);
            }
            activate8<false>(g.act, v, a, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] *= w[e];
            put(g.h, a);  // its rounding: the down projection's operand
        });
    };
    if (out.inside()) way(Yes{});
    else way(No{});
}

template <class G>
__global__ __launch_bounds__(G::NT) void mm_dh_kernel(MmDhArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    TG_LDS char* smem = (TG_LDS char*)smem_raw;
    typedef typename G::T T;
    const MmPlace<G> at(g.grid, xcd_rank(blockIdx.x, gridDim.x));
    typename G::Acc acc;
    G::clear(acc);
    G::product(g.op, at.m0, at.n0, 0, (g.op.K + 63) / 64, smem, acc, at.wm0, at.wn0, at.lane, at.wave);
    const MmOut<G> out(at, g.op.M, (int)g.ld, g.ld);  // rows whole up to their stride: no edge inside them
    typedef float(&F8)[8];
    auto way = [&](auto inside) {
        G::template each_row<Kept24>(acc, smem, at.lane, at.wave, [&](int u, Kept24& k) {
            if (inside.value || out.count(u) > 0) {
                k.g = load16(out.at(static_cast<const T*>(g.gate), u));
                k.u = load16(out.at(static_cast<const T*>(g.up), u));
                k.low = load16(out.at(static_cast<const T*>(g.low), u));
            }
        }, [&](int u, F8 v, F8, Kept24& k) {
            // roundings of du, dg and h: operands of the products that follow
            auto put = [&](void* p, F8 x) {
                if (inside.value || out.count(u) > 0) store8(out.at(static_cast<T*>(p), u), x);
            };
            float gate[8], up[8], a[8], b[8], h[8];
            k.get(gate, up);
            activate8<true>(g.act, gate, a, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = a[e] * up[e];
                a[e] *= v[e];
                b[e] *= up[e] * v[e];
            }
            if (g.h) put(g.h, h);
            if (g.du) put(g.du, a);
            if (g.dg) put(g.dg, b);
        });
    };
    if (out.inside()) way(Yes{});
    else way(No{});
}

constexpr float LOG2E = 1.44269504f;
// exp(z - max) / sum, from (max, log2 sum).  z - max is exact where p is near one.
__device__ __forceinline__ float softmax_of(float z, float2 lse) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(z - lse.x, LOG2E, -lse.y));
}

// A product with as many rows as the device says.
template <class G>
struct MmKnown {
    MmOperands op;
    MmGrid grid;
    int total;
    __device__ __forceinline__ MmKnown(const MmOperands& o, const MmGrid& r, const int32_t* rows) : op(o), grid(r) {
        op.M = *rows;
        grid.tiles_m = (op.M + G::BM - 1) / G::BM;
        total = grid.tiles_m * grid.tiles_n;
    }
};

// The piece of the softmax that a wave's columns make: for each row their
// maximum and the sum of the powers above it.  A row is in lanes l and l + 32.
// KEEP: the powers are stored too, for a backward pass that then needs no logits.
template <class G, bool KEEP>
__global__ __launch_bounds__(G::NT) void mm_stats_kernel(MmStatsArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const MmKnown<G> known(g.op, g.grid, g.rows);
    if ((int)blockIdx.x >= known.total) return;
    const MmPlace<G> at(known.grid, xcd_rank(blockIdx.x, known.total));
    typename G::Acc acc;
    G::clear(acc);
    TG_LDS char* smem = (TG_LDS char*)smem_raw;
    G::product(known.op, at.m0, at.n0, 0, (g.op.K + 63) / 64, smem, acc, at.wm0, at.wn0, at.lane, at.wave);
    const int M = known.op.M, N = g.op.N, n1 = at.col0(), half = 4 * (at.lane >> 5);
    if (n1 >= N) return;                // wave-uniform, as is the next
    const bool edge = n1 + G::WTN > N;
    float2* part = g.part + (int64_t)(n1 / G::WTN) * g.op.M;
#pragma unroll
    for (int i = 0; i < G::FM; ++i) {
        const int m = at.row0() + 32 * i + (at.lane & 31);
        if (edge) {
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (n1 + 32 * j + 8 * (r >> 2) + half + (r & 3) >= N) acc[i][j][r] = -INFINITY;
        }
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) most = fmaxf(most, acc[i][j][r]);
        most = fmaxf(most, __shfl_xor(most, 32));
        const float base = most == -INFINITY ? 0.0f : most;  // nothing here, or nothing but -inf
        const int64_t t = (m < M ? g.target[g.map[m]] : -1) - n1;
        const int want = t >= 0 && t < G::WTN ? (int)t : -1;
        if (__any(want >= 0)) {
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * j + 8 * (r >> 2) + half + (r & 3) == want) g.hit[m] = acc[i][j][r];
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float power = __builtin_amdgcn_exp2f((acc[i][j][r] - base) * LOG2E);
                sum += power;
                if constexpr (KEEP) acc[i][j][r] = power;
            }
        sum += __shfl_xor(sum, 32);
        if (at.lane < 32 && m < M) part[m] = float2{most, sum};
    }
    if constexpr (KEEP) {
        typedef typename G::T T;
        const MmOut<G> out(at, M, (int)g.ldp, g.ldp);  // rows whole up to their stride
        auto way = [&](auto inside) {
            G::each_row(acc, smem, at.lane, at.wave, [&](int u, float (&v)[8], float (&)[8]) {
                i32x4 codes;
#pragma unroll
                for (int e = 0; e < 4; ++e)  // two upper halves
                    codes[e] = (int)__builtin_amdgcn_perm(power_code<T>(v[2 * e + 1]), power_code<T>(v[2 * e]), 0x07060302u);
                if (inside.value || out.count(u) > 0) __builtin_memcpy(out.at(g.powers, u), &codes, 16);
            });
        };
        if (out.inside()) way(Yes{});
        else way(No{});
    }
}

// dz = coef (softmax - [target]), rounded: the operand of the products for dx
// and dw.  Zero in the rows up to the next multiple of 64, so that the product
// over rows has no part of a slice.
template <class G>
__global__ __launch_bounds__(G::NT) void mm_dz_kernel(MmDzArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    TG_LDS char* smem = (TG_LDS char*)smem_raw;
    typedef typename G::T T;
    const MmKnown<G> known(g.op, g.grid, g.rows);
    if ((int)blockIdx.x >= known.total) return;
    const MmPlace<G> at(known.grid, xcd_rank(blockIdx.x, known.total));
    typename G::Acc acc;
    G::clear(acc);
    G::product(known.op, at.m0, at.n0, 0, (g.op.K + 63) / 64, smem, acc, at.wm0, at.wn0, at.lane, at.wave);
    const int M = known.op.M;
    T* dz = static_cast<T*>(g.dz);
    const MmOut<G> out(at, (M + 63) / 64 * 64, (int)g.ldz, g.ldz);  // rows whole up to their stride
    typedef float(&F8)[8];
    struct Row {
        float2 lse;
        float coef;
        int64_t target;
    };
    auto way = [&](auto inside) {
        G::template each_row<Row>(acc, smem, at.lane, at.wave, [&](int u, Row& row) {
            const int m = inside.value ? out.row(u) : min(out.row(u), M - 1);
            row.lse = g.lse[m];
            row.coef = g.coef[m];
            row.target = g.target[g.map[m]] - g.v0;
        }, [&](int u, F8 v, F8, Row& row) {
            const int64_t t = row.target - out.col();
            const int hit = t >= 0 && t < 8 ? (int)t : -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float p = softmax_of(v[e], row.lse);
                if (e == hit) p -= 1.0f;
                v[e] = p * row.coef;
            }
            if (inside.value) {
                store8(out.at(dz, u), v);
            } else {
                if (out.row(u) >= M) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                }
                if (out.count(u) > 0) store8(out.at(dz, u), v);
            }
        });
    };
    if (G::inside(out.m1, out.n1, M, out.N)) way(Yes{});
    else way(No{});
}

// ---- few rows of A -----------------------------------------------------------
// A served batch of up to 16 tokens is bound by one read of the weights (180 MB in
// 34 us, 5.3 TB/s, for one; 4096x11008 block in all 58 us for one token, 68 for
// 16, and 73 on the tiles for 17 to 64).  A workgroup takes 16 rows of B (PAIR: of
// both matrices) and all rows of A; its eight waves deal blocks of 64 k among them,
// operands going straight to registers, U blocks in flight, and add their sums
// through LDS.  v_mfma_f32_16x16x32: lane l holds row l % 16, k 8 (l / 16) .. + 7
// of 32; of a block's 128 bytes of a row it reads chunks l / 16 and 4 + l / 16,
// so one load reads 64 adjacent bytes of each of 16 rows.
constexpr int MM_ROWS = 16;
struct MmRowsArgs {
    MmOperands op;
    void* C;  // M x N, row stride ldc elements
    int64_t ldc;
    int32_t act;
};

template <class Tr, bool PAIR>
__global__ __launch_bounds__(512) void mm_rows_kernel(MmRowsArgs g) {
    constexpr int NW = 8, U = 4, NB = PAIR ? 2 : 1;
    __shared__ float part[NW][NB * 256];
    typedef typename Tr::T T;
    const MmOperands& o = g.op;
    const int lane = lane_id(), wave = wave_id();
    const int n0 = blockIdx.x * 16;
    const int blocks = (o.K + 63) / 64, bytes = o.K * 2, at = (lane >> 4) * 16;
    const char* brow[NB];
    brow[0] = o.b + (int64_t)min(n0 + (lane & 15), o.N - 1) * o.ldb;
    if constexpr (PAIR) brow[1] = o.b2 + (int64_t)min(n0 + (lane & 15), o.N - 1) * o.ldb2;
    const char* arow = o.a + (int64_t)min(lane & 15, o.M - 1) * o.lda;
    f32x4 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f32x4{0, 0, 0, 0};
    struct Block {
        i32x4 b[NB][2], a[2];
    };
    auto load = [&](Block& x, int kb) {
        const int64_t k0 = (int64_t)kb * 128 + at;
        if ((kb + 1) * 64 <= o.K) {  // wave-uniform
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int b = 0; b < NB; ++b) x.b[b][h] = load16(brow[b] + k0 + 64 * h);
                x.a[h] = load16(arow + k0 + 64 * h);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int b = 0; b < NB; ++b) x.b[b][h] = row_end_chunk(brow[b], (int)k0 + 64 * h, bytes);
                x.a[h] = row_end_chunk(arow, (int)k0 + 64 * h, bytes);
            }
        }
    };
    auto multiply = [&](const Block& x) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[b] = Tr::mma16(x.a[h], x.b[b][h], acc[b]);
    };
    int kb = wave;
    for (; kb + (U - 1) * NW < blocks; kb += U * NW) {
        Block x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load(x[u], kb + u * NW);
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(x[u]);
    }
    for (; kb < blocks; kb += NW) {
        Block x;
        load(x, kb);
        multiply(x);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][b * 256 + (4 * (lane >> 4) + r) * 16 + (lane & 15)] = acc[b][r];
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= 256) return;
    float v[8] = {}, w[8] = {}, a[8], d[8];
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        v[0] += part[k][e];
        if constexpr (PAIR) w[0] += part[k][256 + e];
    }
    if constexpr (PAIR) {
        activate8<false>(g.act, v, a, d);
        v[0] = a[0] * w[0];
    }
    const int m = e >> 4, n = n0 + (e & 15);
    if (m < o.M && n < o.N) static_cast<T*>(g.C)[m * g.ldc + n] = (T)v[0];
}

// ---- the table ---------------------------------------------------------------
enum MmForm { FORM_NT = 0, FORM_NN, FORM_TN, FORM_NN_SUM, FORM_GATE, FORM_DH, FORM_STATS, FORM_DZ, FORM_COUNT, FORM_STATS_KEEP /* sized as FORM_STATS */ };
enum MmSize { SIZE_256 = 0, SIZE_128, SIZE_64, SIZE_128_DEEP, SIZE_COUNT };
struct MmKernel {
    const void *fn, *join;
    int bm, bn, threads;  // rows and columns of C a workgroup takes
    int slots, slice, tile_kb;
};
template <class G>
MmKernel mm_entry(const void* fn, const void* join = nullptr) {
    return MmKernel{fn, join, G::BM, G::TILE_N, G::NT, G::SLOTS, G::SLICE_NS, G::TILE_KB};
}

// The tiles.  256 x 256: eight waves of 64 x 128 (four of 128 x 128: 4096^3 alike,
// 110 us, but 4096x11008x4096 ended by the softmax's pieces 313 us against 294,
// where a lone wave a SIMD does the end's arithmetic by itself; the end that loads
// values for each result and makes the activation is better off with four, 378 us
// against 394 with two loads, 419 in a later run with the three of Kept24).  128 x
// 128 twice a compute unit, four waves and two slots each; 64 x 128 likewise with
// three slots, for few rows.  128 x 128 once a unit, eight waves and four slots,
// where there are no more workgroups than units (2048x2048x5440 46 us, twice a unit
// 56; four waves 48).
template <class Tr, int LA, int LB, bool PAIR>
struct MmTiles {
    typedef MmTile<Tr, LA, LB, 256, 256, 4, 2, 2, false, PAIR> T256;
    typedef MmTile<Tr, LA, LB, 256, 256, 2, 2, 2, false, PAIR> T256Loads;
    typedef MmTile<Tr, LA, LB, 128, 128, 2, 2, 2, false, PAIR> T128;
    typedef MmTile<Tr, LA, LB, 64, 128, 2, 2, 3, true, PAIR> T64;
    typedef MmTile<Tr, LA, LB, 128, 128, 4, 2, 4, true, PAIR> T128Deep;
};

}  // namespace tg
