// Softmax cross entropy of a linear layer's logits z = x W^T, without a tensor of
// them: loss = log sum exp z - z[target].
//
// Rows that do not count (a prompt's tokens, padding) are left out of every
// product: the rows of x that count are gathered (and stand on 128-byte lines
// then), their number stays on the device, and workgroups past it end at once.
//
// Forward: the product's kernel ends with the maximum and the sum of powers of
// each wave's 64 or 128 columns; a second one joins them to the row's maximum, the
// logarithm of its sum above that, and the row's loss.  The two stay apart: in
// their sum, of which float holds 24 bits, a likely target's loss and its p - 1
// would lose what the logits' size takes (a loss of 1.6e-3 was 2.0e-3 at logits of
// 16384, and 0 at 65536).  Backward: pieces of the vocabulary, for each the
// product again, ended by dz = coef (p - [target]), p = exp(z - max) / sum, and the
// two products that take it, dx += dz W and dW = dz^T x.
//
// With TGEMM_KEEP_POWERS the forward pass also stores each power in 16 bits (2 V
// bytes written for a row that counts, and room for every row: only the device
// knows how many count), and dz is a pass over them: 6 M V K operations for the
// step, not 8 (8192x4096x128256, 90 % of the rows counting, 25.0 ms -> 19.4).
#include <climits>

#include "tg_mm_host.hpp"

namespace tg {

// Elements of dz that are held at once: 512 MB.  Fewer and larger pieces read and
// write dx's float sums less often.
constexpr int64_t XENT_PIECE = INT64_C(1) << 28;

struct XentLayout {
    MmSize stats, dz, dx, dw;
    int64_t parts;             // pieces of a row that the forward pass joins
    int64_t ldx;               // row stride of the gathered rows of x
    int64_t cols, ldz;         // backward: columns of a piece, row stride of dz
    int64_t count, map, rank, lse;                  // kept
    int64_t powers, ldp;                            // kept as well, or -1; then so are hit and part
    int64_t x, hit, each, part;                     // forward's scratch
    int64_t x2, coef, alpha, row_alpha, back, dzs, sum, split, w2;  // backward's; w2: w on lines, -1: read where it is
    int64_t split_bytes[2];                         // of dx's and dw's launches, which use the same room
    int64_t bytes[3];
};

static_assert(XENT_PIECE / 64 <= MM_MOST, "row stride of dz");
// A row of powers: a lane's place in eight rows is a 32-bit offset.
constexpr int64_t MOST_POWERS = INT64_C(1) << 28;

static int wave_cols(MmSize s) { return s == SIZE_256 ? 128 : 64; }

static XentLayout xent_layout(int64_t M, int64_t V, int64_t K, int keep) {
    XentLayout l{};
    auto take = [&](int which, int64_t n) {
        const int64_t at = l.bytes[which];
        l.bytes[which] += (n + 255) / 256 * 256;
        return at;
    };
    l.count = take(0, 4);  // how many rows count
    l.map = take(0, 4 * M);   // where they stand
    l.rank = take(0, 4 * M);  // each row's number among them, -1
    l.lse = take(0, 8 * M);   // of each of them
    l.ldx = mm_lines(K);
    l.w2 = -1;
    l.stats = mm_size(FORM_STATS, M, V, mm_slices(K), false, K);
    l.parts = (V + wave_cols(l.stats) - 1) / wave_cols(l.stats);
    const bool powers = keep & TGEMM_KEEP_POWERS;
    l.x = take(1, 2 * M * l.ldx);
    l.hit = take(!powers, 4 * M);  // the target's logit of each of them
    l.each = take(1, 4 * M);       // each row's loss
    l.part = take(!powers, 8 * M * l.parts);
    l.ldp = mm_lines(V);
    l.powers = powers ? take(0, 2 * M * l.ldp) : -1;
    if (!(keep & (TGEMM_KEEP_X | TGEMM_KEEP_W))) return l;
    const int64_t padded = (M + 63) / 64 * 64;  // rows, the last of them zero
    // at least 8192 columns: dz is then four times as wide as x often is; at most
    // 2^22, as XENT_PIECE has them for 64 rows: the products' copies reach 64 rows
    // by 32-bit offsets
    const int64_t fit = M > 0 ? XENT_PIECE / padded : V;
    const int64_t most = fit < 8192 ? 8192 : fit;
    const int64_t pieces = V > 0 ? (V + most - 1) / most : 1;
    l.cols = ((V + pieces - 1) / pieces + 255) / 256 * 256;
    if (l.cols < 256) l.cols = 256;  // of an empty vocabulary too: the walk over pieces ends
    l.ldz = l.cols;
    const int64_t cols = l.cols < V ? l.cols : V;
    const MmShape dx{M, K}, dw{cols, K};
    const bool pack = mm_packs(K, M) && cols <= MM_WAVE_ROWS;  // as far as a launch of a wave a row reaches
    l.dz = mm_size(FORM_DZ, M, cols, mm_slices(K), false, pack ? 0 : K);
    l.x2 = take(2, 2 * padded * l.ldx);
    l.coef = take(2, 4 * M);
    l.alpha = take(2, 4);
    l.row_alpha = take(2, 4 * M);
    l.back = take(2, 4 * M);
    l.dzs = take(2, 2 * padded * l.ldz);
    if (keep & TGEMM_KEEP_X) {
        // the sums over several pieces are not shared out as well
        l.dx = mm_size(pieces > 1 ? FORM_NN_SUM : FORM_NN, M, K, mm_slices(cols), pieces == 1, 0);
        if (pieces > 1) l.sum = take(2, 4 * M * K);
        else l.split_bytes[0] = mm_split_bytes(FORM_NN, l.dx, &dx, 1, mm_slices(cols), true);
    }
    if (keep & TGEMM_KEEP_W) {
        l.dw = mm_size(FORM_TN, cols, K, mm_slices(M), true, 0);
        l.split_bytes[1] = mm_split_bytes(FORM_TN, l.dw, &dw, 1, mm_slices(M), true);
    }
    if (pack) l.w2 = take(2, 2 * cols * l.ldx);
    l.split = take(2, l.split_bytes[0] > l.split_bytes[1] ? l.split_bytes[0] : l.split_bytes[1]);
    return l;
}

static bool xent_sizes_ok(int64_t M, int64_t V, int64_t K, int32_t keep) {
    if (M < 0 || V < 0 || K < 0 || M > MM_WAVE_ROWS || V > MM_MOST_ROWS || K > MM_MOST ||
        (keep & ~(TGEMM_KEEP_X | TGEMM_KEEP_W | TGEMM_KEEP_POWERS)) || ((keep & TGEMM_KEEP_POWERS) && V > MOST_POWERS)) {
        set_error("M=%lld V=%lld K=%lld keep=%d out of range", (long long)M, (long long)V, (long long)K, keep);
        return false;
    }
    return true;
}

// Workgroups of a row in the pass over the powers.
static int64_t powers_chunks(const XentLayout& l) { return (l.ldz + 16 * wave_cols(l.stats) - 1) / (16 * wave_cols(l.stats)); }
// Whether grids hold the launches of the backward pass.
static int xent_check_grids(const XentLayout& l, int64_t M, int64_t V, int64_t K, int keep) {
    int rc = TGEMM_OK;
    if (!(keep & (TGEMM_KEEP_X | TGEMM_KEEP_W))) return rc;
    const int64_t cols = l.cols < V ? l.cols : V;
    rc = l.powers >= 0 ? mm_check_grid("gradient of the logits", (double)powers_chunks(l) * (double)((M + 63) / 64 * 4), 256)
                       : mm_check_tiles("gradient of the logits", FORM_DZ, l.dz, M, cols);
    // scales of the rows: no more workgroups than 16 rows and 1024 columns make
    if (rc == TGEMM_OK) rc = mm_check_grid("gradient of the logits", (double)((cols + 1023) / 1024) * (double)((M + 15) / 16), 256);
    if (rc == TGEMM_OK && (keep & TGEMM_KEEP_X)) {
        rc = mm_check_tiles("gradient of x", l.cols < V ? FORM_NN_SUM : FORM_NN, l.dx, M, K);
        if (rc == TGEMM_OK && l.cols < V) rc = mm_check_grid("gradient of x", (double)M * (double)((K + 3) / 4) / 256 + 1, 256);
    }
    if (rc == TGEMM_OK && (keep & TGEMM_KEEP_W)) rc = mm_check_tiles("gradient of w", FORM_TN, l.dw, cols, K);
    return rc;
}

static int xent_common(int32_t dtype, int32_t reduction, const void* target, int64_t M) {
    if (dtype != TGEMM_BF16 && dtype != TGEMM_F16) {
        set_error("dtype %d is not bfloat16 or float16", dtype);
        return TGEMM_E_ARG;
    }
    if (reduction < TGEMM_NONE || reduction > TGEMM_MEAN) {
        set_error("unknown reduction %d", reduction);
        return TGEMM_E_ARG;
    }
    if (M > 0 && !target) {
        set_error("target: NULL pointer");
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)target % 8) {
        set_error("target: not aligned to its element size");
        return TGEMM_E_ALIGN;
    }
    return TGEMM_OK;
}
static int check_floats(const char* name, const void* p, int64_t count) {
    if (count > 0 && !p) {
        set_error("%s: NULL pointer", name);
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)p % 4) {
        set_error("%s: not aligned to its element size", name);
        return TGEMM_E_ALIGN;
    }
    return TGEMM_OK;
}

// ---- the rows that count -------------------------------------------------------
struct ScanArgs {
    int64_t M, ignore;
    const int64_t* target;
    int32_t *count, *map, *rank;
};

// One workgroup: each wave takes a run of rows, counts its own, and after the
// waves' counts are added gives them their numbers.
__global__ __launch_bounds__(1024) void xent_scan_kernel(ScanArgs g) {
    __shared__ int held[16];
    const int lane = lane_id(), wave = wave_id();
    const int64_t run = ((g.M + 15) / 16 + 63) / 64 * 64, begin = run * wave, end = min(begin + run, g.M);
    int n = 0;
    for (int64_t m = begin + lane; m < end; m += 64) n += g.target[m] != g.ignore;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    if (lane == 0) held[wave] = n;
    __syncthreads();
    int at = 0, total = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < wave) at += held[w];
        total += held[w];
    }
    if (threadIdx.x == 0) *g.count = total;
    for (int64_t m0 = begin; m0 < end; m0 += 64) {
        const int64_t m = m0 + lane;
        const bool counts = m < end && g.target[m] != g.ignore;
        const uint64_t mask = __ballot(counts);
        const int mine = at + __popcll(mask & ((uint64_t(1) << lane) - 1));
        if (m < end) g.rank[m] = counts ? mine : -1;
        if (counts) g.map[mine] = (int32_t)m;
        at += __popcll(mask);
    }
}

struct GatherArgs {
    int64_t M, K, ldx, ldto, lddx;
    const uint16_t* x;
    uint16_t* to;
    float* loss;   // not NULL: zero for rows that do not count
    uint16_t* dx;  // likewise
    const int32_t *count, *rank;
};

// A row by a wave: gathered, or zeros for a row that does not count.
__device__ __forceinline__ void gather_row(const GatherArgs& g, int64_t m, int r, int lane) {
    const i32x4 zero{0, 0, 0, 0};
    if (r < 0) {
        if (g.loss && lane == 0) g.loss[m] = 0.0f;
        if (g.dx) {
            uint16_t* dst = g.dx + m * g.lddx;
            for (int64_t k = 8 * lane; k < g.K; k += 512) {
                if (k + 8 <= g.K) __builtin_memcpy(dst + k, &zero, 16);
                else
                    for (int64_t e = k; e < g.K; ++e) dst[e] = 0;
            }
        }
        return;
    }
    const uint16_t* src = g.x + m * g.ldx;
    uint16_t* dst = g.to + r * g.ldto;  // rows of whole lines
    for (int64_t k = 8 * lane; k < g.K; k += 512) {
        i32x4 v;
        if (k + 8 <= g.K) {
            v = load16(src + k);
        } else {
            union { i32x4 v; uint16_t e[8]; } u;
#pragma unroll
            for (int e = 0; e < 8; ++e) u.e[e] = load_or_zero(src + k + e, k + e < g.K);
            v = u.v;
        }
        *reinterpret_cast<i32x4*>(dst + k) = v;
    }
}
__global__ __launch_bounds__(256) void xent_gather_kernel(GatherArgs g) {
    const int64_t m = (int64_t)blockIdx.x * 4 + wave_id();
    if (m < g.M) gather_row(g, m, g.rank[m], lane_id());
}

// Both at once for up to SCAN_ROWS rows: each workgroup counts the rows before its
// own four by itself (a launch less: 4 us; all workgroups together read M^2 / 8
// targets, which 4096 rows keep under 2 us).
constexpr int64_t SCAN_ROWS = 4096;
__global__ __launch_bounds__(256) void xent_scan_gather_kernel(ScanArgs s, GatherArgs g) {
    __shared__ int held[4];
    const int lane = lane_id(), wave = wave_id();
    const int64_t m0 = (int64_t)blockIdx.x * 4, m = m0 + wave;
    int n = 0;
    for (int64_t i = threadIdx.x; i < m0; i += 256) n += s.target[i] != s.ignore;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    if (lane == 0) held[wave] = n;
    __syncthreads();
    n = held[0] + held[1] + held[2] + held[3];
    int before = 0;
    for (int i = 0; i < 4; ++i) {
        const bool counts = m0 + i < s.M && s.target[m0 + i] != s.ignore;
        if (i < wave) before += counts;
        if (i == wave && m < s.M) {
            const int r = counts ? n + before : -1;
            if (lane == 0) {
                s.rank[m] = r;
                if (counts) s.map[r] = (int32_t)m;
                if (m == s.M - 1) *s.count = n + before + counts;
            }
            gather_row(g, m, r, lane);
        }
    }
}

// ---- the loss ------------------------------------------------------------------
struct RowsArgs {
    int64_t M, V, parts;
    const int32_t *count, *map;
    const int64_t* target;
    const float2* part;
    const float* hit;
    float2* lse;  // (max, log2 of the sum of 2^((z - max) log2 e)) of each row that counts
    float* loss;  // of each row
};

// 16 rows a workgroup, 32 threads a row.
__global__ __launch_bounds__(512) void xent_rows_kernel(RowsArgs g) {
    __shared__ float2 held[32][16];
    const int r = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int64_t m = (int64_t)blockIdx.x * 16 + r;
    const int M = *g.count;
    float most = -INFINITY, sum = 0.0f;
    auto join = [&](float2 p) {
        // NaN sums come through; pieces of nothing but -inf add nothing
        const float to = fmaxf(most, p.x), base = to == -INFINITY ? 0.0f : to;
        sum = sum * expf(most - base) + p.y * expf(p.x - base);
        most = to;
    };
    if (m < M) {
        int64_t p = y;
        for (; p + 96 < g.parts; p += 128) {
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = g.part[(p + 32 * u) * g.M + m];
#pragma unroll
            for (int u = 0; u < 4; ++u) join(v[u]);
        }
        for (; p < g.parts; p += 32) join(g.part[p * g.M + m]);
    }
    held[y][r] = float2{most, sum};
    __syncthreads();
    if (y != 0 || m >= M) return;
    for (int k = 1; k < 32; ++k) join(held[k][r]);
    g.lse[m] = float2{most, log2f(sum)};
    const int to = g.map[m];
    const int64_t t = g.target[to];
    // a target outside the vocabulary has no logit: its loss is NaN
    g.loss[to] = t >= 0 && t < g.V ? (most - g.hit[m]) + logf(sum) : NAN;
}

struct ReduceArgs {
    const int32_t *count, *map;
    const float* rows;
    float* loss;
    int32_t mean;
};

__global__ __launch_bounds__(1024) void xent_reduce_kernel(ReduceArgs g) {
    __shared__ double held[16];
    const int M = *g.count;
    double sum = 0.0;
    for (int m = threadIdx.x; m < M; m += 1024) sum += g.rows[g.map[m]];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) held[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) sum += held[w];
    *g.loss = (float)(g.mean ? sum / M : sum);
}

struct CoefArgs {
    int64_t V;
    const int32_t *count, *map;
    const int64_t* target;
    const float* dloss;
    float *coef, *alpha;
    float *row_alpha, *back;  // not NULL: rows have scales of their own
    int32_t reduction;
};

// The factor of each row's dz and the products' factor alpha.  Rows' factors are
// divided by the largest and taken times 2^14, which alpha takes out again: dz
// holds values from 2^14 down, where float16 keeps 11 bits to 2^-14
// (probabilities of 2^-28), whatever the loss was scaled by.  Where all rows have
// one factor, as the mean and the sum give them, it is thus exact: scaled by a
// power of two alone, an unlikely target's element is the factor itself, and its
// rounding, the same in every row, does not average out of dx and dw
// (8192x4096x128256: 3.5e-3 of their norm, now 1.8e-3).
//
// In float16 a row whose factor is 2^-25 of the largest would have no normal number
// left in dz, though its dx may hold it (reduction "none").  Where rows have scales
// of their own, each factor is brought to 2^13 .. 2^14 by a power of two more, 2^k;
// dx's product takes it out again, row_alpha = alpha 2^-k, and dz is multiplied by
// back = 2^-k before dw's, which adds rows up.
__device__ __forceinline__ void xent_factors(const CoefArgs& g) {
    __shared__ float held[16];
    const int M = *g.count;
    const float scalar = g.reduction == TGEMM_NONE ? 0.0f : g.reduction == TGEMM_MEAN ? *g.dloss / (float)M : *g.dloss;
    auto of = [&](int m) {
        const int to = g.map[m];
        const int64_t t = g.target[to];
        if (t < 0 || t >= g.V) return NAN;
        return g.reduction == TGEMM_NONE ? g.dloss[to] : scalar;
    };
    float most = 0.0f;  // of the finite ones
    for (int m = threadIdx.x; m < M; m += 1024) {
        const float a = fabsf(of(m));
        if (a < INFINITY) most = fmaxf(most, a);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
    if ((threadIdx.x & 63) == 0) held[threadIdx.x >> 6] = most;
    __syncthreads();
    for (int w = 0; w < 16; ++w) most = fmaxf(most, held[w]);
    if (most == 0.0f) most = 1.0f;
    const int low = ilogbf(most) + 100, e = low < 14 ? low : 14;  // alpha is a normal number
    int top;
    const float top_part = frexpf(most, &top);
    for (int m = threadIdx.x; m < M; m += 1024) {
        const float c = of(m);
        if (!g.row_alpha) {
            g.coef[m] = ldexpf(c / most, e);
            continue;
        }
        float r = c / most;
        int k = 0;
        if (c != 0.0f && fabsf(c) < INFINITY) {
            int at;
            r = frexpf(c, &at) / top_part;  // c / most = r 2^-k
            k = top - at;
            if (fabsf(r) > 1.0f) {
                r *= 0.5f;
                --k;
            }
        }
        g.coef[m] = ldexpf(r, e);
        g.row_alpha[m] = ldexpf(most, -e - k);
        g.back[m] = ldexpf(1.0f, -k);
    }
    if (threadIdx.x == 0) *g.alpha = ldexpf(most, -e);
}

// The first workgroup: the factors.  The others: rows of x, 16 each, and behind
// them the zero rows up to the next multiple of 64.
__global__ __launch_bounds__(1024) void xent_prepare_kernel(CoefArgs c, GatherArgs g) {
    if (blockIdx.x == 0) {
        xent_factors(c);
        return;
    }
    const int lane = lane_id();
    const int64_t m = ((int64_t)blockIdx.x - 1) * 16 + wave_id();
    if (m < g.M) {
        gather_row(g, m, g.rank[m], lane);
    } else {
        const int count = *g.count;
        const int64_t r = count + (m - g.M);
        if (r < (count + 63) / 64 * 64) {
            const i32x4 zero{0, 0, 0, 0};
            for (int64_t k = 8 * lane; k < g.ldto; k += 512) *reinterpret_cast<i32x4*>(g.to + r * g.ldto + k) = zero;
        }
    }
}

struct PowersArgs {
    int32_t V, n, wide, chunks;  // columns of this piece; columns that share a maximum; workgroups of a row
    int64_t M, v0, ldp, ldz;
    const int32_t *count, *map;
    const int64_t* target;
    const float2* part;
    const float *hit, *coef;
    const float2* lse;
    const uint16_t* powers;
    void* dz;
};

// dz of a piece of the vocabulary from the kept powers: one pass over them, bound by
// memory (3686 rows of 32000 in 86 us, 5.5 TB/s read and written).  A workgroup
// takes 16 rows and 16 maxima's columns (1024 or 2048): a thread makes the factor
// coef exp(max' - max) / sum of one row and maximum, then each wave walks four
// rows.  The target's element is coef (exp(z - max) / sum - 1) from its logit
// in float: near one, a rounded power would leave nothing of the difference.
// Zero in the rows up to the next multiple of 64.
template <class T>
__global__ __launch_bounds__(256) void xent_powers_kernel(PowersArgs g) {
    __shared__ float held[16][17];
    __shared__ float one[16];
    __shared__ int64_t aim[16];
    const int M = *g.count, group = (int)blockIdx.x / g.chunks, m0 = 16 * group, c0 = 16 * g.wide * ((int)blockIdx.x - group * g.chunks);
    if (m0 >= (M + 63) / 64 * 64) return;
    {
        const int r = threadIdx.x & 15, p = threadIdx.x >> 4, m = m0 + r;
        const int64_t v = g.v0 + c0 + p * g.wide;
        float f = 0.0f;
        if (m < M && v < g.V) f = Power<T>::BACK * g.coef[m] * softmax_of(g.part[v / g.wide * g.M + m].x, g.lse[m]);
        held[r][p] = f;
        if (p == 0) {
            aim[r] = m < M ? g.target[g.map[m]] - g.v0 : -1;
            one[r] = aim[r] >= 0 && aim[r] < g.n ? g.coef[m] * (softmax_of(g.hit[m], g.lse[m]) - 1.0f) : 0.0f;
        }
    }
    __syncthreads();
    const int c1 = min(c0 + 16 * g.wide, (int)g.ldz);
    for (int r = wave_id(); r < 16; r += 4) {
        const uint16_t* from = g.powers + (int64_t)(m0 + r) * g.ldp + g.v0;
        T* to = static_cast<T*>(g.dz) + (int64_t)(m0 + r) * g.ldz;
        const bool zero = m0 + r >= M;
        for (int c = c0 + 8 * lane_id(); c < c1; c += 512) {
            Raw8 raw{};
            if (!zero && g.v0 + c < g.ldp) load8(raw, from + c);
            float v[8];
            const float f = zero ? 0.0f : held[r][(c - c0) / g.wide];
            const int64_t t = aim[r] - c;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t two = (uint32_t)raw.v[e >> 1];
                v[e] = zero ? 0.0f : e == t ? one[r] : power_of<T>(e & 1 ? two >> 16 : two) * f;
            }
            store8(to + c, v);
        }
    }
}

struct BackArgs {
    int32_t n, chunks;  // columns; workgroups of 16 rows
    int64_t ldz;
    const int32_t* count;
    const float* back;
    void* dz;
};

// dz from the rows' own scales to the common one, where they differ: 16 rows and
// 2048 columns a workgroup.
template <class T>
__global__ __launch_bounds__(256) void xent_back_kernel(BackArgs g) {
    const int M = *g.count, group = (int)blockIdx.x / g.chunks, c0 = 2048 * ((int)blockIdx.x - group * g.chunks), c1 = min(c0 + 2048, g.n);
    for (int r = wave_id(); r < 16; r += 4) {
        const int m = 16 * group + r;
        if (m >= M) return;
        const float f = g.back[m];
        if (f == 1.0f) continue;
        T* row = static_cast<T*>(g.dz) + (int64_t)m * g.ldz;  // whole up to its stride
        for (int c = c0 + 8 * lane_id(); c < c1; c += 512) {
            Raw8 raw;
            load8<T>(raw, row + c);
            float v[8];
            values8<T>(v, raw);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= f;
            store8(row + c, v);
        }
    }
}

}  // namespace tg

extern "C" {

int tgemm_xent_bytes(int64_t M, int64_t V, int64_t K, int32_t keep, int64_t* bytes) {
    using namespace tg;
    if (!bytes) {
        set_error("NULL bytes");
        return TGEMM_E_NULL;
    }
    if (!xent_sizes_ok(M, V, K, keep)) return TGEMM_E_ARG;
    const XentLayout l = xent_layout(M, V, K, keep);
    for (int i = 0; i < 3; ++i) bytes[i] = l.bytes[i];
    clear_error();
    return TGEMM_OK;
}

int tgemm_xent_forward(int64_t M, int64_t V, int64_t K, int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                       const int64_t* target, int64_t ignore, int32_t reduction, int32_t keep, float* loss, void* saved,
                       void* scratch, void* stream) {
    using namespace tg;
    if (!xent_sizes_ok(M, V, K, keep)) return TGEMM_E_ARG;
    const XentLayout l = xent_layout(M, V, K, keep & TGEMM_KEEP_POWERS);
    int rc = xent_common(dtype, reduction, target, M);
    if (rc == TGEMM_OK) rc = mm_check("x", x, M, K, ldx);
    if (rc == TGEMM_OK) rc = mm_check("w", w, V, K, ldw);
    if (rc == TGEMM_OK) rc = check_floats("loss", loss, reduction == TGEMM_NONE ? M : 1);
    if (rc == TGEMM_OK) rc = mm_check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = mm_check_buffer("scratch", scratch, l.bytes[1]);
    if (rc == TGEMM_OK && M > 0 && V > 0) rc = mm_check_tiles("logits", FORM_STATS, l.stats, M, V);
    if (rc == TGEMM_OK) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *v = static_cast<char*>(saved), *s = static_cast<char*>(scratch);
    int32_t *count = reinterpret_cast<int32_t*>(v + l.count), *map = reinterpret_cast<int32_t*>(v + l.map),
            *rank = reinterpret_cast<int32_t*>(v + l.rank);
    char* where = l.powers >= 0 ? v : s;
    float* hit = reinterpret_cast<float*>(where + l.hit);
    float2 *lse = reinterpret_cast<float2*>(v + l.lse), *part = reinterpret_cast<float2*>(where + l.part);
    float* each = reduction == TGEMM_NONE ? loss : reinterpret_cast<float*>(s + l.each);
    ScanArgs c{M, ignore, target, count, map, rank};
    GatherArgs into{M, K, ldx, l.ldx, 0, static_cast<const uint16_t*>(x), reinterpret_cast<uint16_t*>(s + l.x),
                    reduction == TGEMM_NONE ? loss : nullptr, nullptr, count, rank};
    if (M > 0 && M <= SCAN_ROWS) {
        void* both[] = {&c, &into};
        rc = mm_launch_list(reinterpret_cast<const void*>(xent_scan_gather_kernel), (M + 3) / 4, 256, both, "rows that count", st);
    } else {
        rc = mm_launch(reinterpret_cast<const void*>(xent_scan_kernel), 1, 1024, &c, "rows that count", st);
        if (rc == TGEMM_OK && M > 0)
            rc = mm_launch(reinterpret_cast<const void*>(xent_gather_kernel), (M + 3) / 4, 256, &into, "rows that count", st);
    }
    if (rc == TGEMM_OK && M > 0 && V > 0) {
        const MmKernel& k = mm_kernels(dtype, l.powers >= 0 ? FORM_STATS_KEEP : FORM_STATS)[l.stats];
        MmStatsArgs a{MmOperands{s + l.x, static_cast<const char*>(w), nullptr, 2 * l.ldx, 2 * ldw, 0, (int32_t)M, (int32_t)V,
                                 (int32_t)K},
                      mm_grid(k, M, V), count, map, target, part, hit,
                      l.powers >= 0 ? reinterpret_cast<uint16_t*>(v + l.powers) : nullptr, l.ldp};
        rc = mm_launch(k.fn, (int64_t)a.grid.tiles_m * a.grid.tiles_n, k.threads, &a, "logits", st);
    }
    if (rc == TGEMM_OK && M > 0) {
        RowsArgs a{M, V, V > 0 ? l.parts : 0, count, map, target, part, hit, lse, each};
        rc = mm_launch(reinterpret_cast<const void*>(xent_rows_kernel), (M + 15) / 16, 512, &a, "rows of the loss", st);
    }
    if (rc == TGEMM_OK && reduction != TGEMM_NONE) {
        ReduceArgs a{count, map, each, loss, reduction == TGEMM_MEAN};
        rc = mm_launch(reinterpret_cast<const void*>(xent_reduce_kernel), 1, 1024, &a, "sum of the loss", st);
    }
    if (rc == TGEMM_OK) clear_error();
    return rc;
}

int tgemm_xent_backward(int64_t M, int64_t V, int64_t K, int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                        const int64_t* target, int32_t reduction, const float* dloss, const void* saved, int32_t keep, void* dx,
                        int64_t lddx, void* dw, int64_t lddw, void* scratch, void* stream) {
    using namespace tg;
    if (!xent_sizes_ok(M, V, K, keep)) return TGEMM_E_ARG;
    const XentLayout l = xent_layout(M, V, K, keep);
    const bool kx = keep & TGEMM_KEEP_X, kw = keep & TGEMM_KEEP_W;
    int rc = xent_common(dtype, reduction, target, M);
    if (rc == TGEMM_OK) rc = mm_check("x", x, M, K, ldx);
    if (rc == TGEMM_OK) rc = mm_check("w", w, V, K, ldw);
    if (rc == TGEMM_OK && kx) rc = mm_check("dx", dx, M, K, lddx);
    if (rc == TGEMM_OK && kw) rc = mm_check("dw", dw, V, K, lddw);
    if (rc == TGEMM_OK) rc = check_floats("dloss", dloss, reduction == TGEMM_NONE ? M : 1);
    if (rc == TGEMM_OK) rc = mm_check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = mm_check_buffer("scratch", scratch, l.bytes[2]);
    if (rc == TGEMM_OK) rc = xent_check_grids(l, M, V, K, keep);
    if (rc == TGEMM_OK && (kx || kw) && (M > 0 || V > 0)) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    if (!kx && !kw) {
        clear_error();
        return TGEMM_OK;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const char* v = static_cast<const char*>(saved);
    char* s = static_cast<char*>(scratch);
    const int32_t *count = reinterpret_cast<const int32_t*>(v + l.count), *map = reinterpret_cast<const int32_t*>(v + l.map);
    float *coef = reinterpret_cast<float*>(s + l.coef), *alpha = reinterpret_cast<float*>(s + l.alpha);
    const char* wp = static_cast<const char*>(w);
    // rows' own scales: dx's alone, and needed where they differ and the type is short of range
    const bool own = kx && reduction == TGEMM_NONE && dtype == TGEMM_F16;
    float *row_alpha = own ? reinterpret_cast<float*>(s + l.row_alpha) : nullptr, *back = own ? reinterpret_cast<float*>(s + l.back) : nullptr;
    CoefArgs c{V, count, map, target, dloss, coef, alpha, row_alpha, back, reduction};
    GatherArgs into{M, K, ldx, l.ldx, lddx, static_cast<const uint16_t*>(x), reinterpret_cast<uint16_t*>(s + l.x2), nullptr,
                    kx ? static_cast<uint16_t*>(dx) : nullptr, count, reinterpret_cast<const int32_t*>(v + l.rank)};
    void* both[] = {&c, &into};
    rc = mm_launch_list(reinterpret_cast<const void*>(xent_prepare_kernel), 1 + (M + 63 + 15) / 16, 1024, both, "factors of the rows", st);
    const bool pieces = l.cols < V;
    MmStoreArgs into_x{}, into_w{};
    into_x.alpha = into_w.alpha = alpha;
    into_x.row_alpha = row_alpha;
    into_x.rows = into_w.rows = count;
    into_x.jobs = into_w.jobs = 1;
    into_x.map = map;
    into_w.rows_are_k = 1;
    if (l.split_bytes[0] > 0) into_x.split = reinterpret_cast<float*>(s + l.split);
    if (l.split_bytes[1] > 0) into_w.split = reinterpret_cast<float*>(s + l.split);
    // at least one round: without a vocabulary dx is zero
    for (int64_t v0 = 0; rc == TGEMM_OK && (v0 < V || v0 == 0); v0 += l.cols) {
        const int64_t n = V - v0 < l.cols ? V - v0 : l.cols;
        const char* wv = wp + v0 * ldw * 2;
        int64_t ldv = ldw;
        if (M > 0 && l.w2 >= 0 && (kx || l.powers < 0) && !mm_aligned(wv, ldw)) {
            const MmPack p{wv, ldw, n, K, s + l.w2};
            rc = mm_pack(&p, 1, st);
            wv = s + l.w2;
            ldv = l.ldx;
        }
        if (rc == TGEMM_OK && M > 0 && n > 0 && l.powers >= 0) {
            const int wide = wave_cols(l.stats);
            const int64_t chunks = powers_chunks(l);
            PowersArgs a{(int32_t)V, (int32_t)n, wide, (int32_t)chunks, M, v0, l.ldp, l.ldz, count, map, target,
                         reinterpret_cast<const float2*>(v + l.part), reinterpret_cast<const float*>(v + l.hit), coef,
                         reinterpret_cast<const float2*>(v + l.lse), reinterpret_cast<const uint16_t*>(v + l.powers), s + l.dzs};
            const void* fn = dtype == TGEMM_BF16 ? reinterpret_cast<const void*>(xent_powers_kernel<__bf16>)
                                                 : reinterpret_cast<const void*>(xent_powers_kernel<_Float16>);
            rc = mm_launch(fn, chunks * ((M + 63) / 64 * 4), 256, &a, "gradient of the logits", st);
        } else if (rc == TGEMM_OK && M > 0 && n > 0) {
            const MmKernel& k = mm_kernels(dtype, FORM_DZ)[l.dz];
            MmDzArgs a{MmOperands{s + l.x2, wv, nullptr, 2 * l.ldx, 2 * ldv, 0, (int32_t)M, (int32_t)n, (int32_t)K},
                       mm_grid(k, M, n), count, map, target, v0, reinterpret_cast<const float2*>(v + l.lse), coef, s + l.dzs,
                       l.ldz};
            rc = mm_launch(k.fn, (int64_t)a.grid.tiles_m * a.grid.tiles_n, k.threads, &a, "gradient of the logits", st);
        }
        if (rc == TGEMM_OK && kx) {
            into_x.job[0] = MmJob{{MmOperands{s + l.dzs, wv, nullptr, 2 * l.ldz, 2 * ldv, 0, (int32_t)M, (int32_t)K, (int32_t)n, 1,
                                              wv == s + l.w2}, {}},
                                  1, {}, dx, lddx, pieces ? reinterpret_cast<float*>(s + l.sum) : nullptr, v0 > 0};
            rc = mm_store(dtype, pieces ? FORM_NN_SUM : FORM_NN, l.dx, into_x, st);
        }
        if (rc == TGEMM_OK && kw && own && M > 0 && n > 0) {
            const int64_t chunks = (n + 2047) / 2048;
            BackArgs a{(int32_t)n, (int32_t)chunks, l.ldz, count, back, s + l.dzs};
            rc = mm_launch(reinterpret_cast<const void*>(xent_back_kernel<_Float16>), chunks * ((M + 15) / 16), 256, &a, "scales of the rows", st);
        }
        if (rc == TGEMM_OK && kw && n > 0) {
            into_w.job[0] = MmJob{{MmOperands{s + l.dzs, s + l.x2, nullptr, 2 * l.ldz, 2 * l.ldx, 0, (int32_t)n, (int32_t)K,
                                              (int32_t)((M + 63) / 64 * 64), 1, 1}, {}},
                                  1, {}, static_cast<char*>(dw) + v0 * lddw * 2, lddw, nullptr, 0};
            rc = mm_store(dtype, FORM_TN, l.dw, into_w, st);
        }
    }
    if (rc == TGEMM_OK && kx && pieces) rc = mm_round(dtype, into_x, st);
    if (rc == TGEMM_OK) clear_error();
    return rc;
}

}  // extern "C"
