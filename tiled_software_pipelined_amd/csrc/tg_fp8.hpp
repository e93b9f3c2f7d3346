// Block-scaled 8-bit products: kernels, and the table that the host picks
// from.  C = sum over 128-blocks kb of 2^(sa + sb) * (A_kb B_kb^T), C bfloat16.
#pragma once

#include "tg_nt.hpp"

namespace tg {

struct Fp8Args {
    NtOperands op;
    uint16_t* C;             // element (m, n) at C[m row + n col]; tiled kernels: col = 1
    int64_t row, col;
    int32_t tiles_m, tiles_n;
    int32_t stream;  // 1: C's rows are whole cache lines, written past the L2
};

typedef void (*Fp8Fn)(Fp8Args);

// One compiled kernel.  bm, bn: rows and columns of C per workgroup.  bytes:
// for operands with rows that do not start on 4-byte boundaries.
struct Fp8Kernel {
    Fp8Fn fn, bytes;
    int bm, bn, threads;
    char name[64];
};

// Tiles, from the largest; and the kernels for few rows of A.
enum Fp8Pick { PICK_256 = 0, PICK_128, PICK_128_PAIR, PICK_64, PICK_ROWS16, PICK_ROWS32, PICK_COUNT };

const Fp8Kernel* fp8_kernels_e4m3_e4m3();
const Fp8Kernel* fp8_kernels_e4m3_e5m2();
const Fp8Kernel* fp8_kernels_e5m2_e4m3();
const Fp8Kernel* fp8_kernels_e5m2_e5m2();

// bfloat16 bits, to nearest even: the one rounding of a result
__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

// N results past the L2: C is not read here, and the launch ends sooner than
// with 32 MB of it to be written back at its end (e4m3 4096^3 57 -> 53 us).
template <int N>
__device__ __forceinline__ void store_stream(uint16_t* dst, const uint16_t (&v)[N]) {
    typedef uint32_t Words __attribute__((ext_vector_type(N >= 2 ? N / 2 : 1)));
    Words w;
    __builtin_memcpy(&w, v, sizeof v);
    __builtin_nontemporal_store(w, reinterpret_cast<Words*>(dst));
}

// Tiled kernel.
template <class G>
__device__ __forceinline__ void fp8_tile(const Fp8Args& g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const int lane = lane_id(), wave = wave_id();
    constexpr int WAVES_N = G::BN / G::WTN;
    int tm, tn;
    grouped_tile(xcd_rank(blockIdx.x, gridDim.x), g.tiles_m, g.tiles_n, 4, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int wm0 = (wave / WAVES_N) * G::WTM, wn0 = (wave % WAVES_N) * G::WTN;
    typename G::Acc acc[G::FM][G::FN];
    G::product(g.op, m0, n0, (TG_LDS char*)smem_raw, acc, wm0, wn0, lane, wave);

    // a lane's FN results of one row are adjacent: one store, of any alignment.
    // Which lanes have them inside the row is decided once, not for each row
    // (a branch a store took a wave of a column's last tile 14 us longer:
    // 5632x5696x128 34 us, now 19.7); then element stores where the row
    // ends inside a lane's results.
    const int n = n0 + wn0 + G::col_of(0, lane), m1 = m0 + wm0;
    auto each = [&](auto store) {
#pragma unroll
        for (int i = 0; i < G::FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int m = m1 + G::row_of(i, r, lane);
                uint16_t v[G::FN];
#pragma unroll
                for (int j = 0; j < G::FN; ++j) v[j] = bf16_bits(acc[i][j][r]);
                if (m < g.op.M) store(g.C + (int64_t)m * g.row + n, v);
            }
    };
    typedef const uint16_t (&Values)[G::FN];
    if (n + G::FN <= g.op.N) {
        if (G::FN >= 2 && g.stream) each([](uint16_t* dst, Values v) { store_stream(dst, v); });
        else each([](uint16_t* dst, Values v) { __builtin_memcpy(dst, v, sizeof v); });
    } else if (n < g.op.N) {
        each([&](uint16_t* dst, Values v) {
#pragma unroll
            for (int j = 0; j < G::FN - 1; ++j)
                if (n + j < g.op.N) dst[j] = v[j];
        });
    }
}

template <class G>
__global__ __launch_bounds__(G::NT) void fp8_tile_kernel(Fp8Args g) {
    fp8_tile<G>(g);
}

// Few rows of A (a decode batch; or, with the operands and C's strides
// swapped, few rows of B): bound by one read of B.  A workgroup takes
// 16 rows of B and 16 MT rows of A; its NW waves deal the 128-blocks of K
// among them, operands going straight to registers (a wave's blocks are its
// own: nothing to share through LDS), and add their sums through LDS at the
// end.  v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16, chunks
// l / 16 and 4 + l / 16 of the block's eight 16-byte chunks, so one load
// instruction reads 64 adjacent bytes of each of 16 rows.  BYTES: rows may
// start at any byte.  Loads that are not 4-byte aligned take three times as
// long (20x64x6681 19.4 us, with rows 6684 apart 7.5), so a chunk is then the
// four words it starts in and the word behind them, shifted together.
template <int FA, int FB, int MT, int NW, int U, bool BYTES>
__global__ __launch_bounds__(64 * NW) void fp8_rows_kernel(Fp8Args g) {
    __shared__ float part[NW][MT * 256];
    const NtOperands& o = g.op;
    const int lane = lane_id(), wave = wave_id();
    const int tn = blockIdx.x % g.tiles_n, tm = blockIdx.x / g.tiles_n;
    const int m0 = tm * 16 * MT, n0 = tn * 16;
    const int blocks = (o.k + 127) / 128;
    const int at = (lane >> 4) * 16;
    const int nb = min(n0 + (lane & 15), o.N - 1);
    const char* brow = o.b + (int64_t)nb * o.ldb + at;
    const uint8_t* bs = o.sb + nb;
    const char* arow[MT];
    const uint8_t* as[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int ma = min(m0 + 16 * t + (lane & 15), o.M - 1);
        arow[t] = o.a + (int64_t)ma * o.lda + at;
        as[t] = o.sa + ma;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};

    // bytes past a 4-byte boundary at which a row starts
    const int off_b = BYTES ? (int)((uintptr_t)brow & 3) : 0;
    int off_a[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) off_a[t] = BYTES ? (int)((uintptr_t)arow[t] & 3) : 0;
    struct Chunk {
        i32x4 v;
        uint32_t next;  // BYTES: the word behind
    };
    struct Block {
        Chunk b[2], a[MT][2];
        int sb, sa[MT];
        bool whole;
    };
    auto load_chunk = [&](Chunk& x, const char* p, int off) {
        x.v = load16(__builtin_assume_aligned(p - off, 4));
        // a chunk on a boundary has no part in the word behind, which may be
        // past the operand's end
        if constexpr (BYTES) x.next = *reinterpret_cast<const uint32_t*>(p - off + (off ? 16 : 12));
    };
    auto chunk = [&](const Chunk& x, int off) {
        if constexpr (!BYTES) return x.v;
        return i32x4{(int)__builtin_amdgcn_alignbyte(x.v[1], x.v[0], off), (int)__builtin_amdgcn_alignbyte(x.v[2], x.v[1], off),
                     (int)__builtin_amdgcn_alignbyte(x.v[3], x.v[2], off), (int)__builtin_amdgcn_alignbyte(x.next, x.v[3], off)};
    };
    auto load = [&](Block& x, int kb) {
        const int64_t k0 = (int64_t)kb * 128;
        x.whole = k0 + 128 <= o.k;  // wave-uniform
        if (x.whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                load_chunk(x.b[h], brow + k0 + 64 * h, off_b);
#pragma unroll
                for (int t = 0; t < MT; ++t) load_chunk(x.a[t][h], arow[t] + k0 + 64 * h, off_a[t]);
            }
        } else {
            // the last, partial block: zero past the row's end
            const int p = (int)k0 + at;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x.b[h] = Chunk{row_end_chunk(brow - at, p + 64 * h, o.k), 0};
#pragma unroll
                for (int t = 0; t < MT; ++t) x.a[t][h] = Chunk{row_end_chunk(arow[t] - at, p + 64 * h, o.k), 0};
            }
        }
        x.sb = bs[(int64_t)kb * o.ldsb];
#pragma unroll
        for (int t = 0; t < MT; ++t) x.sa[t] = as[t][(int64_t)kb * o.ldsa];
    };
    auto multiply = [&](const Block& x) {
        const int ob = x.whole ? off_b : 0;
        const i32x8 vb = __builtin_shufflevector(chunk(x.b[0], ob), chunk(x.b[1], ob), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int oa = x.whole ? off_a[t] : 0;
            const i32x8 va = __builtin_shufflevector(chunk(x.a[t][0], oa), chunk(x.a[t][1], oa), 0, 1, 2, 3, 4, 5, 6, 7);
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc[t], FA, FB, 0, x.sa[t], 0, x.sb);
        }
    };
    // U blocks in flight per wave; whole rounds first, then one at a time
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
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][t * 256 + (4 * (lane >> 4) + r) * 16 + (lane & 15)] = acc[t][r];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * 256; e += 64 * NW) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += part[w][e];
        const int m = m0 + (e >> 4), n = n0 + (e & 15);
        if (m < o.M && n < o.N) g.C[(int64_t)m * g.row + (int64_t)n * g.col] = bf16_bits(sum);
    }
}

// The kernels of one pair of formats, in the order of Fp8Pick.
template <int FA, int FB>
const Fp8Kernel* fp8_kernel_table() {
    typedef NtF8<FA, FB> Tr;
    // 256 x 256: four waves of 128 x 128, one a SIMD.  Against eight of 128 x
    // 64 they read a third less from LDS for the same matrix instructions,
    // which leaves the power budget a higher clock (e4m3 8192^3 354 us against
    // 366, 4096^3 both 52.5).  Of the cycles that a longer K adds (4096 x 4096, K
    // from 4096 to 32768) the matrix cores are busy 85 %.
    typedef NtGemm<Tr, 256, 256, 2, 2, 2, false> G256;
    // 128 x 128 with a compute unit to itself: eight waves, four slots (four
    // waves: 1024x4096x4096 24.5 us against 22.7).  Where there are several
    // rounds: two slots, two workgroups a unit (2048x4096x4096 42 us -> 34.5).
    typedef NtGemm<Tr, 128, 128, 2, 4, 4, true> G128;
    typedef NtGemm<Tr, 128, 128, 2, 2, 2, true> G128P;
    // 64 x 64: four slots, two workgroups a unit (eight and one: as fast
    // alone, 512x4096x4096 19.9 us against 16.5).
    typedef NtGemm<Tr, 64, 64, 2, 2, 4, true> G64;
    static const Fp8Kernel table[PICK_COUNT] = {
        {fp8_tile_kernel<G256>, fp8_tile_kernel<G256>, G256::BM, G256::BN, G256::NT, "t256x256x128_w2x2_s2"},
        {fp8_tile_kernel<G128>, fp8_tile_kernel<G128>, G128::BM, G128::BN, G128::NT, "t128x128x128_w2x4_s4_slice"},
        {fp8_tile_kernel<G128P>, fp8_tile_kernel<G128P>, G128P::BM, G128P::BN, G128P::NT, "t128x128x128_w2x2_s2_slice"},
        {fp8_tile_kernel<G64>, fp8_tile_kernel<G64>, G64::BM, G64::BN, G64::NT, "t64x64x128_w2x2_s4_slice"},
        {fp8_rows_kernel<FA, FB, 1, 8, 4, false>, fp8_rows_kernel<FA, FB, 1, 8, 4, true>, 16, 16, 512, "rows16_w8"},
        {fp8_rows_kernel<FA, FB, 2, 8, 4, false>, fp8_rows_kernel<FA, FB, 2, 8, 4, true>, 32, 16, 512, "rows32_w8"},
    };
    return table;
}

}  // namespace tg
