// Products of 16-bit operands (bfloat16 or float16, float sums) whose results
// go through a fused end: the tile kernel's template.
//
// C (M x N) = sum over k of a(m, k) b(n, k).  Each operand stands either
// ALONG k (element (r, k) at r ld + k) or ACROSS it (at k ld + r), so that a
// layer's forward product and both of its backward ones read the tensors as
// they are.  A workgroup computes one BM x BN tile; its waves form a WAVES_M x
// WAVES_N grid of WTM x WTN blocks of 32 x 32 matrix-core tiles.  The K loop
// walks slices of 64 k through a ring of STAGES LDS slots that direct global ->
// LDS copies fill, one barrier a slice.
//
// In LDS an operand ALONG k has rows of 128 bytes (the slice's k of one r), read
// 16 bytes at a time; one ACROSS k has a row for each k, of all the tile's r,
// read by the transposing read (ds_read_b64_tr_b16: in a group of 16 lanes,
// lane j points at 4 adjacent r of row j / 4 and gets 4 adjacent k of r number
// j).  16-byte chunks are permuted inside their rows so that neither read has
// bank conflicts.
//
// The matrix instruction takes b's fragment first, so that a lane's results are
// of one row m: registers 4 g .. 4 g + 3 of a 32 x 32 tile hold columns 8 g + 4
// (lane / 32) .. + 3 of row lane % 32.  Sums over a row stay inside a lane, and
// a wave turns its block into rows for wide stores through its own part of
// the LDS, without a barrier (each_row).
#pragma once

#include "tg_nt.hpp"

namespace tg {

enum MmLay { ALONG = 0, ACROSS = 1 };

struct MmBf16 {
    typedef __bf16 T;
    __device__ static __forceinline__ f32x16 mma(i32x4 x, i32x4 y, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    }
    __device__ static __forceinline__ f32x4 mma16(i32x4 x, i32x4 y, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    }
};
struct MmF16 {
    typedef _Float16 T;
    __device__ static __forceinline__ f32x16 mma(i32x4 x, i32x4 y, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    }
    __device__ static __forceinline__ f32x4 mma16(i32x4 x, i32x4 y, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    }
};

// The operands of one product, strides in bytes.  b2: with PAIR, the matrix of
// the second half of each wave's columns.  a_padded, b_padded: every row, the
// last too, may be read up to the next multiple of 8 elements.
struct MmOperands {
    const char* a;
    const char* b;
    const char* b2;
    int64_t lda, ldb, ldb2;
    int32_t M, N, K;
    int32_t a_padded, b_padded;
};

// Slices of 64 k that direct copies may read of an operand ACROSS k with
// `width` elements a row: their 16-byte chunks may pass a row's end, which must
// not be the last row's.
__device__ __forceinline__ int mm_direct_slices(int lay, int K, int width, int64_t ld, bool padded) {
    if (lay == ALONG || width % 8 == 0 || padded) return K / 64;
    const int last = (int)((14 + ld - 1) / ld);  // rows that end within 14 bytes of the operand's end
    return K > last ? (K - last) / 64 : 0;
}

template <class Tr_, int LA_, int LB_, int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, bool AHEAD_, bool PAIR_ = false>
struct MmTile {
    typedef Tr_ Tr;
    typedef typename Tr::T T;
    static constexpr int LA = LA_, LB = LB_, BM = BM_, BN = BN_;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr bool AHEAD = AHEAD_, PAIR = PAIR_;
    static constexpr int WAVES = WAVES_M * WAVES_N, NT = 64 * WAVES;
    static constexpr int BK = 64, ROW = 128, KSUB = 4;
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
    static constexpr int FM = WTM / 32, FN = WTN / 32;
    static constexpr int A_BYTES = BM * ROW, B_BYTES = BN * ROW, SLOT = A_BYTES + B_BYTES;
    static constexpr int RING = STAGES * SLOT, STAGE_BYTES = WAVES * 32 * WTN * 4;
    static constexpr int LDS_BYTES = RING > STAGE_BYTES ? RING : STAGE_BYTES;
    static constexpr int A_PER = BM * 8 / NT, B_PER = BN * 8 / NT, N_CP = A_PER + B_PER;
    static constexpr int NM = FM * FN;
    static constexpr int RA = LA == ALONG ? 1 : 2, RB = LB == ALONG ? 1 : 2;  // LDS reads per fragment
    static constexpr int NR = RA * FM + RB * FN;
    // columns of C: with PAIR, of each of the two matrices
    static constexpr int TILE_N = PAIR ? BN / 2 : BN, WAVE_N = PAIR ? WTN / 2 : WTN;

    // workgroups on the machine at once; nanoseconds of a slice where it is not
    // full; kilobytes of a tile's float sums
    static constexpr int SLOTS = LDS_BYTES > 80 * 1024 ? 256 : 512;
    static constexpr int SLICE_NS = BM * BN >= 65536 ? 1100 : BM * BN < 16384 ? 350 : SLOTS == 512 ? 650 : 400;
    static constexpr int TILE_KB = BM * BN / 256;

    typedef f32x16 Acc[FM][FN];

    static_assert(BM % (32 * WAVES_M) == 0 && BN % (32 * WAVES_N) == 0, "wave tile");
    static_assert((BM * 8) % NT == 0 && (BN * 8) % NT == 0, "even split of the copies");
    static_assert(!PAIR || (LB == ALONG && FN % 2 == 0), "pairs of fragments");
    static_assert(STAGES >= 2 && LDS_BYTES <= 160 * 1024, "LDS per CU");
    static_assert(N_CP * (STAGES - 2) <= 63, "vmcnt range");

    // ---- LDS layout ------------------------------------------------------------
    // ALONG: two 128-byte rows share the 256 bytes of all banks; 16 rows' chunks of
    // a read land on 16 different places.
    __device__ static __forceinline__ int along_chunk(int row, int c) { return c ^ ((row >> 1) & 7); }
    // ACROSS: the 4 rows x 64 bytes that 32 lanes of a transposing read touch
    // land on 4 different quarters of the banks.
    template <int W>
    __device__ static __forceinline__ int across_chunk(int k, int c) {
        return W >= 128 ? c ^ ((k & 3) << 2) : c ^ (((k >> 1) & 1) << 2);
    }
    // row of operand b that stands at LDS row p, relative to the tile's first; and
    // which matrix it is of
    __device__ static __forceinline__ int b_row(int p) { return PAIR ? (p / WTN) * WAVE_N + p % WAVE_N : p; }
    __device__ static __forceinline__ int b_half(int p) { return PAIR ? (p % WTN) / WAVE_N : 0; }

    // ---- copies ----------------------------------------------------------------
    // Per-lane byte offsets from the slice's first byte of the tile (the host keeps
    // them inside 32 bits).  Rows past an operand's last (ALONG) are read from the
    // last, chunks past a row's end (ACROSS) from the tile's first: they feed
    // only elements of C that are never stored.
    struct Offsets {
        uint32_t a[A_PER], b[B_PER];
    };
    template <int L, int W>
    __device__ static __forceinline__ uint32_t offset_of(int pos, int r0, int row, int rows, int64_t ld) {
        if constexpr (L == ALONG) {
            return (uint32_t)((int64_t)(min(r0 + row, rows - 1) - r0) * ld + along_chunk(pos >> 3, pos & 7) * 16);
        } else {
            const int k = pos / (W / 8), c = across_chunk<W>(k, pos % (W / 8));
            return (uint32_t)(k * ld + (r0 + c * 8 < rows ? c * 16 : 0));
        }
    }
    __device__ static __forceinline__ void offsets(Offsets& o, const MmOperands& g, int m0, int n0) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int q = 0; q < A_PER; ++q) o.a[q] = offset_of<LA, BM>(q * NT + tid, m0, (q * NT + tid) >> 3, g.M, g.lda);
#pragma unroll
        for (int q = 0; q < B_PER; ++q) {
            const int p = (q * NT + tid) >> 3;
            o.b[q] = offset_of<LB, BN>(q * NT + tid, n0, b_row(p), g.N, b_half(p) ? g.ldb2 : g.ldb);
        }
    }
    struct Source {
        const char *a, *b, *b2;
    };
    template <int L>
    __device__ static __forceinline__ const char* slice_at(const char* p, int64_t ld, int r0, int t) {
        return L == ALONG ? p + (int64_t)r0 * ld + (int64_t)t * ROW : p + (int64_t)t * BK * ld + (int64_t)r0 * 2;
    }
    __device__ static __forceinline__ Source source(const MmOperands& g, int m0, int n0, int t) {
        return Source{slice_at<LA>(g.a, g.lda, m0, t), slice_at<LB>(g.b, g.ldb, n0, t),
                      PAIR ? slice_at<LB>(g.b2, g.ldb2, n0, t) : nullptr};
    }
    __device__ static __forceinline__ void copy_one(int i, TG_LDS char* slot, const Offsets& o, const Source& s, int wave) {
        const uint32_t lds = (uint32_t)(uintptr_t)slot;
        if (i < A_PER) {
            copy16_to_lds(lds + (i * NT + wave * 64) * 16, o.a[i < A_PER ? i : 0], s.a);
        } else {
            const int q = i - A_PER;
            // the 8 LDS rows of one copy are of one matrix
            const bool second = PAIR && b_half((q * NT + wave * 64) >> 3);
            copy16_to_lds(lds + A_BYTES + (q * NT + wave * 64) * 16, o.b[q < B_PER ? q : 0], second ? s.b2 : s.b);
        }
    }
    __device__ static __forceinline__ void copy_slice(TG_LDS char* slot, const Offsets& o, const Source& s, int wave) {
#pragma unroll
        for (int i = 0; i < N_CP; ++i) copy_one(i, slot, o, s, wave);
    }

    // Slices that direct copies must not read (a row's end inside the slice, or
    // the operand's last rows): through registers, zero outside the operands.
    // Whole chunks take one load each (of zeros where there is nothing); the
    // chunk that a row ends in is cut out where rows are no whole chunks.
    template <int L, int W>
    __device__ static __forceinline__ i32x4 tail_chunk(int pos, int r0, int row, int rows, const char* p, int64_t ld, int t, int K) {
        const int line = pos / (L == ALONG ? 8 : W / 8);
        const int c = L == ALONG ? along_chunk(line, pos & 7) : across_chunk<W>(line, pos % (W / 8));
        // the operand's row, the chunk's first byte in it, the row's end
        const int r = L == ALONG ? min(r0 + row, rows - 1) : t * BK + line;
        const int at = L == ALONG ? t * ROW + c * 16 : (r0 + c * 8) * 2;
        const int end = L == ALONG ? K * 2 : rows * 2;
        const bool inside = L == ALONG || r < K;
        const char* q = p + (int64_t)(inside ? r : 0) * ld;
        const bool whole = inside && at + 16 <= end;
        i32x4 v = load16(whole ? q + at : reinterpret_cast<const char*>(g_zeros));
        if (end & 15) {  // wave-uniform
            const i32x4 cut = row_end_chunk(q, at, end);
            if (inside && !whole) v = cut;
        }
        return v;
    }
    __device__ static __forceinline__ void fill_slice(TG_LDS char* slot, const MmOperands& g, int m0, int n0, int t) {
        const int tid = threadIdx.x;
#pragma unroll 4
        for (int q = 0; q < A_PER; ++q)
            *reinterpret_cast<TG_LDS i32x4*>(slot + (q * NT + tid) * 16) =
                tail_chunk<LA, BM>(q * NT + tid, m0, (q * NT + tid) >> 3, g.M, g.a, g.lda, t, g.K);
#pragma unroll 4
        for (int q = 0; q < B_PER; ++q) {
            const int p = (q * NT + tid) >> 3;
            const bool second = PAIR && b_half(p);
            *reinterpret_cast<TG_LDS i32x4*>(slot + A_BYTES + (q * NT + tid) * 16) =
                tail_chunk<LB, BN>(q * NT + tid, n0, b_row(p), g.N, second ? g.b2 : g.b, second ? g.ldb2 : g.ldb, t, g.K);
        }
    }

    // ---- fragments -------------------------------------------------------------
    // Lane l holds r = r0 + l % 32, k 16 s + 8 (l / 32) .. + 7.
    struct Frags {
        i32x4 a[FM], b[FN];
    };
    template <int L, int W>
    __device__ static __forceinline__ void read_part(i32x4& f, const TG_LDS char* rows, int r0, int s, int h, int lane) {
        if constexpr (L == ALONG) {
            const int row = r0 + (lane & 31);
            f = *reinterpret_cast<const TG_LDS i32x4*>(rows + row * ROW + along_chunk(row, 2 * s + (lane >> 5)) * 16);
        } else {
            const int grp = lane >> 4, j = lane & 15;
            const int k = s * 16 + 8 * (grp >> 1) + (j >> 2) + 4 * h;
            const int r = r0 + 16 * (grp & 1) + 4 * (j & 3);
            const TG_LDS char* p = rows + k * (2 * W) + across_chunk<W>(k, r >> 3) * 16 + (r & 7) * 2;
            const i32x2 v = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS i16x4*)p));
            if (h == 0) {
                f.x = v.x;
                f.y = v.y;
            } else {
                f.z = v.x;
                f.w = v.y;
            }
        }
    }
    // LDS read number r of K step s, in the order the matrix instructions use
    // them: a0, b0 .. b(FN-1), a1 ..
    __device__ static __forceinline__ void read_one(Frags& f, const TG_LDS char* slot, int s, int r, int wm0, int wn0, int lane) {
        if (r < RA) {
            read_part<LA, BM>(f.a[0], slot, wm0, s, r, lane);
        } else if (r < RA + RB * FN) {
            const int j = (r - RA) / RB;
            read_part<LB, BN>(f.b[j < FN ? j : 0], slot + A_BYTES, wn0 + 32 * j, s, (r - RA) % RB, lane);
        } else {
            const int i = 1 + (r - RA - RB * FN) / RA;
            read_part<LA, BM>(f.a[i < FM ? i : 0], slot, wm0 + 32 * i, s, (r - RA - RB * FN) % RA, lane);
        }
    }
    __device__ static __forceinline__ void read_frags(Frags& f, const TG_LDS char* slot, int s, int wm0, int wn0, int lane) {
#pragma unroll
        for (int r = 0; r < NR; ++r) read_one(f, slot, s, r, wm0, wn0, lane);
    }
    __device__ static __forceinline__ void mma_one(int k, Acc& acc, const Frags& f) {
        acc[k / FN][k % FN] = Tr::mma(f.b[k % FN], f.a[k / FN], acc[k / FN][k % FN]);
    }

    // ---- the K loop ------------------------------------------------------------
    template <int A>
    __device__ static __forceinline__ void wait_ahead(int ahead) {
        if constexpr (A > 0) {
            if (ahead >= A) {
                wait_vm_then_barrier<A * N_CP>();
                return;
            }
            wait_ahead<A - 1>(ahead);
        } else {
            wait_vm_then_barrier<0>();
        }
    }
    // wait until at most `ahead` later slices' copies are in flight, then barrier
    __device__ static __forceinline__ void wait_slice(int ahead) { wait_ahead<STAGES - 2>(ahead); }

    // memory instructions [mem_begin(k), mem_begin(k + 1)) follow matrix
    // instruction k when `total` are spread over instructions first .. NM-1
    __device__ static constexpr int mem_begin(int k, int first, int total) {
        return k <= first ? 0 : ((k - first) * total + (NM - first) - 1) / (NM - first);
    }

    // One K step on `cur` with the reads of (rslot, rs) into `nxt` between the
    // matrix instructions; BARRIER: first meet the other waves (next slice
    // landed, this slot read), COPY: then also start a later slice.
    template <bool READS, bool BARRIER, bool COPY>
    __device__ static __forceinline__ void kstep(Acc& acc, const Frags& cur, Frags& nxt, const TG_LDS char* rslot, int rs,
                                                 int ahead, TG_LDS char* cslot, const Offsets& off, const Source& src, int wm0,
                                                 int wn0, int lane, int wave) {
        constexpr int BAR_K = (BARRIER && NM >= 8) ? 1 : 0;
        constexpr int NREAD = READS ? NR : 0, NC = COPY ? N_CP : 0, TOTAL = NREAD + NC, PER = TOTAL > 0 ? TOTAL : 1;
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            mma_one(k, acc, cur);
            if (BARRIER && k == BAR_K) wait_slice(ahead);
#pragma unroll
            for (int m = mem_begin(k, BAR_K, TOTAL); m < mem_begin(k + 1, BAR_K, TOTAL); ++m) {
                const int c0 = m * NC / PER, c1 = (m + 1) * NC / PER;
                if (c1 > c0) copy_one(c0, cslot, off, src, wave);
                else read_one(nxt, rslot, rs, m - c1, wm0, wn0, lane);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    template <int S, bool NEXT, bool COPY>
    __device__ static __forceinline__ void slice_steps(Acc& acc, Frags (&f)[2], TG_LDS char* cur, const TG_LDS char* next,
                                                       int ahead, const Offsets& off, const Source& src, int wm0, int wn0,
                                                       int lane, int wave) {
        if constexpr (S + 1 < KSUB) {
            kstep<true, false, false>(acc, f[S & 1], f[(S + 1) & 1], cur, S + 1, 0, cur, off, src, wm0, wn0, lane, wave);
            slice_steps<S + 1, NEXT, COPY>(acc, f, cur, next, ahead, off, src, wm0, wn0, lane, wave);
        } else {
            kstep<NEXT, NEXT, COPY>(acc, f[S & 1], f[(S + 1) & 1], next, 0, ahead, cur, off, src, wm0, wn0, lane, wave);
        }
    }
    // AHEAD: every fragment register is refilled with the next slice's values
    // right after its use (waves with few matrix instructions per K step).
    template <bool NEXT, bool COPY>
    __device__ static __forceinline__ void slice_ahead(Acc& acc, Frags (&F)[KSUB], TG_LDS char* cur, const TG_LDS char* next,
                                                       int ahead, const Offsets& off, const Source& src, int wm0, int wn0,
                                                       int lane, int wave) {
#pragma unroll
        for (int s = 0; s < KSUB; ++s) {
#pragma unroll
            for (int k = 0; k < NM; ++k) mma_one(k, acc, F[s]);
            if constexpr (NEXT) {
                if (s == 0) wait_slice(ahead);
                read_frags(F[s], next, s, wm0, wn0, lane);
            }
            if constexpr (COPY) {
                if (s == 0) copy_slice(cur, off, src, wave);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    __device__ static __forceinline__ void clear(Acc& acc) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    }

    // Adds slices t0 .. t1 - 1 of the product of tile (m0, n0) to acc.  Ends with
    // every wave past its last LDS read.
    __device__ static __forceinline__ void product(const MmOperands& g, int m0, int n0, int t0, int t1, TG_LDS char* smem,
                                                   Acc& acc, int wm0, int wn0, int lane, int wave) {
        const int direct = min(mm_direct_slices(LA, g.K, g.M, g.lda, g.a_padded), mm_direct_slices(LB, g.K, g.N, g.ldb, g.b_padded));
        const int n = min(t1, direct) - t0;  // slices by direct copies
        if (n > 0) {
            Offsets off;
            offsets(off, g, m0, n0);
            auto slot = [&](int t) { return smem + (t % STAGES) * SLOT; };
            auto from = [&](int t) { return source(g, m0, n0, t0 + t); };
            // slices 0 .. STAGES-2 in flight; with slice 0 in LDS, start slice
            // STAGES-1 and read the first fragments
#pragma unroll
            for (int t = 0; t < STAGES - 1; ++t)
                if (t < n) copy_slice(slot(t), off, from(t), wave);
            const Source none{g.a, g.b, g.b2};
            wait_slice(min(STAGES - 2, n - 1));
            if (STAGES - 1 < n) copy_slice(slot(STAGES - 1), off, from(STAGES - 1), wave);
            int t = 0;
            if constexpr (AHEAD) {
                Frags F[KSUB];
#pragma unroll
                for (int s = 0; s < KSUB; ++s) read_frags(F[s], smem, s, wm0, wn0, lane);
                for (; t + STAGES < n; ++t)
                    slice_ahead<true, true>(acc, F, slot(t), slot(t + 1), STAGES - 2, off, from(t + STAGES), wm0, wn0, lane, wave);
                for (; t + 1 < n; ++t)
                    slice_ahead<true, false>(acc, F, slot(t), slot(t + 1), min(STAGES - 2, n - 2 - t), off, none, wm0, wn0, lane, wave);
                slice_ahead<false, false>(acc, F, smem, smem, 0, off, none, wm0, wn0, lane, wave);
            } else {
                Frags f[2];
                read_frags(f[0], smem, 0, wm0, wn0, lane);
                for (; t + STAGES < n; ++t)
                    slice_steps<0, true, true>(acc, f, slot(t), slot(t + 1), STAGES - 2, off, from(t + STAGES), wm0, wn0, lane, wave);
                for (; t + 1 < n; ++t)
                    slice_steps<0, true, false>(acc, f, slot(t), slot(t + 1), min(STAGES - 2, n - 2 - t), off, none, wm0, wn0, lane, wave);
                slice_steps<0, false, false>(acc, f, slot(t), smem, 0, off, none, wm0, wn0, lane, wave);
            }
            wait_lds_then_barrier();
        }
        for (int t = max(t0, min(t1, direct)); t < t1; ++t) {
            fill_slice(smem, g, m0, n0, t);
            wait_lds_then_barrier();
            Frags f;
#pragma unroll 1
            for (int s = 0; s < KSUB; ++s) {
                if (t * BK + s * 16 >= g.K) break;
                read_frags(f, smem, s, wm0, wn0, lane);
#pragma unroll
                for (int k = 0; k < NM; ++k) mma_one(k, acc, f);
            }
            wait_lds_then_barrier();
        }
    }

    // ---- the way out -----------------------------------------------------------
    // Calls each(u, v, w, data) for every 8 adjacent columns of the wave's block:
    // those at lane_col(lane) of row u + lane_row(lane), u the same for the whole
    // wave; v their sums, w (PAIR) those of the second matrix.  32 rows at a time go
    // through the wave's own LDS; before that, fetch(u, data) starts the loads that
    // `each` will want, all of the 32 rows' in flight together.  The walk over the
    // 32-row blocks is a loop, so that `each` stands in the code once.
    static constexpr int PER_ROW = WAVE_N / 8;     // lanes a row
    static constexpr int ROWS = 64 / PER_ROW;      // rows an instruction
    static constexpr int PIECES = 32 / ROWS;       // instructions a block
    template <int I>
    __device__ static __forceinline__ void stage(int i, const Acc& acc, TG_LDS char* mine, int lane) {
        if constexpr (I < FM) {
            if (i == I) {
                // the empty statements keep the compiler from merging the blocks
                // into one that indexes acc, which would then stand in memory
                asm volatile("; block %0 from here" ::"n"(I) : "memory");
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *reinterpret_cast<TG_LDS f32x4*>(staged(mine, lane & 31, 8 * j + 2 * r + (lane >> 5))) =
                            f32x4{acc[I][j][4 * r], acc[I][j][4 * r + 1], acc[I][j][4 * r + 2], acc[I][j][4 * r + 3]};
                asm volatile("; block %0 to here" ::"n"(I) : "memory");
            } else {
                stage<I + 1>(i, acc, mine, lane);
            }
        }
    }
    __device__ static __forceinline__ TG_LDS char* staged(TG_LDS char* mine, int row, int c) {
        return mine + row * (WTN * 4) + (c ^ (row & (WTN / 4 - 1))) * 16;
    }
    __device__ static __forceinline__ int lane_row(int lane) { return lane / PER_ROW; }
    __device__ static __forceinline__ int lane_col(int lane) { return 8 * (lane % PER_ROW); }
    template <class Data, class Fetch, class Each>
    __device__ static __forceinline__ void each_row(const Acc& acc, TG_LDS char* smem, int lane, int wave, Fetch fetch, Each each) {
        TG_LDS char* mine = smem + wave * (32 * WTN * 4);
        const int r0 = lane_row(lane), c = lane_col(lane) / 4;
#pragma unroll 1
        for (int i = 0; i < FM; ++i) {
            Data data[PIECES];
#pragma unroll
            for (int q = 0; q < PIECES; ++q) fetch(32 * i + q * ROWS, data[q]);
            stage<0>(i, acc, mine, lane);
            asm volatile("" ::: "memory");  // a wave's LDS accesses stay in order
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int row = q * ROWS + r0;
                float v[8], w[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 x = *reinterpret_cast<const TG_LDS f32x4*>(staged(mine, row, c + h));
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * h + e] = x[e];
                    if constexpr (PAIR) {
                        const f32x4 y = *reinterpret_cast<const TG_LDS f32x4*>(staged(mine, row, WTN / 8 + c + h));
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[4 * h + e] = y[e];
                    }
                }
                each(32 * i + q * ROWS, v, w, data[q]);
            }
            asm volatile("" ::: "memory");
        }
    }
    struct Nothing {};
    template <class Each>
    __device__ static __forceinline__ void each_row(const Acc& acc, TG_LDS char* smem, int lane, int wave, Each each) {
        each_row<Nothing>(acc, smem, lane, wave, [](int, Nothing&) {},
                          [&](int u, float (&v)[8], float (&w)[8], Nothing&) { each(u, v, w); });
    }
    // Whether the wave's block, at row m1 and column n1 of M x N results, lies
    // inside them: decided once, the way out then has no checks.
    __device__ static __forceinline__ bool inside(int m1, int n1, int M, int N) { return m1 + WTM <= M && n1 + WAVE_N <= N; }
};

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// 8 adjacent values in memory.
struct Raw8 {
    i32x4 v;
};
template <class T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
    T o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (T)v[e];  // to nearest even
    __builtin_memcpy(dst, o, 16);
}
// The same past the caches.
template <class T>
__device__ __forceinline__ void stream8(T* dst, const float (&v)[8]) {
    T o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (T)v[e];
    i32x4 w;
    __builtin_memcpy(&w, o, 16);
    __builtin_nontemporal_store(w, reinterpret_cast<i32x4*>(dst));
}
// `count` of them, which may be none, inside the row.  The empty statements keep
// the compiler from making one run of element stores of both branches.
template <class T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8], int count) {
    if (count >= 8) {
        store8(dst, v);
    } else {
        asm volatile("; part of 8" ::: "memory");
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < count) dst[e] = (T)v[e];
        asm volatile("; part of 8 ends" ::: "memory");
    }
}
template <class T>
__device__ __forceinline__ void load8(Raw8& x, const T* src) { x.v = load16(src); }
template <class T>
__device__ __forceinline__ void values8(float (&v)[8], const Raw8& x) {
    T o[8];
    __builtin_memcpy(o, &x.v, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)o[e];
}

}  // namespace tg
