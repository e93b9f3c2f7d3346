// Matrix products C = A B^T with both operands K-contiguous (rows of A and
// rows of B run along K), on the matrix cores: 8-bit floating point operands
// with a power-of-two scale for each 128 of a row, and half precision
// operands.  What happens to a workgroup's block of C is an epilogue given
// as a template parameter.
//
// A workgroup computes one BM x BN tile; its waves form a WAVES_M x WAVES_N
// grid, each wave owning a WTM x WTN block of 32 x 32 matrix-core tiles.  The
// K loop walks slices of 128 bytes of a row (128 8-bit or 64 half precision
// values: for 8-bit operands a slice is one scale block) through a ring of
// STAGES LDS slots filled by direct global -> LDS copies, with one barrier a
// slice.
//
// Rows inside a wave's block are dealt to its 32-row fragments in turn: row
// F r + i of the block is row r of fragment i (F fragments; F = WTM / 32 for
// A and WTN / 32 for B).  Three things follow.  The scales of one lane's row
// in all F fragments are F adjacent bytes: one LDS read of F bytes serves
// them, and the matrix instruction picks its byte (op_sel), so scaling costs
// no vector instruction.  The F results of one C row in one lane are F
// adjacent columns: one store of F values, 32 lanes covering a whole line.
// And the 4 F results of one column that four registers of F fragments hold
// are 4 F adjacent rows, so a transposed copy of C takes wide stores as well.
// In LDS the rows stand in fragment order, so fragment reads see the usual
// 128-byte rows: the copy fetches them from where they are.
#pragma once

#include "tg_device.hpp"

namespace tg {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Formats of 8-bit operands, in the matrix instruction's numbering.
enum Fp8Format { FMT_E4M3 = 0, FMT_E5M2 = 1 };

template <int LB>
struct NtFrag {
    i32x4 v[LB / 16];
};

// v_mfma_scale_f32_32x32x64_f8f6f4: each lane holds 32 bytes of one row.  A
// lane's scale byte (2^(byte - 127)) stands for its 32 values of K, all of
// one 128-block here.  It adds in float, but aligns the products of a group
// of eight to the largest of them and keeps 13 bits below it (measured: random
// sums are off by about 2^-17 of the sum of |a b|), enough for a bfloat16
// result.
template <int FA, int FB>
struct NtF8 {
    static constexpr int LB = 32;     // bytes a lane holds of its row in one K step
    static constexpr bool SCALED = true;
    static constexpr bool PARTIAL = true;  // rows may end inside a slice
    typedef NtFrag<32> Frag;
    template <int OA, int OB>
    __device__ static __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c, int sa, int sb) {
        const i32x8 x = __builtin_shufflevector(a.v[0], a.v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 y = __builtin_shufflevector(b.v[0], b.v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, FA, FB, OA, sa, OB, sb);
    }
};

// v_mfma_f32_32x32x16_f16.
struct NtF16 {
    static constexpr int LB = 16;
    static constexpr bool SCALED = false;
    static constexpr bool PARTIAL = false;
    typedef NtFrag<16> Frag;
    template <int, int>
    __device__ static __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c, int, int) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.v[0]),
                                                      __builtin_bit_cast(f16x8, b.v[0]), c, 0, 0, 0);
    }
};

// The operands of one product.  A: M rows of `k` bytes, row stride lda bytes;
// B: N rows.  Scales (8-bit operands): one byte per row and 128-block,
// sa[block * ldsa + row], rows of the table 4-byte aligned and readable up to
// the row count rounded up to 4.
struct NtOperands {
    const char* a;
    const char* b;
    const uint8_t* sa;
    const uint8_t* sb;
    int32_t M, N, k;
    int64_t lda, ldb, ldsa, ldsb;
};

// Rank of workgroup b among `total` when consecutive ranks run on one XCD:
// the hardware deals workgroups to the 8 XCDs in turn, and ranks that share
// operand panels should share an L2.
__device__ __forceinline__ int xcd_rank(int b, int total) {
    const int x = b & 7, per = total >> 3, more = total & 7;
    return x * per + min(x, more) + (b >> 3);
}

// Tile of rank r in groups of `group` tile rows walked column by column.
__device__ __forceinline__ void grouped_tile(int r, int tiles_m, int tiles_n, int group, int& tm, int& tn) {
    const int per_group = group * tiles_n;
    const int g = r / per_group;
    const int rows = min(tiles_m - g * group, group);
    const int in_group = r - g * per_group;
    tm = g * group + in_group % rows;
    tn = in_group / rows;
}

// Bytes at .. at + 15 of a row of `end` bytes, zero past its end: one 16-byte
// load that ends inside the row, shifted into place (rows shorter than that:
// byte loads).
__device__ __forceinline__ i32x4 row_end_chunk(const char* row, int at, int end) {
    if (end >= 16) {  // wave-uniform
        const int sh = max(at - (end - 16), 0);
        const i32x4 x = load16(row + (at - sh));
        const i32x4 y = funnel16(x, i32x4{0, 0, 0, 0}, sh & 15);
        return sh < 16 ? y : i32x4{0, 0, 0, 0};
    }
    union { i32x4 v; uint8_t b[16]; } u;
#pragma unroll
    for (int t = 0; t < 16; ++t) u.b[t] = load_or_zero(reinterpret_cast<const uint8_t*>(row) + at + t, at + t < end);
    return u.v;
}

// AHEAD: every fragment register is refilled with the next slice's values
// right after its use, a whole slice ahead (waves with few matrix
// instructions per K step); otherwise fragments are double-buffered by K
// step and the reads spread between matrix instructions.
template <class Tr, int BM_, int BN_, int WAVES_M, int WAVES_N, int STAGES, bool AHEAD>
struct NtGemm {
    static constexpr int BM = BM_, BN = BN_;
    static constexpr int WAVES = WAVES_M * WAVES_N;
    static constexpr int NT = 64 * WAVES;
    static constexpr int ROW = 128;  // bytes of K per slice
    static constexpr int LB = Tr::LB;
    static constexpr int KSUB = ROW / (2 * LB);
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
    static constexpr int FM = WTM / 32, FN = WTN / 32;
    static constexpr int A_BYTES = BM * ROW, B_BYTES = BN * ROW;
    // scales in a slot: 256 bytes for each wave's copy, of which the first
    // 4 S_PER count (see copy_one)
    static constexpr int S_BYTES = Tr::SCALED ? 256 * WAVES : 0;
    static constexpr int SLOT = A_BYTES + B_BYTES + S_BYTES;
    static constexpr int SLOTS = STAGES;
    static constexpr int LDS_BYTES = SLOTS * SLOT;
    static constexpr int A_PER = BM * 8 / NT, B_PER = BN * 8 / NT;
    static constexpr int S_PER = (BM + BN) / 4 / WAVES;  // scale dwords each wave copies
    static constexpr int N_CP = A_PER + B_PER + (Tr::SCALED ? 1 : 0);
    // an epilogue's inputs fit in registers beside the product's
    static constexpr bool EARLY = FM * FN * WAVES <= 16;
    static constexpr int NM = FM * FN;
    static constexpr int RB = LB / 16;  // LDS reads per fragment
    static constexpr int NS = Tr::SCALED ? 2 : 0;
    static constexpr int NR = NS + RB * (FM + FN);

    typedef typename Tr::Frag Frag;
    typedef f32x16 Acc;

    static_assert(BM % (32 * WAVES_M) == 0 && BN % (32 * WAVES_N) == 0, "wave tile");
    static_assert(!Tr::SCALED || ((FM == 1 || FM == 2 || FM == 4) && (FN == 1 || FN == 2 || FN == 4)),
                  "scale bytes of a lane are read at once");
    static_assert((BM * 8) % NT == 0 && (BN * 8) % NT == 0, "even split of the copies");
    static_assert(!Tr::SCALED || ((BM / 4) % S_PER == 0 && S_PER <= 64 && (S_PER & (S_PER - 1)) == 0),
                  "a wave's scale copy is of one operand");
    static_assert(STAGES >= 2 && LDS_BYTES <= 160 * 1024, "LDS per CU");
    static_assert(N_CP * (STAGES - 2) <= 63, "vmcnt range");
    static_assert(SLOT % 16 == 0, "slots stay aligned");

    // 16-byte chunk c of LDS row r stands at chunk c ^ key(r): two 128-byte
    // rows share one 256-byte bank window, so the 16 rows that 16 lanes of a
    // 16-byte read touch land on 16 different chunks of it.
    __device__ static __forceinline__ int chunk_of(int row, int c) { return c ^ ((row >> 1) & 7); }

    // tile row that stands at LDS row p (wave blocks of WT rows)
    template <int WT>
    __device__ static __forceinline__ int row_at(int p) {
        return (p / WT) * WT + (WT / 32) * (p & 31) + (p % WT) / 32;
    }

    struct Offsets {
        uint32_t a[A_PER], b[B_PER], s;
    };
    // per-lane byte offsets of the copies from the slice's first byte of the
    // tile's first row (scales: from the wave's operand's table row); rows
    // past the operand's last are read from the last: they only feed elements
    // of C that are never stored.  Rows shorter than a slice: chunks that pass
    // the row's end are its last 16 bytes.
    __device__ static __forceinline__ void offsets(Offsets& o, const NtOperands& g, int m0, int n0, int wave,
                                                   int lane) {
        const int tid = threadIdx.x, most = Tr::PARTIAL ? g.k - 16 : ROW;
#pragma unroll
        for (int q = 0; q < A_PER; ++q) {
            const int p = (q * NT + tid) >> 3, c = chunk_of(p, tid & 7);
            o.a[q] = (uint32_t)((int64_t)(min(m0 + row_at<WTM>(p), g.M - 1) - m0) * g.lda + min(c * 16, most));
        }
#pragma unroll
        for (int q = 0; q < B_PER; ++q) {
            const int p = (q * NT + tid) >> 3, c = chunk_of(p, tid & 7);
            o.b[q] = (uint32_t)((int64_t)(min(n0 + row_at<WTN>(p), g.N - 1) - n0) * g.ldb + min(c * 16, most));
        }
        if constexpr (Tr::SCALED) {
            const int d = wave * S_PER + lane % S_PER;  // dword of the tile's scales: A's, then B's
            o.s = d < BM / 4 ? min(m0 + 4 * d, (g.M - 1) & ~3) : min(n0 + 4 * (d - BM / 4), (g.N - 1) & ~3);
        }
    }

    // where the copies of one slice come from: wave-uniform addresses.  A last,
    // partial slice is the row's last 128 bytes, of which the first were in the
    // slice before: no copy leaves its row.
    struct Source {
        const char* a;
        const char* b;
        const uint8_t* s;
    };
    __device__ static __forceinline__ Source source(const NtOperands& g, int m0, int n0, int sl, int wave) {
        Source r;
        const int64_t at = Tr::PARTIAL ? max(min((int64_t)sl * ROW, (int64_t)g.k - ROW), (int64_t)0) : (int64_t)sl * ROW;
        r.a = g.a + (int64_t)m0 * g.lda + at;
        r.b = g.b + (int64_t)n0 * g.ldb + at;
        r.s = nullptr;
        if constexpr (Tr::SCALED)
            r.s = wave * S_PER < BM / 4 ? g.sa + (int64_t)sl * g.ldsa : g.sb + (int64_t)sl * g.ldsb;
        return r;
    }

    // copy number i of a slice (0 <= i < N_CP).  The scales: S_PER dwords for
    // each wave, which every group of S_PER lanes fetches again, so that the
    // copy needs no branch (one splits the K loop for the compiler, which
    // then spills fragments) and no wave copies more than another (one wait
    // count serves all).
    __device__ static __forceinline__ void copy_one(int i, TG_LDS char* slot, const Offsets& o, const Source& s,
                                                    int wave) {
        const uint32_t lds = (uint32_t)(uintptr_t)slot;
        if (i < A_PER) copy16_to_lds(lds + (i * NT + wave * 64) * 16, o.a[i < A_PER ? i : 0], s.a);
        else if (i < A_PER + B_PER)
            copy16_to_lds(lds + A_BYTES + ((i - A_PER) * NT + wave * 64) * 16, o.b[i - A_PER < B_PER ? i - A_PER : 0],
                          s.b);
        else copy4_to_lds(lds + A_BYTES + B_BYTES + wave * 256, o.s, s.s);
    }
    __device__ static __forceinline__ void copy_slice(TG_LDS char* slot, const Offsets& o, const Source& s, int wave) {
#pragma unroll
        for (int i = 0; i < N_CP; ++i) copy_one(i, slot, o, s, wave);
    }

    // ---- fragments ---------------------------------------------------------
    struct Frags {
        Frag a[FM], b[FN];
        int sa, sb;
    };
    // The F scale bytes of rows at, at + 1 .. (at a multiple of F) of the
    // tile's BM + BN rows.
    template <int F>
    __device__ static __forceinline__ int read_scales(const TG_LDS char* slot, int at) {
        const TG_LDS char* p = slot + A_BYTES + B_BYTES + at / (4 * S_PER) * 256 + at % (4 * S_PER);
        if constexpr (F == 4) return *reinterpret_cast<const TG_LDS int32_t*>(p);
        else if constexpr (F == 2) return *reinterpret_cast<const TG_LDS uint16_t*>(p);
        else return *reinterpret_cast<const TG_LDS uint8_t*>(p);
    }
    // read h of the fragment at LDS row `row0`, K step s.  Which of the
    // step's chunks a lane takes is free as long as A and B agree: lanes
    // 0-31 read one chunk, lanes 32-63 the next.
    __device__ static __forceinline__ i32x4 read_chunk(const TG_LDS char* rows, int row0, int s, int h, int lane) {
        const int row = row0 + (lane & 31);
        const int c = 2 * RB * s + 2 * h + (lane >> 5);
        return *reinterpret_cast<const TG_LDS i32x4*>(rows + row * ROW + chunk_of(row, c) * 16);
    }
    // LDS read number r of K step s, in the order the matrix instructions
    // use them: scales, a0, b0 .. b(FN-1), a1 ..
    __device__ static __forceinline__ void read_one(Frags& f, const TG_LDS char* slot, int s, int r, int wm0, int wn0,
                                                    int lane) {
        if (r < NS) {
            if (r == 0) f.sa = read_scales<FM>(slot, wm0 + FM * (lane & 31));
            else f.sb = read_scales<FN>(slot, BM + wn0 + FN * (lane & 31));
            return;
        }
        const int q = (r - NS) / RB, h = (r - NS) % RB;
        if (q == 0) f.a[0].v[h] = read_chunk(slot, wm0, s, h, lane);
        else if (q <= FN) f.b[q - 1 < FN ? q - 1 : 0].v[h] = read_chunk(slot + A_BYTES, wn0 + 32 * (q - 1), s, h, lane);
        else f.a[q - FN < FM ? q - FN : 0].v[h] = read_chunk(slot, wm0 + 32 * (q - FN), s, h, lane);
    }
    __device__ static __forceinline__ void read_frags(Frags& f, const TG_LDS char* slot, int s, int wm0, int wn0,
                                                      int lane) {
#pragma unroll
        for (int r = 0; r < NR; ++r) read_one(f, slot, s, r, wm0, wn0, lane);
    }

    // matrix instruction number k of a K step; the byte of the scale
    // registers is an immediate, so k selects among compile-time instances
    template <int K = 0>
    __device__ static __forceinline__ void mma_one(int k, Acc (&acc)[FM][FN], const Frags& f) {
        if constexpr (K < NM) {
            if (k == K) acc[K / FN][K % FN] = Tr::template mma<K / FN, K % FN>(f.a[K / FN], f.b[K % FN],
                                                                               acc[K / FN][K % FN], f.sa, f.sb);
            else mma_one<K + 1>(k, acc, f);
        }
    }

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

    // One K step on `cur` with the reads of (rslot, rs) into `nxt` between
    // the matrix instructions; BARRIER: first meet the other waves (next
    // slice landed, this slot read), COPY: then also start a later slice.
    template <bool READS, bool BARRIER, bool COPY>
    __device__ static __forceinline__ void kstep(Acc (&acc)[FM][FN], const Frags& cur, Frags& nxt,
                                                 const TG_LDS char* rslot, int rs, int ahead, TG_LDS char* cslot,
                                                 const Offsets& off, const Source& src, int wm0, int wn0, int lane,
                                                 int wave) {
        constexpr int BAR_K = (BARRIER && NM >= 8) ? 1 : 0;
        constexpr int NREAD = READS ? NR : 0, TOTAL = NREAD + (COPY ? N_CP : 0);
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            mma_one(k, acc, cur);
            if (BARRIER && k == BAR_K) wait_slice(ahead);
#pragma unroll
            for (int m = mem_begin(k, BAR_K, TOTAL); m < mem_begin(k + 1, BAR_K, TOTAL); ++m) {
                // copies and reads in turn: copies after all the reads would
                // have less than a slice to land (8192^3 e4m3: 439 us against
                // 425), reads after all the copies would come late for the
                // next K step with one wave a SIMD (4096^3: 61 against 57)
                constexpr int NC = TOTAL - NREAD, PER = TOTAL > 0 ? TOTAL : 1;
                const int c0 = m * NC / PER, c1 = (m + 1) * NC / PER;
                if (c1 > c0) copy_one(c0, cslot, off, src, wave);
                else read_one(nxt, rslot, rs, m - c1, wm0, wn0, lane);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Slice t: K steps 0 .. KSUB-1; the last reads slice t+1's first
    // fragments (NEXT) after the slice's barrier and starts slice t+STAGES
    // into the slot that this one leaves (COPY).
    template <int S, bool NEXT, bool COPY>
    __device__ static __forceinline__ void slice_steps(Acc (&acc)[FM][FN], Frags (&f)[2], TG_LDS char* cur,
                                                       const TG_LDS char* next, int ahead, const Offsets& off,
                                                       const Source& src, int wm0, int wn0, int lane, int wave) {
        if constexpr (S + 1 < KSUB) {
            kstep<true, false, false>(acc, f[S & 1], f[(S + 1) & 1], cur, S + 1, 0, cur, off, src, wm0, wn0, lane,
                                      wave);
            slice_steps<S + 1, NEXT, COPY>(acc, f, cur, next, ahead, off, src, wm0, wn0, lane, wave);
        } else {
            kstep<NEXT, NEXT, COPY>(acc, f[S & 1], f[(S + 1) & 1], next, 0, ahead, cur, off, src, wm0, wn0, lane,
                                    wave);
        }
    }

    // Slice t with whole-slice read-ahead: step s's registers are refilled
    // from slice t+1 right after their use.  The barrier follows step 0: this
    // wave read all of its slot during slice t-1.
    template <bool NEXT, bool COPY>
    __device__ static __forceinline__ void slice_ahead(Acc (&acc)[FM][FN], Frags (&F)[KSUB], TG_LDS char* cur,
                                                       const TG_LDS char* next, int ahead, const Offsets& off,
                                                       const Source& src, int wm0, int wn0, int lane, int wave) {
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

    // ---- rows of less than 16 bytes --------------------------------------------
    // Through registers: zero past the row's end (a zero in both operands adds
    // nothing).
    __device__ static __forceinline__ void fill_short(TG_LDS char* slot, const NtOperands& g, int m0, int n0) {
        const int tid = threadIdx.x;
        // every chunk's load is in flight before the first is stored
        i32x4 v[A_PER + B_PER];
#pragma unroll
        for (int q = 0; q < A_PER + B_PER; ++q) {
            const bool a = q < A_PER;
            const int p = ((a ? q : q - A_PER) * NT + tid) >> 3, c = chunk_of(p, tid & 7);
            const char* rowp = a ? g.a + (int64_t)min(m0 + row_at<WTM>(p), g.M - 1) * g.lda
                                 : g.b + (int64_t)min(n0 + row_at<WTN>(p), g.N - 1) * g.ldb;
            v[q] = row_end_chunk(rowp, c * 16, g.k);
        }
#pragma unroll
        for (int q = 0; q < A_PER + B_PER; ++q)
            *reinterpret_cast<TG_LDS i32x4*>(slot + (q < A_PER ? 0 : A_BYTES) +
                                             ((q < A_PER ? q : q - A_PER) * NT + tid) * 16) = v[q];
        if constexpr (Tr::SCALED) {
            if (tid < (BM + BN) / 4) {
                const uint8_t* p = tid < BM / 4
                    ? g.sa + min(m0 + 4 * tid, (g.M - 1) & ~3)
                    : g.sb + min(n0 + 4 * (tid - BM / 4), (g.N - 1) & ~3);
                *reinterpret_cast<TG_LDS int32_t*>(slot + A_BYTES + B_BYTES + tid / S_PER * 256 + tid % S_PER * 4) =
                    *reinterpret_cast<const int32_t*>(p);
            }
        }
    }

    // Fragments of K step s of the partial slice, zero where its copies hold
    // bytes that do not count: the first 128 - left of them, which were in the
    // slice before; in rows shorter than a slice (`alone`), those that the last
    // chunk repeats and the chunks behind it.
    __device__ static __forceinline__ void mask_partial(Frags& f, int s, int left, bool alone, int lane) {
#pragma unroll
        for (int h = 0; h < RB; ++h) {
            const int c = 2 * RB * s + 2 * h + (lane >> 5);  // this lane's chunk
            const int gone = !alone ? ROW - left - 16 * c : c < left / 16 ? 0 : c == left / 16 ? 16 - left % 16 : 16;
            i32x4 keep;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int n = min(max(gone - 4 * w, 0), 4);
                keep[w] = n == 4 ? 0 : (int)(0xffffffffu << (8 * n));
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) f.a[i].v[h] &= keep;
#pragma unroll
            for (int j = 0; j < FN; ++j) f.b[j].v[h] &= keep;
        }
    }

    // The product of tile (m0, n0) into acc.
    __device__ static __forceinline__ void product(const NtOperands& g, int m0, int n0, TG_LDS char* smem,
                                                   Acc (&acc)[FM][FN], int wm0, int wn0, int lane, int wave) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        // whole slices, and with a partial one (of `left` bytes) behind them,
        // which is copied like the others
        const int full = g.k / ROW, left = g.k % ROW, total = Tr::PARTIAL && g.k >= 16 && left > 0 ? full + 1 : full;
        Offsets off;
        offsets(off, g, m0, n0, wave, lane);
        auto slot = [&](int t) { return smem + (t % STAGES) * SLOT; };
        auto copy = [&](int t) { copy_slice(slot(t), off, source(g, m0, n0, t, wave), wave); };
        const Source none{g.a, g.b, g.sa};
        // prologue: slices 0 .. STAGES-2 in flight; with slice 0 in LDS, start
        // slice STAGES-1 and read the first fragments
#pragma unroll
        for (int t = 0; t < STAGES - 1; ++t)
            if (t < total) copy(t);
        if constexpr (AHEAD) {
            Frags F[KSUB];
            if (full > 0) {
                wait_slice(min(STAGES - 2, total - 1));
                if (STAGES - 1 < total) copy(STAGES - 1);
#pragma unroll
                for (int s = 0; s < KSUB; ++s) read_frags(F[s], smem, s, wm0, wn0, lane);
            }
            int t = 0;
            for (; t + STAGES < total; ++t)
                slice_ahead<true, true>(acc, F, slot(t), slot(t + 1), STAGES - 2, off,
                                        source(g, m0, n0, t + STAGES, wave), wm0, wn0, lane, wave);
            for (; t + 1 < full; ++t)
                slice_ahead<true, false>(acc, F, slot(t), slot(t + 1), min(STAGES - 2, total - 2 - t), off, none, wm0,
                                         wn0, lane, wave);
            if (t < full) slice_ahead<false, false>(acc, F, smem, smem, 0, off, none, wm0, wn0, lane, wave);
        } else {
            Frags f[2];
            static_assert(AHEAD || KSUB % 2 == 0, "a slice starts on buffer 0");
            if (full > 0) {
                wait_slice(min(STAGES - 2, total - 1));
                if (STAGES - 1 < total) copy(STAGES - 1);
                read_frags(f[0], smem, 0, wm0, wn0, lane);
            }
            int t = 0;
            for (; t + STAGES < total; ++t)
                slice_steps<0, true, true>(acc, f, slot(t), slot(t + 1), STAGES - 2, off,
                                           source(g, m0, n0, t + STAGES, wave), wm0, wn0, lane, wave);
            for (; t + 1 < full; ++t)
                slice_steps<0, true, false>(acc, f, slot(t), slot(t + 1), min(STAGES - 2, total - 2 - t), off, none,
                                            wm0, wn0, lane, wave);
            if (t < full) slice_steps<0, false, false>(acc, f, slot(t), smem, 0, off, none, wm0, wn0, lane, wave);
        }
        if (Tr::PARTIAL && left > 0) {
            TG_LDS char* s = slot(full);
            if (g.k >= 16) {
                wait_slice(0);
            } else {
                fill_short(s, g, m0, n0);
                wait_lds_then_barrier();
            }
            const bool alone = full == 0;
            Frags f;
            for (int u = alone ? 0 : (ROW - left) / (2 * LB); u * (2 * LB) < (alone ? left : ROW); ++u) {
                read_frags(f, s, u, wm0, wn0, lane);
                if (g.k >= 16) mask_partial(f, u, left, alone, lane);
#pragma unroll
                for (int k = 0; k < NM; ++k) mma_one(k, acc, f);
            }
        }
    }

    // Element (row, column) of the wave's block that register r of tile
    // (i, j) holds in this lane.
    __device__ static __forceinline__ int row_of(int i, int r, int lane) {
        return FM * (8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) + i;
    }
    __device__ static __forceinline__ int col_of(int j, int lane) { return FN * (lane & 31) + j; }
};

}  // namespace tg
