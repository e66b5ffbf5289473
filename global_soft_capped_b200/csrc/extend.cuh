// extend.cuh -- attention of a chunk of new tokens per sequence (1 .. some
// tens) over a paged KV cache with pages of any power of two of rows, for
// B200 / sm_100a.
//
// Operation: as the prefill of packed sequences, q_offset_s = S_s - T_s: query
// i of sequence s sits at position p = S_s - T_s + i and sees keys j <= p, on a
// local layer those with p - j < window; s_j = C tanh(x_j / C) (or x_j),
// out = sum_j softmax_j(s) v_j, lse = ln sum_j exp(s_j).
//
// What bounds it: every visible K and V row is read once from HBM for all the
// chunk's queries and both heads of its group; the products are small next to
// that. So the matrix products are turned round: S^T = K Q^T has the 128 keys of a
// tile as the rows M of the MMA and the chunk's rows (position, head) as its
// columns N = R = 16, 32 or 64, and O^T = V^T P^T has the d columns as M. A
// short chunk then costs no padding to 128 rows, every softmax thread owns
// one key (a TMEM lane) for R/2 rows, and K and V are each read from shared
// memory once per tile.
//
// Work split: units are (sequence, KV head, R/2 positions), each a run of
// 128-key tiles. All tiles of the launch are numbered in one line (with some empty
// places after each unit, for what its end costs) and each CTA takes an equal
// stretch of it, crossing from unit to unit without emptying
// its pipeline, so that ragged lengths and few sequences load every SM alike.
// A unit cut by a stretch's end leaves unnormalised partial results (O, max,
// sums) in the workspace, at most two per CTA, and extend_merge joins them in
// the order of the keys (no atomics: results do not depend on timing).
//
// One CTA per SM, warps in this order:
//   softmax      2 warpgroups (R = 64: 4, so that enough warps hide each other's
//                latencies), each with its R / 2 (R / 4) rows of S^T, thread =
//                key; writes P as bf16 into shared memory; at a unit's end
//                reads O^T (lane = d column) and writes out or the partial.
//   1 warp       tensor memory, one thread issues the UMMAs.
//   2 producers  K and V into a ring of 128-byte-swizzled tiles, by TMA, a box per
//                page; a box that no query sees is read from outside the cache, as
//                zeros. Boxes seen in part (a sequence's end, a window's
//                start), pages under 8 rows and Q come by 16-byte asynchronous
//                copies, with zeros for rows that no query sees (what the cache
//                holds there, NaN included, does not matter). Whole tiles by such
//                copies wherever one row was not seen: 64 sequences of 64 keys, d = 128,
//                pages of 16: 29.7 us against 22.3; of 150 keys and 32 tokens: 69 against 60.
//   1 warp       writes the CTA's merge record.
// Softmax: fp32, log2 domain. With the cap the prefill's fixed shift where it
// fits. Else a reference per row that is the row's maximum over its first tile
// and is only raised (and O and the sums rescaled) when a score of the row passes
// it by more than 2^8, as in the prefill: weights up to 2^8 lose nothing in fp32 or
// bf16 and leave V all but the last 2^8 of its range, and the usual tile needs
// one vote per warp and no exchange of maxima. P is rounded to bf16 for
// the product; out is normalised by the sum of the rounded weights, lse
// uses the unrounded sum.
#pragma once

#include "common.cuh"
#include "prefill_sm100.cuh"

namespace g2 {

// wait sites of the device error word, after those of the other kernels
constexpr unsigned int SITE_EX_PROD = 22;  // producers: slot or Q buffer free
constexpr unsigned int SITE_EX_MMA = 23;   // issuer: slot or weights ready
constexpr unsigned int SITE_EX_SM = 24;    // softmax: S, P buffer, O or the other warps

constexpr int EX_BN = 128;            // keys per tile
constexpr int EX_PROD_WARPS = 2;
constexpr int EX_S_BUFS = 3;          // S tiles in tensor memory
constexpr int EX_LAG = EX_S_BUFS - 1; // tiles by which V and its product follow K and S
constexpr int EX_MAX_SLOTS = 12;      // ring slots, whatever fits
constexpr int EX_MAX_SEQS = 1024;     // per-launch table in shared memory
constexpr int EX_MAX_CTAS = 160;      // partial-result slots: two per CTA
// Places that a launch's line has at most: calls whose shapes allow for more are
// refused (malformed offsets can still make more; those are cut off).
constexpr long long EX_MAX_TILES = 0x7fffffffll;
constexpr float EX_RAISE_LOG2 = PF_RESCALE_LOG2;   // see the softmax above
constexpr float EX_NO_MAX = -3.402823466e38f;      // reference of a row that saw no key yet

// Places in the line of tiles that a unit takes besides its tiles: what its
// start and end cost, in tiles (a tile's time goes with d, a unit's end much less).
// Over 54 shapes (d = 64, 128, 256; 4, 9-16, 17-32 tokens; 64 to 8,192 keys;
// with and without the cap) the times of 0, 384 / d and 768 / d to those of 512 / d
// are 1.08, 0.99 and 1.02 in the mean; 384 / d is slower for long chunks (24
// sequences of 1,000 to 16,000 keys, 17-32 tokens, d = 128, uncapped: 252 us
// against 244; d = 256, 500 to 8,192 keys: 177 against 172), 768 / d for short
// ones (4 tokens, 200 to 2,000 keys, d = 128: 72 against 69).
constexpr int ex_unit_cost(int d) { return 512 / d; }

template <int D, int R>
struct ExCfg {
    static constexpr int TQ = R / 2;                      // positions per unit
    static constexpr int UNIT_COST = ex_unit_cost(D);
    static constexpr int NWG = R == 64 ? 4 : 2;           // softmax warpgroups
    static constexpr int HC = R / NWG;                    // rows per softmax warpgroup
    static constexpr int SM_WARPS = 4 * NWG;
    static constexpr int WARP_MMA = SM_WARPS;
    static constexpr int WARP_PROD = SM_WARPS + 1;
    static constexpr int WARP_RECORD = WARP_PROD + EX_PROD_WARPS;
    static constexpr int THREADS = 32 * (WARP_RECORD + 1);  // 384 or 640
    static constexpr int SLOT_COLS = D < 128 ? D : 128;   // d columns of a slot
    static constexpr int SLOT_BYTES = EX_BN * SLOT_COLS * 2;
    static constexpr int KSL = D / SLOT_COLS;             // slots per K (or V) tile
    static constexpr int NCH = SLOT_COLS / 64;            // 64-column chunks per slot
    static constexpr int CH_BYTES = EX_BN * 128;          // 16 KB
    static constexpr int Q_BYTES = R * D * 2;
    static constexpr int QB = R == 64 ? 1 : 2;            // Q buffers (R = 64: more ring slots)
    static constexpr int P_BYTES = R * EX_BN * 2;
    // P with its rows contiguous (R = 64: a key's 64 rows are one 128-byte
    // line, which a thread writes 16 bytes at a time) or its keys (R < 64)
    static constexpr bool P_ROWS = R == 64;
    // R = 64: the sums of the rounded weights come from the tensor core, as one
    // more block of O^T whose "V" is all ones, 8 columns of tensor memory (16
    // registers and a fifth of the weights' instructions less per thread)
    static constexpr int ONES = R == 64 ? 1 : 0;
    static constexpr int FIXED = QB * Q_BYTES + 2 * P_BYTES;
    // rows 64..127 of the d = 64 product read one chunk past their slot: the
    // tiles after the ring must span that
    static constexpr int PAD = D == 64 && FIXED < CH_BYTES ? CH_BYTES - FIXED : 0;
    static constexpr int CUM_BYTES = 4 * (EX_MAX_SEQS + 1);
    static constexpr int CTRL_BYTES = 512 + (8 + (ONES ? 8 : 16) + 6) * R * 4;
    static constexpr int BUDGET = 227 * 1024 - 1024 - FIXED - PAD - CUM_BYTES - CTRL_BYTES - 64;
    static constexpr int NS_FIT = BUDGET / SLOT_BYTES;
    static constexpr int NS = NS_FIT > EX_MAX_SLOTS ? EX_MAX_SLOTS : NS_FIT;
    static constexpr int SMEM_BYTES =
        1024 + NS * SLOT_BYTES + FIXED + PAD + CUM_BYTES + CTRL_BYTES + 64;
    static constexpr int O_BLOCKS = D <= 128 ? 1 : D / 128;  // M = 128 blocks of O^T
    static constexpr int O_COL = EX_S_BUFS * R;
    static constexpr int ONES_COL = O_COL + (O_BLOCKS + ONES) * R;
    static constexpr int TMEM_USED = ONES_COL + 8 * ONES;
    static constexpr int TMEM_COLS =
        TMEM_USED <= 64 ? 64 : (TMEM_USED <= 128 ? 128 : (TMEM_USED <= 256 ? 256 : 512));
    static_assert(NS >= 2 * KSL && SMEM_BYTES <= 227 * 1024 && TMEM_USED <= 512, "budget");
};

struct ExParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* out;
    float* lse;
    const int* cu_q;
    const int* table;
    const int* lens;
    float* ws_o;     // [2 * EX_MAX_CTAS][R][D]
    float* ws_s;     // [2 * EX_MAX_CTAS][R][4]: reference, fp32 sum, sum of rounded weights, -
    int4* ws_rec;    // [EX_MAX_CTAS][2]: merge records
    int num_seqs, total_q, num_blocks, block_shift, max_blocks;
    int H, Hkv, window;
    float k_exp, cap_l2, scale_l2, fixed_ref;
    float series[4];     // capped score in log2 units = x (s0 + s1 x^2 + s2 x^4 + s3 x^6)
    float series_max;    // for |x| up to this (|x / C| <= 1/4)
    int has_cap;
    int box_rows;    // rows of a TMA box: min(page, 128), a unit's tiles start at multiples of it
    int use_tma;     // pages of at least 8 rows (a swizzle atom)
    unsigned long long timeout_ns;
};

// A unit and its stretch of the line of tiles.
struct ExUnit {
    int seq, g, t0;      // first query row of the unit within its sequence
    int T, L, q0;        // the sequence's queries and keys, packed row of its first query
    int tvalid;          // the unit's query rows (1 .. TQ)
    int qrow;            // packed row of query t0
    int p0;              // position of query t0
    int lo, hi;          // visible keys [lo, hi) of the whole unit
    int base;            // first key of tile 0
    int tiles;
    long long first;     // number of its first tile in the line
};

__device__ __forceinline__ int ex_len(const ExParams& P, int s) {
    const long long cap = static_cast<long long>(P.max_blocks) << P.block_shift;
    return static_cast<int>(max(0ll, min(static_cast<long long>(P.lens[s]), cap)));
}

// Visible keys and tiles (at least one, so that every unit writes its rows) of
// positions p0 .. p0 + n - 1 of a sequence of length L. Tile 0 starts at the box
// that holds the first visible key.
__device__ __forceinline__ int ex_range(const ExParams& P, int p0, int n, int L, int& lo, int& hi) {
    // (compared first: p0 - window wraps round for the largest windows and p0 < 0)
    lo = P.window > 0 && p0 >= P.window ? p0 - P.window + 1 : 0;
    hi = min(max(0, p0 + n), L);
    return max(1, (hi - (lo & -P.box_rows) + EX_BN - 1) / EX_BN);
}

template <int TQ, int COST>
__device__ __forceinline__ long long ex_seq_tiles(const ExParams& P, int s) {
    int qb, T;
    pf_seq_rows(P.cu_q, s, P.total_q, &qb, &T);
    const int L = ex_len(P, s);
    long long n = 0;
    for (int t = 0; t < T; t += TQ) {
        int lo, hi;
        n += COST + ex_range(P, L - T + t, min(TQ, T - t), L, lo, hi);
    }
    return n * P.Hkv;
}

// cum[s] = places before sequence s, cum[num_seqs] = all. Whole CTA.
template <int TQ, int COST>
__device__ __forceinline__ void ex_cum(const ExParams& P, unsigned int* cum) {
    for (int s = threadIdx.x; s < P.num_seqs; s += blockDim.x)
        cum[s + 1] = static_cast<unsigned int>(min(ex_seq_tiles<TQ, COST>(P, s), EX_MAX_TILES));
    if (threadIdx.x == 0) cum[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        long long base = 0;
        for (int b = 1; b <= P.num_seqs; b += 32) {
            const int i = b + threadIdx.x;
            long long x = i <= P.num_seqs ? cum[i] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (static_cast<int>(threadIdx.x) >= o) x += y;
            }
            x = min(x + base, EX_MAX_TILES);
            if (i <= P.num_seqs) cum[i] = static_cast<unsigned int>(x);
            base = __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
}

// CTAs that take part: every one of them gets at least one place (more than one,
// fewer CTAs, measured slower on short caches and no different on long ones).
__device__ __forceinline__ long long ex_ctas(long long all, int grid) {
    return all < grid ? all : grid;
}

// First place of CTA c's stretch, and the CTA that has a place.
__device__ __forceinline__ long long ex_start(long long c, long long all, long long ctas) {
    return c * all / ctas;
}
__device__ __forceinline__ long long ex_owner(long long tile, long long all, long long ctas) {
    return ((tile + 1) * ctas - 1) / all;
}

__device__ __forceinline__ void ex_load_seq(const ExParams& P, int s, ExUnit& U) {
    U.seq = s;
    pf_seq_rows(P.cu_q, s, P.total_q, &U.q0, &U.T);
    U.L = ex_len(P, s);
}

// The rest of U from seq, g and t0.
template <int TQ>
__device__ __forceinline__ void ex_fill_unit(const ExParams& P, ExUnit& U) {
    U.tvalid = min(TQ, U.T - U.t0);
    U.p0 = U.L - U.T + U.t0;
    U.tiles = ex_range(P, U.p0, U.tvalid, U.L, U.lo, U.hi);
    U.qrow = U.q0 + U.t0;
    U.base = U.lo & -P.box_rows;
}

// The unit that holds place `x` of the line (a tile, or the empty places after
// its last one).
template <int TQ, int COST>
__device__ __forceinline__ void ex_unit(const ExParams& P, const unsigned int* cum, long long x,
                                        ExUnit& U) {
    int lo = 0, hi = P.num_seqs - 1;  // last s with cum[s] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= x) lo = mid; else hi = mid - 1;
    }
    ex_load_seq(P, lo, U);
    const unsigned int n = cum[lo + 1] - cum[lo], at = static_cast<unsigned int>(x) - cum[lo];
    const unsigned int per_g = max(1u, n / static_cast<unsigned int>(P.Hkv));
    U.g = static_cast<int>(min(at / per_g, static_cast<unsigned int>(P.Hkv) - 1));
    unsigned int rem = at - U.g * per_g;
    for (U.t0 = 0;; U.t0 += TQ) {
        ex_fill_unit<TQ>(P, U);
        if (rem < static_cast<unsigned int>(U.tiles + COST) || U.t0 + TQ >= U.T) break;
        rem -= U.tiles + COST;
    }
    U.first = x - min(rem, static_cast<unsigned int>(U.tiles + COST) - 1);
}

// Walks the tiles of a stretch [x0, x1) of the line: unit U, its tile t, of
// which [begin, end) lie in the stretch.
template <int TQ, int COST>
struct ExWalk {
    ExUnit U;
    int t, begin, end;
    bool more;
    __device__ __forceinline__ void start(const ExParams& P, const unsigned int* cum, long long x0,
                                          long long x1) {
        more = x0 < x1;
        if (!more) return;
        ex_unit<TQ, COST>(P, cum, x0, U);
        begin = t = static_cast<int>(x0 - U.first);
        end = static_cast<int>(min(static_cast<long long>(U.tiles), x1 - U.first));
        if (t >= end) next_unit(P, cum, x1);  // in the empty places
    }
    // Units follow one another by position, KV head, sequence (a search for
    // each would cost more than a short unit's tiles).
    __device__ __forceinline__ void next_unit(const ExParams& P, const unsigned int* cum,
                                              long long x1) {
        U.first += U.tiles + COST;
        more = U.first < x1;
        if (!more) return;
        U.t0 += TQ;
        if (U.t0 >= U.T) {
            U.t0 = 0;
            if (++U.g == P.Hkv) {
                U.g = 0;
                int s = U.seq + 1;
                while (s < P.num_seqs && cum[s + 1] == cum[s]) ++s;  // without queries
                more = s < P.num_seqs;
                if (!more) return;
                ex_load_seq(P, s, U);
            }
        }
        ex_fill_unit<TQ>(P, U);
        begin = t = 0;
        end = static_cast<int>(min(static_cast<long long>(U.tiles), x1 - U.first));
    }
};

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}\n"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
// Bytes that asynchronous copies will count on `bar` in this phase.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}
// Whether the phase of the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Arrives on `bar` once every copy this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}
// Shared-memory writes ordered before this thread (its own, or those it waited
// for at an mbarrier) come before the tensor core's reads issued after this.
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// N = 8, 16 or 32 columns of this warp's 32 TMEM lanes; waits for the data.
template <int N>
__device__ __forceinline__ void ex_tmem_ld(uint32_t a, float (&f)[N]) {
    static_assert(N == 8 || N == 16 || N == 32, "columns");
    uint32_t r[N];
    if constexpr (N == 8) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7])
            : "r"(a)
            : "memory");
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(a)
            : "memory");
    } else {
        tmem_ld32(a, r);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void ex_tmem_st(uint32_t a, const float (&f)[N]) {
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __float_as_uint(f[i]);
    if constexpr (N == 8) {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
            : "memory");
    } else if constexpr (N == 16) {
        tmem_st16(a, r);
    } else {
        tmem_st32(a, r);
    }
}

// Combines N values per lane over the 32 lanes of a warp (sum or max): halves the
// columns of a lane with every exchange, so N + log2(32 / N) - 1 shuffles in
// all. Lane l ends with column ex_col<N>(l) of the result.
template <int N, bool MAX>
__device__ __forceinline__ float ex_reduce(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = N, o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n / 2) {
                    const float send = up ? v[i] : v[i + n / 2];
                    const float keep = up ? v[i + n / 2] : v[i];
                    const float got = __shfl_xor_sync(0xffffffffu, send, o);
                    v[i] = MAX ? fmaxf(keep, got) : keep + got;
                }
            }
            n >>= 1;
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return v[0];
}
template <int N>
__device__ __forceinline__ int ex_col(int lane) {
    return N == 32 ? lane : (N == 16 ? lane >> 1 : lane >> 2);
}

// Of this lane's key and HC rows, from the products in TMEM: with the cap scores
// in log2 units, less the fixed shift; without it the products as they are.
template <int HC, bool FIX>
__device__ __forceinline__ void ex_scores(const ExParams& P, uint32_t addr, float (&p)[HC]) {
    ex_tmem_ld<HC>(addr, p);
    if (FIX || P.has_cap) {
        const float sh = FIX ? -P.fixed_ref : 0.f;
        float ax = 0.f;
#pragma unroll
        for (int c = 0; c < HC; c += 2) ax = fmax3f(ax, fabsf(p[c]), fabsf(p[c + 1]));
        if (__all_sync(0xffffffffu, ax <= P.series_max)) {
            // tanh's series, two rows per instruction
            const float2 s0 = make_float2(P.series[0], P.series[0]);
            const float2 s1 = make_float2(P.series[1], P.series[1]);
            const float2 s2 = make_float2(P.series[2], P.series[2]);
            const float2 s3 = make_float2(P.series[3], P.series[3]);
#pragma unroll
            for (int c = 0; c < HC; c += 2) {
                const float2 v = make_float2(p[c], p[c + 1]);
                const float2 v2 = mul2(v, v);
                const float2 h = fma2(v2, fma2(v2, fma2(v2, s3, s2), s1), s0);
                const float2 y = fma2(v, h, make_float2(sh, sh));
                p[c] = y.x;
                p[c + 1] = y.y;
            }
        } else {
#pragma unroll
            for (int c = 0; c < HC; ++c)
                p[c] = fmaf(-2.0f * P.cap_l2, rcp_approx(1.0f + ex2_approx(p[c] * P.k_exp)),
                            P.cap_l2 + sh);
        }
    }
}

// SM = PF_SM_FIXED or PF_SM_CAP (any running max; has_cap tells the cap).
template <int D, int R, int SM>
__global__ void __launch_bounds__(ExCfg<D, R>::THREADS, 1) extend_sm100(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
    const ExParams P) {
    using C = ExCfg<D, R>;
    constexpr int HC = C::HC;
    constexpr bool FIX = SM == PF_SM_FIXED;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* sSlots = smem;
    unsigned char* sQ = sSlots + C::NS * C::SLOT_BYTES;
    unsigned char* sP = sQ + C::QB * C::Q_BYTES;
    unsigned char* ctrl = sP + 2 * C::P_BYTES + C::PAD;
    unsigned int* cum = reinterpret_cast<unsigned int*>(ctrl);
    uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl + ((C::CUM_BYTES + 63) / 64) * 64);
    uint64_t* slot_full = bars;                       // [EX_MAX_SLOTS]
    uint64_t* slot_empty = bars + EX_MAX_SLOTS;       // [EX_MAX_SLOTS]
    uint64_t* q_empty = bars + 24;         // [2]
    uint64_t* s_full = bars + 26;          // [EX_S_BUFS]
    uint64_t* p_full = bars + 29;          // [2]
    uint64_t* p_empty = bars + 31;         // [2]
    uint64_t* o_full = bars + 33;
    uint64_t* drain = bars + 34;
    uint64_t* wg_max = bars + 35;          // [4] warpgroup exchanges
    uint64_t* wg_sum = bars + 39;          // [4]
    uint64_t* wg_vote = bars + 43;         // [4]
    // votes of the warps of a warpgroup, a byte each [tile parity][warpgroup]
    volatile unsigned char* votes = reinterpret_cast<volatile unsigned char*>(bars + 48);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(bars + 52);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 53);
    // row statistics that they exchange: maxima [exchange parity][warpgroup]
    // [warp][HC], sums [unit parity][..][..][1 or 2][HC]
    float* s_max = reinterpret_cast<float*>(bars + 54);
    float* s_sum = s_max + 8 * R;
    float* s_fac = s_sum + (C::ONES ? 8 : 16) * R;  // factors of a raise [warp][HC]
    float* s_ref = s_fac + 4 * R;   // negated references [buffer][warpgroup][HC]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t lim = P.timeout_ns;
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&slot_full[i], EX_PROD_WARPS * 32);
            mbar_init(&slot_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_empty[i], 1);
            mbar_init(&p_full[i], C::SM_WARPS * 32);
            mbar_init(&p_empty[i], 1);
        }
        for (int i = 0; i < C::NWG; ++i) {
            mbar_init(&wg_max[i], 128);
            mbar_init(&wg_vote[i], 4);
            mbar_init(&wg_sum[i], 128);
        }
        for (int i = 0; i < EX_S_BUFS; ++i) mbar_init(&s_full[i], 1);
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) {
        tmem_alloc(tmem_ptr, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    ex_cum<C::TQ, C::UNIT_COST>(P, cum);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    if constexpr (C::ONES != 0) {
        if (warp < 4) {  // bf16 ones: 16 keys (8 columns) for all 128 rows
            const float one = __uint_as_float(0x3F803F80u);
            const float v[8] = {one, one, one, one, one, one, one, one};
            ex_tmem_st<8>(tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::ONES_COL, v);
            tmem_wait_st();
        }
        // read by the issuer only after p_full, which these warps arrive on later
    }
    // the merge may be scheduled; it waits for this grid before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const long long all = cum[P.num_seqs];
    const long long ctas = ex_ctas(all, gridDim.x);
    long long x0 = 0, x1 = 0;
    if (static_cast<long long>(blockIdx.x) < ctas) {
        x0 = ex_start(blockIdx.x, all, ctas);
        x1 = ex_start(blockIdx.x + 1ll, all, ctas);
    }

    if (warp >= C::WARP_PROD && warp < C::WARP_RECORD) {
        // -------------------------------------------------------- producers
        constexpr int RW = EX_BN / EX_PROD_WARPS;  // rows of a tile per warp
        constexpr int RL = RW / 32;                // of which a lane looks up this many
        const int pw = warp - C::WARP_PROD;
        const int pt = tid - C::WARP_PROD * 32;
        uint32_t fill = 0;                         // slots filled
        bool ok = true;
        auto await = [&](uint64_t* bar, uint32_t parity) {
            ok = mbar_wait(bar, parity, abort_flag, lim, SITE_EX_PROD);
            ok = __all_sync(0xffffffffu, ok);
        };
        const long long rstride = static_cast<long long>(P.Hkv) * D;
        constexpr int LPR = C::SLOT_COLS / 8;  // lanes per row of a slot
        constexpr int RPI = 32 / LPR;          // rows per instruction
        constexpr int PER8 = 8 / RPI;          // instructions per 8 rows (the swizzle's period)
        constexpr int BATCH = 8;
        const int piece = lane % LPR;          // this lane's 16 bytes of a row
        uint32_t dst8[PER8];                   // their places in the first rows of a slot
#pragma unroll
        for (int i = 0; i < PER8; ++i) {
            const int r = i * RPI + lane / LPR;
            dst8[i] = smem_u32(sSlots) + (piece >> 3) * C::CH_BYTES + (pw * RW + r) * 128 +
                      (((piece & 7) ^ (r & 7)) << 4);
        }
        // TMA boxes of a tile (pages of at least 8 rows): a page, or 128 rows of
        // it, by 64 columns; lane b knows the row of box b.
        const int box_shift = min(P.block_shift, 7);
        const int per_chunk = EX_BN >> box_shift;
        const int box = lane & (per_chunk - 1);
        struct Tile {
            int rows[RL];  // pages under 8 rows: this lane's cache rows, -1: no query
                           // sees them; else the tile's rows [first, end) that are seen
            int row;       // first cache row of box lane mod per_chunk
            int g;         // KV head
            uint32_t parts;  // boxes that are seen in part (bits)
        };
        static_assert(RL == 2, "rows or the seen range");
        // 32 entries of the sequence's table from page `w_page` on, one per lane,
        // and the 32 after them, loaded long before they are needed: loading a
        // tile's entries when it comes up leaves most of their latency in the
        // producers' way (32 ragged sequences of 500 to 8,192 keys in pages of 16,
        // 16 KV heads, d = 128, 1-8 tokens: 218 us against 207, 9-16 tokens: 203
        // against 193; one sequence of 30,001 keys, d = 256: 32.9 against 32.4).
        int w_seq = -1, w_page = 0, w_now = 0, w_next = 0;
        auto entry_of = [&](int seq, int page) -> int {
            return page < P.max_blocks ? P.table[static_cast<size_t>(seq) * P.max_blocks + page] : 0;
        };
        const int tile_pages = max(1, EX_BN >> P.block_shift);
        auto window = [&](int seq, int page) {  // `page`: a tile's first one
            if (w_seq == seq && page >= w_page && page + tile_pages <= w_page + 32) return;
            if (w_seq == seq && page == w_page + 32) {
                w_now = w_next;
            } else {
                w_seq = seq;
                w_now = entry_of(seq, page + lane);
            }
            w_page = page;
            w_next = entry_of(seq, page + 32 + lane);
        };
        auto cache_row = [&](int entry, int key) -> int {
            return (max(0, min(entry, P.num_blocks - 1)) << P.block_shift) +
                   (key & ((1 << P.block_shift) - 1));
        };
        // Boxes that queries see whole come by TMA, and so do those that none
        // sees, from rows outside the cache, as zeros.
        auto find_tile = [&](const ExUnit& U, int t, Tile& T) {
            const int k0 = U.base + t * EX_BN;
            T.g = U.g;
            T.parts = 0;
            // pages of 1 and 2 rows: more than a window per tile
            const bool wide = P.block_shift >= 2;
            if (wide) window(U.seq, k0 >> P.block_shift);
            if (P.use_tma != 0) {
                const int key = k0 + box * P.box_rows, end = key + P.box_rows;
                const int e =
                    __shfl_sync(0xffffffffu, w_now, ((key >> P.block_shift) - w_page) & 31);
                // the usual tile (without this short cut 24 ragged sequences of 500 to
                // 8,192 keys, 17-32 tokens, d = 128, take 185 us instead of 180)
                if (k0 >= U.lo && k0 + EX_BN <= U.hi) {
                    T.row = cache_row(e, key);
                    return;
                }
                const bool none = end <= U.lo || key >= U.hi;
                const bool part = !none && (key < U.lo || end > U.hi);
                T.row = none ? -EX_BN : cache_row(e, key);
                T.parts = __ballot_sync(0xffffffffu, part && lane < per_chunk);
                T.rows[0] = U.lo - k0;
                T.rows[1] = U.hi - k0;
                return;
            }
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const int key = k0 + pw * RW + i * 32 + lane;
                const bool seen = key >= U.lo && key < U.hi;
                int e = __shfl_sync(0xffffffffu, w_now, ((key >> P.block_shift) - w_page) & 31);
                if (!wide) e = seen ? entry_of(U.seq, key >> P.block_shift) : 0;
                T.rows[i] = seen ? cache_row(e, key) : -1;
            }
        };
        auto load_tile = [&](const CUtensorMap* map, const __nv_bfloat16* cache, const Tile& T,
                             int s0) {
            const uint32_t s = fill % C::NS;
            if (fill >= static_cast<uint32_t>(C::NS)) await(&slot_empty[s], ((fill / C::NS) - 1) & 1);
            if (!ok) return;
            const uint32_t slot = s * C::SLOT_BYTES;
            const __nv_bfloat16* src0 =
                cache + static_cast<long long>(T.g) * D + s0 * C::SLOT_COLS + piece * 8;
            if (P.use_tma != 0) {
                if (pt == 0)
                    mbar_expect_tx(&slot_full[s],
                                   C::SLOT_BYTES - (__popc(T.parts) << box_shift) *
                                                       (C::SLOT_COLS * 2));
                // a 64-column chunk per warp, or every other box: a copy takes its
                // warp some 90 cycles to issue, 16 of them a slot at pages of 16
                // (the whole slot by warp 0: 64 sequences of 500 keys, 4 tokens, d = 128,
                // take 69 us instead of 57)
                const int chunk = C::NCH == 2 ? pw : 0;
                if (lane < per_chunk && ((T.parts >> lane) & 1) == 0 &&
                    (C::NCH == 2 || (lane & 1) == pw))
                    tma_load_3d(sSlots + slot + chunk * C::CH_BYTES + (lane << (box_shift + 7)), map,
                                &slot_full[s], s0 * C::SLOT_COLS + chunk * 64, T.row, T.g);
                __syncwarp();
                // the boxes at the ends of what is seen (one or two): the warps take
                // groups of 8 of their rows in turn
                for (uint32_t m = T.parts; m != 0; m &= m - 1) {
                    const int b = __ffs(m) - 1;
                    const int r0 = b << box_shift;  // the box's first row of the tile
                    const int row0 = __shfl_sync(0xffffffffu, T.row, b);
                    for (int j = pw * 8; j < P.box_rows; j += EX_PROD_WARPS * 8) {
#pragma unroll
                        for (int i = 0; i < PER8; ++i) {
                            const int in = j + i * RPI + lane / LPR, r = r0 + in;
                            const bool seen = r >= T.rows[0] && r < T.rows[1];
                            cp_async16(dst8[i] + slot + (r0 + j - pw * RW) * 128,
                                       src0 + (seen ? row0 + in : 0) * rstride, seen ? 16 : 0);
                        }
                    }
                }
            } else {
                // in batches: the exchanges of a batch overlap (one by one, their
                // latency was most of a producer's time)
#pragma unroll
                for (int i0 = 0; i0 < RW / RPI; i0 += BATCH) {
                    int row[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        row[i] = __shfl_sync(0xffffffffu, T.rows[(i0 + i) * RPI / 32],
                                             ((i0 + i) * RPI + lane / LPR) & 31);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        cp_async16(dst8[(i0 + i) % PER8] + slot + ((i0 + i) / PER8) * 1024,
                                   src0 + max(row[i], 0) * rstride, row[i] >= 0 ? 16 : 0);
                }
            }
            cp_async_arrive(&slot_full[s]);  // counts the unit's Q rows in, too
            ++fill;
        };
        auto load_q = [&](const ExUnit& U, uint32_t unit) {
            const uint32_t b = unit % C::QB;
            if (unit >= static_cast<uint32_t>(C::QB)) await(&q_empty[b], ((unit / C::QB) - 1) & 1);
            if (!ok) return;
            const uint32_t dst = smem_u32(sQ) + b * C::Q_BYTES;
            constexpr int CPR = D / 8;  // 16-byte pieces per row
            for (int e = pt; e < R * CPR; e += EX_PROD_WARPS * 32) {
                const int r = e / CPR, c = e % CPR;
                const bool in = (r >> 1) < U.tvalid;
                const int t = in ? r >> 1 : 0;
                const __nv_bfloat16* src = P.q +
                    (static_cast<size_t>(U.qrow + t) * P.H + 2 * U.g + (r & 1)) * D + c * 8;
                cp_async16(dst + (c >> 3) * (R * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), src,
                           in ? 16 : 0);
            }
        };
        // K of tile x goes before V of tile x - EX_LAG, the order of their use: V
        // then lands when its weights are ready, and no slot waits for them.
        Tile now, past[EX_LAG];
        uint32_t unit = 0;
        ExWalk<C::TQ, C::UNIT_COST> W;
        W.start(P, cum, x0, x1);
        for (int it = 0, left = EX_LAG; left > 0 && ok; ++it) {
            if (W.more) {
                const ExUnit& U = W.U;
                if (W.t == W.begin) {
                    load_q(U, unit++);
                    if (!ok) break;
                }
                find_tile(U, W.t, now);
                for (int s = 0; s < C::KSL && ok; ++s) load_tile(&map_k, P.k, now, s);
                if (++W.t == W.end) W.next_unit(P, cum, x1);
            } else {
                if (it == 0) break;  // an empty stretch
                --left;
            }
            if (it >= EX_LAG)
                for (int s = 0; s < C::KSL && ok; ++s) load_tile(&map_v, P.v, past[EX_LAG - 1], s);
#pragma unroll
            for (int i = EX_LAG - 1; i > 0; --i) past[i] = past[i - 1];
            past[0] = now;
        }
        // every copy has landed before the CTA ends, also after a wait gave up
        for (uint32_t i = 0; i < static_cast<uint32_t>(C::NS) && i < fill; ++i) {
            const uint32_t f = fill - 1 - i;
            if (!mbar_wait_drain(&slot_full[f % C::NS], (f / C::NS) & 1, lim)) break;
        }
        cp_async_wait_all();
    } else if (warp == C::WARP_RECORD) {
        // ----------------------------------------------------- merge record
        // Where this CTA's stretch starts inside a unit: the unit's rows, the
        // CTAs c0 .. c1 that work on it, and this cut's share of the joining.
        if (lane == 0) {
            int4 a = make_int4(-1, 0, 0, 0), b = make_int4(0, 0, 0, 0);
            if (x0 < x1) {
                ExUnit U;
                ex_unit<C::TQ, C::UNIT_COST>(P, cum, x0, U);
                if (U.first < x0 && x0 < U.first + U.tiles) {
                    const int c0 = static_cast<int>(ex_owner(U.first, all, ctas));
                    const int c1 = static_cast<int>(ex_owner(U.first + U.tiles - 1, all, ctas));
                    // c0's partial: its last segment, slot 1 unless also its first
                    // (c0 starts here or in the empty places before)
                    const int slot0 = ex_start(c0, all, ctas) >= U.first - C::UNIT_COST ? 0 : 1;
                    a = make_int4(U.qrow, U.g, U.tvalid, slot0);
                    b = make_int4(c0, c1, static_cast<int>(blockIdx.x) - c0 - 1, c1 - c0);
                }
            }
            P.ws_rec[2 * blockIdx.x] = a;
            P.ws_rec[2 * blockIdx.x + 1] = b;
        }
        __syncwarp();
    } else if (warp == C::WARP_MMA) {
        // ------------------------------------------------------ UMMA issuer
        // The whole warp runs the loop (its values stay in uniform registers, as
        // the instructions want them) and one elected lane issues.
        if (x0 < x1) {
            const bool leader = elect_one();
            constexpr uint32_t IDESC_S = idesc_bf16(128, R, false);
            constexpr uint32_t IDESC_O = idesc_bf16(128, R, C::P_ROWS) | (1u << 15);  // A MN-major
            constexpr uint32_t HI = sdesc_hi(1024);
            const uint32_t k_lo0 = sdesc_lo(smem_u32(sSlots), 16);
            const uint32_t v_lo0 = sdesc_lo(smem_u32(sSlots), C::CH_BYTES);  // 64-column chunks
            const uint32_t q_lo0 = sdesc_lo(smem_u32(sQ), 16);
            const uint32_t p_lo0 = sdesc_lo(smem_u32(sP), 16);
            constexpr uint32_t IDESC_1 = idesc_bf16(128, R, C::P_ROWS);  // ones: A K-major
            const uint32_t tmem_o = tmem + C::O_COL;
            uint32_t fill = 0, unit = 0;
            bool ok = true;
            // The PV product runs EX_LAG tiles behind and only needs to know the
            // first and last tile of a unit (bit i: of the tile i before this one).
            uint32_t firsts = 0, lasts = 0;
            ExWalk<C::TQ, C::UNIT_COST> W;
            W.start(P, cum, x0, x1);
            uint32_t it = 0;
            for (int left = EX_LAG; left > 0 && ok; ++it) {
                firsts <<= 1;
                lasts <<= 1;
                const bool has_s = W.more;
                if (!has_s) {
                    if (it == 0) break;  // an empty stretch
                    --left;
                } else {
                    if (W.t == W.begin) {
                        firsts |= 1;
                        ++unit;
                    }
                    if (++W.t == W.end) {
                        lasts |= 1;
                        W.next_unit(P, cum, x1);
                    }
                }
                // slots in the order of their filling: K of this tile, V of the
                // tile EX_LAG before
                const uint32_t k_fill = fill, v_fill = fill + (has_s ? C::KSL : 0);
                auto do_s = [&]() -> bool {
                    const uint32_t qb = (unit - 1) % C::QB;
                    const uint32_t q_lo = q_lo0 + qb * (C::Q_BYTES >> 4);
#pragma unroll
                    for (int s = 0; s < C::KSL; ++s) {
                        const uint32_t f = k_fill + s, slot = f % C::NS;
                        bool k = mbar_wait(&slot_full[slot], (f / C::NS) & 1, abort_flag, lim,
                                           SITE_EX_MMA);
                        k = __all_sync(0xffffffffu, k);
                        if (!k) return false;
                        fence_async_smem();
                        tc_fence_after();
                        const uint32_t a0 = k_lo0 + slot * (C::SLOT_BYTES >> 4);
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < C::SLOT_COLS / 16; ++kk)
                                umma_ss_lh(tmem + (it % EX_S_BUFS) * R,
                                           a0 + (kk / 4) * (C::CH_BYTES >> 4) + (kk % 4) * 2,
                                           q_lo + (s * C::NCH + kk / 4) * ((R * 128) >> 4) +
                                               (kk % 4) * 2,
                                           HI, IDESC_S, (s | kk) != 0);
                            umma_commit(&slot_empty[slot]);
                        }
                    }
                    if (leader) {
                        umma_commit(&s_full[it % EX_S_BUFS]);
                        if (lasts & 1) umma_commit(&q_empty[qb]);
                    }
                    return true;
                };
                const uint32_t pv = it - EX_LAG, b = pv & 1;
                auto do_pv = [&]() -> bool {
                    const bool first_v = (firsts >> EX_LAG) & 1;
                    bool k = mbar_wait(&p_full[b], (pv >> 1) & 1, abort_flag, lim, SITE_EX_MMA);
                    k = __all_sync(0xffffffffu, k);
                    if (!k) return false;
                    tc_fence_after();
                    const uint32_t p_lo = p_lo0 + b * (C::P_BYTES >> 4);
                    auto p_step = [&](int kk) -> uint32_t {
                        return C::P_ROWS ? p_lo + kk * ((16 * 128) >> 4)
                                         : p_lo + (kk / 4) * ((R * 128) >> 4) + (kk % 4) * 2;
                    };
                    if (C::ONES != 0 && leader) {
#pragma unroll
                        for (int kk = 0; kk < EX_BN / 16; ++kk)
                            umma_ts_lh(tmem_o + C::O_BLOCKS * R, tmem + C::ONES_COL, p_step(kk), HI,
                                       IDESC_1, !(first_v && kk == 0));
                    }
#pragma unroll
                    for (int s = 0; s < C::KSL; ++s) {
                        const uint32_t f = v_fill + s, slot = f % C::NS;
                        k = mbar_wait(&slot_full[slot], (f / C::NS) & 1, abort_flag, lim,
                                      SITE_EX_MMA);
                        k = __all_sync(0xffffffffu, k);
                        if (!k) return false;
                        fence_async_smem();
                        tc_fence_after();
                        const uint32_t a0 = v_lo0 + slot * (C::SLOT_BYTES >> 4);
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < EX_BN / 16; ++kk)
                                umma_ss_lh(tmem_o + s * R, a0 + kk * ((16 * 128) >> 4), p_step(kk),
                                           HI, IDESC_O, !(first_v && kk == 0));
                            umma_commit(&slot_empty[slot]);
                        }
                    }
                    if (leader) {
                        umma_commit(&p_empty[b]);
                        if ((lasts >> EX_LAG) & 1) umma_commit(o_full);
                    }
                    return true;
                };
                // Whichever is ready goes first: a unit's last product must not
                // wait for the next units' keys. (Softmax relies on the order
                // of different turns only.)
                const bool has_pv = it >= EX_LAG;
                bool pv_done = false;
                if (has_s && has_pv) {
                    const uint32_t kf = k_fill + C::KSL - 1, vf = v_fill + C::KSL - 1;
                    const uint64_t t0 = globaltimer_ns();
                    for (;;) {
                        if (__all_sync(0xffffffffu,
                                       mbar_test_wait(&slot_full[kf % C::NS], (kf / C::NS) & 1)))
                            break;
                        if (__all_sync(0xffffffffu,
                                       mbar_test_wait(&p_full[b], (pv >> 1) & 1) &&
                                           mbar_test_wait(&slot_full[vf % C::NS], (vf / C::NS) & 1))) {
                            ok = do_pv();
                            pv_done = true;
                            break;
                        }
                        // (do_s then gives up in the same way; voted, as each lane
                        // has its own timer and all must leave together)
                        if (__any_sync(0xffffffffu,
                                       *abort_flag != 0 || globaltimer_ns() - t0 > lim))
                            break;
                    }
                }
                if (ok && has_s) ok = do_s();
                if (ok && has_pv && !pv_done) ok = do_pv();
                fill = v_fill + (has_pv ? C::KSL : 0);
            }
            if (leader) {
                umma_commit(drain);
                mbar_wait_drain(drain, 0, lim);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        const int wg = warp >> 2, qd = warp & 3;
        const int key_l = (qd << 5) | lane;                  // key of the tile == TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(qd * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + wg * HC;
        const uint32_t o_addr = tmem + lane_addr + C::O_COL + wg * HC;
        // P, keys contiguous: row r, this thread's pair of keys (even, odd) is
        // one 32-bit word. Even lanes store rows c8 + 0..3, odd lanes rows c8 +
        // 4..7; a row's swizzle depends on r mod 8 only, so four addresses
        // serve every c8. Rows contiguous: the key's line, this warpgroup's
        // 16-byte pieces of it.
        const bool odd = lane & 1;
        const uint32_t p_sel = odd ? 0x3276u : 0x5410u;  // (got, own) high or (own, got) low halves
        uint32_t p_addr[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r8 = k + (odd ? 4 : 0);
            p_addr[k] = C::P_ROWS
                ? smem_u32(sP) + key_l * 128 + (((wg * HC / 8 + k) ^ (key_l & 7)) << 4)
                : (smem_u32(sP) + (key_l >> 6) * (R * 128) + (wg * HC + r8) * 128 +
                   (key_l & 62) * 2) ^ (r8 << 4);
        }
        // rows of pair c: c and c + 4 of every eight (keys contiguous), or 2c and 2c + 1
        auto pair_row = [](int c, int second) -> int {
            return C::P_ROWS ? 2 * c + second : (c >> 2) * 8 + (c & 3) + 4 * second;
        };
        bool ok = true;
        uint32_t unit = 0, raises = 0, refs = 0;
        float* neg = nullptr;  // this warpgroup's negated references
        // what turns a score into log2 units (see ex_scores)
        const float unit_l2 = P.has_cap ? 1.0f : P.scale_l2;
        uint32_t done = 0;  // tiles of the stretch's units before this one
        ExWalk<C::TQ, C::UNIT_COST> W;
        for (W.start(P, cum, x0, x1); W.more && ok; W.next_unit(P, cum, x1)) {
            const ExUnit& U = W.U;
            const int t_begin = W.begin, t_end = W.end;
            // sums of the weights of pairs of rows (see pair_row), fp32 ones and
            // the rounded ones
            float2 l32[HC / 2], lr[C::ONES ? 1 : HC / 2];
#pragma unroll
            for (int c = 0; c < HC / 2; ++c) {
                l32[c] = make_float2(0.f, 0.f);
                if constexpr (!C::ONES) lr[c] = make_float2(0.f, 0.f);
            }
            if constexpr (!FIX) {
                neg = s_ref + ((++refs & 1) * C::NWG + wg) * HC;
                // all four warps write the same; rows that only fill the unit
                // (products of 0) never ask for a raise
                if (lane < HC) neg[lane] = wg * HC + lane < 2 * U.tvalid ? -EX_NO_MAX : 0.f;
                __syncwarp();
            }
            // Scores in log2 units less their rows' references: rounded in between, as
            // the references are, so that a row's largest score comes to 0 exactly
            // whatever its size (fused, a score of 2^31 would be off by 2^6).
            auto shift = [&](float (&x)[HC]) {
#pragma unroll
                for (int c = 0; c < HC; c += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(neg + c);
                    const float2 by = make_float2(unit_l2, unit_l2);
                    const float2 u =
                        add2(mul2(make_float2(x[c], x[c + 1]), by), make_float2(f.x, f.y));
                    const float2 v =
                        add2(mul2(make_float2(x[c + 2], x[c + 3]), by), make_float2(f.z, f.w));
                    x[c] = u.x;
                    x[c + 1] = u.y;
                    x[c + 2] = v.x;
                    x[c + 3] = v.y;
                }
            };
            // Waits for a tile's scores and reads them; with a running reference
            // also shifts them by it and votes on raising it: whether a score
            // (also of a key that its row does not see, which errs on the safe
            // side) passes its row's reference by too much. A segment's first tile
            // sets the references: its scores stay as they are.
            float next[HC];
            auto peek = [&](bool first, uint32_t it) -> bool {
                const uint32_t sb = it % EX_S_BUFS;
                bool k = mbar_wait(&s_full[sb], (it / EX_S_BUFS) & 1, abort_flag, lim, SITE_EX_SM);
                k = __all_sync(0xffffffffu, k);
                if (!k) return false;
                tc_fence_after();
                ex_scores<HC, FIX>(P, s_addr + sb * R, next);
                if constexpr (!FIX) {
                    bool raise = true;
                    if (!first) {
                        shift(next);
                        float top = next[0];
#pragma unroll
                        for (int c = 1; c + 1 < HC; c += 2) top = fmax3f(top, next[c], next[c + 1]);
                        raise = __any_sync(0xffffffffu, fmaxf(top, next[HC - 1]) > EX_RAISE_LOG2);
                    }
                    if (lane == 0) {
                        votes[((it & 1) * C::NWG + wg) * 4 + qd] = raise;
                        mbar_arrive(&wg_vote[wg]);
                    }
                }
                return true;
            };
            // Scores that a row does not see, in the tiles where there are any.
            auto mask = [&](int t, float (&p)[HC]) {
                const int k0 = U.base + t * EX_BN, key = k0 + key_l;
                // an inner tile is seen whole by every row
                if (k0 + EX_BN - 1 <= U.p0 && k0 + EX_BN <= U.hi &&
                    (P.window == 0 || U.p0 + U.tvalid - 1 - k0 < P.window))
                    return;
#pragma unroll
                for (int c = 0; c < HC; ++c) {
                    const int pos = U.p0 + ((wg * HC + c) >> 1);
                    if (key > pos || key >= U.hi || (P.window > 0 && pos - key >= P.window))
                        p[c] = -INFINITY;
                }
            };
            ok = peek(true, done);
            for (int t = t_begin; t < t_end && ok; ++t) {
                const uint32_t it = done + (t - t_begin);
                const uint32_t b = it & 1;
                if constexpr (!FIX) {
                    ok = mbar_wait(&wg_vote[wg], it & 1, abort_flag, lim, SITE_EX_SM);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // the same decision in the whole warpgroup
                    if (*reinterpret_cast<volatile uint32_t*>(votes + (b * C::NWG + wg) * 4) != 0) {
                        float* st = s_max + ((raises & 1) * C::NWG + wg) * 4 * HC;
                        // without the shift
                        if (t > t_begin) ex_scores<HC, FIX>(P, s_addr + (it % EX_S_BUFS) * R, next);
                        {
                            float mx[HC];
#pragma unroll
                            for (int c = 0; c < HC; ++c) mx[c] = next[c] * unit_l2;
                            mask(t, mx);
                            const float w = ex_reduce<HC, true>(mx);
                            if ((lane & (32 / HC - 1)) == 0) st[qd * HC + ex_col<HC>(lane)] = w;
                        }
                        mbar_arrive(&wg_max[wg]);
                        ok = mbar_wait(&wg_max[wg], raises & 1, abort_flag, lim, SITE_EX_SM);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        ++raises;
                        // new references into the other buffer (the other warps
                        // may still read this one), and the factors of what was
                        // summed so far (0 where nothing was)
                        float* to = s_ref + ((++refs & 1) * C::NWG + wg) * HC;
                        float* fac = s_fac + warp * HC;
                        if (lane < HC) {
                            const float m = -neg[lane];
                            const float n = fmaxf(fmaxf(m, st[lane]),
                                                  fmax3f(st[HC + lane], st[2 * HC + lane],
                                                         st[3 * HC + lane]));
                            to[lane] = -n;
                            fac[lane] = ex2_approx(m - n);
                        }
                        neg = to;
                        __syncwarp();
                        shift(next);
#pragma unroll
                        for (int c = 0; c < HC / 2; ++c) {
                            const float fx = fac[pair_row(c, 0)], fy = fac[pair_row(c, 1)];
                            l32[c].x *= fx;
                            l32[c].y *= fy;
                            if constexpr (!C::ONES) {
                                lr[c].x *= fx;
                                lr[c].y *= fy;
                            }
                        }
                        if (t > t_begin) {  // O must hold every tile before this
                            const uint32_t pv = it - 1;
                            ok = mbar_wait(&p_empty[pv & 1], (pv >> 1) & 1, abort_flag, lim,
                                           SITE_EX_SM);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int o = 0; o < C::O_BLOCKS + C::ONES; ++o) {
#pragma unroll
                                for (int c8 = 0; c8 < HC; c8 += 8) {
                                    float a[8];
                                    ex_tmem_ld<8>(o_addr + o * R + c8, a);
#pragma unroll
                                    for (int c = 0; c < 8; ++c) a[c] *= fac[c8 + c];
                                    ex_tmem_st<8>(o_addr + o * R + c8, a);
                                }
                            }
                            tmem_wait_st();
                        }
                        __syncwarp();  // fac is read before the next raise writes it
                    }
                }
                float p[HC];
#pragma unroll
                for (int c = 0; c < HC; ++c) p[c] = next[c];
                mask(t, p);
                // the next tile's scores (and vote) while this one's weights go out
                if (t + 1 < t_end) {
                    ok = peek(false, it + 1);
                    if (!ok) break;
                }
#pragma unroll
                for (int c = 0; c < HC; ++c) p[c] = ex2_approx(p[c]);
                // The P buffer is free once the product of tile it - 2 has read it.
                // S of tile it + 1 was issued after that product, so where it
                // was awaited above its completion counted that in.
                const uint32_t p_buf = b * C::P_BYTES;
                if (t + 1 >= t_end && it >= 2) {
                    ok = mbar_wait(&p_empty[b], ((it >> 1) - 1) & 1, abort_flag, lim, SITE_EX_SM);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
#pragma unroll
                for (int c8 = 0; c8 < HC; c8 += 8) {
                    uint32_t line[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // the pair of rows that share a word or an exchange
                        const int c = c8 + (C::P_ROWS ? 2 * k : k), d = C::P_ROWS ? 1 : 4;
                        const int i = c8 / 2 + k;
                        const uint32_t own = pack_bf16x2(p[c], p[c + d]);
                        l32[i] = add2(l32[i], make_float2(p[c], p[c + d]));
                        if constexpr (!C::ONES) lr[i] = add_bf16x2_f32(lr[i], own);
                        if constexpr (C::P_ROWS) {
                            line[k] = own;
                        } else {
                            // lanes 2j, 2j+1 swap halves and store the key pair of
                            // one row each (a warp's store hits every bank once)
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, own, 1);
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(
                                             p_addr[k] + p_buf + c8 * 128),
                                         "r"(__byte_perm(own, got, p_sel))
                                         : "memory");
                        }
                    }
                    if constexpr (C::P_ROWS)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         p_addr[c8 / 8] + p_buf),
                                     "r"(line[0]), "r"(line[1]), "r"(line[2]), "r"(line[3])
                                     : "memory");
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[b]);
            }
            if (!ok) break;
            // row sums over the 128 keys' threads
            constexpr int NSUM = C::ONES ? 1 : 2;
            float* ssum = s_sum + ((unit & 1) * C::NWG + wg) * 4 * NSUM * HC;
            {
                float v[HC];
#pragma unroll
                for (int c = 0; c < HC / 2; ++c) {
                    v[pair_row(c, 0)] = l32[c].x;
                    v[pair_row(c, 1)] = l32[c].y;
                }
                const float a = ex_reduce<HC, false>(v);
                float r = 0.f;
                if constexpr (!C::ONES) {
#pragma unroll
                    for (int c = 0; c < HC / 2; ++c) {
                        v[pair_row(c, 0)] = lr[c].x;
                        v[pair_row(c, 1)] = lr[c].y;
                    }
                    r = ex_reduce<HC, false>(v);
                }
                if ((lane & (32 / HC - 1)) == 0) {
                    ssum[qd * NSUM * HC + ex_col<HC>(lane)] = a;
                    if constexpr (!C::ONES) ssum[(qd * NSUM + 1) * HC + ex_col<HC>(lane)] = r;
                }
                mbar_arrive(&wg_sum[wg]);
                ok = mbar_wait(&wg_sum[wg], unit & 1, abort_flag, lim, SITE_EX_SM);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            ok = mbar_wait(o_full, unit & 1, abort_flag, lim, SITE_EX_SM);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            float lsum[HC];  // sums of the rounded weights
            if constexpr (C::ONES != 0) {
                ex_tmem_ld<HC>(o_addr + C::O_BLOCKS * R, lsum);
            } else {
#pragma unroll
                for (int c = 0; c < HC; c += 4) {
                    float4 l = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float4 x =
                            *reinterpret_cast<const float4*>(ssum + (w * NSUM + 1) * HC + c);
                        l = make_float4(l.x + x.x, l.y + x.y, l.z + x.z, l.w + x.w);
                    }
                    lsum[c] = l.x;
                    lsum[c + 1] = l.y;
                    lsum[c + 2] = l.z;
                    lsum[c + 3] = l.w;
                }
            }
            const bool whole = t_begin == 0 && t_end == U.tiles;
            // a stretch's first segment has slot 0, its last one slot 1
            const size_t ws = static_cast<size_t>(blockIdx.x) * 2 + (unit == 0 ? 0 : 1);
            const int rows = 2 * U.tvalid;
            const long long pair = static_cast<long long>(P.H) * D;  // the two heads of a position
            __nv_bfloat16* out0 = P.out + (static_cast<size_t>(U.qrow) * P.H + 2 * U.g) * D;
#pragma unroll
            for (int o = 0; o < C::O_BLOCKS; ++o) {
                float a[HC];
                ex_tmem_ld<HC>(o_addr + o * R, a);
                const int dcol = o * 128 + key_l;
                if (D < 128 && key_l >= D) continue;
                if (whole) {
                    __nv_bfloat16* to = out0 + (wg * HC / 2) * pair + dcol;
#pragma unroll
                    for (int c = 0; c < HC; c += 2, to += pair) {
                        if (wg * HC + c >= rows) break;  // (rows is even)
                        // A query before the first key sees none, every other one
                        // its own position: the sums do not decide that, as those
                        // of a NaN must stay NaN.
                        const bool sees = U.p0 + ((wg * HC + c) >> 1) >= 0;
                        to[0] = __float2bfloat16_rn(sees ? a[c] * rcp_approx(lsum[c]) : 0.f);
                        to[D] =
                            __float2bfloat16_rn(sees ? a[c + 1] * rcp_approx(lsum[c + 1]) : 0.f);
                    }
                } else {
                    float* to = P.ws_o + (ws * R + wg * HC) * D + dcol;
#pragma unroll
                    for (int c = 0; c < HC; ++c)
                        if (wg * HC + c < rows) to[c * D] = a[c];
                }
            }
            if (key_l < HC && wg * HC + key_l < rows) {
                const int r = wg * HC + key_l;
                float a = 0.f, l = 0.f, mm = FIX ? P.fixed_ref : EX_NO_MAX;
#pragma unroll
                for (int w = 0; w < 4; ++w) a += ssum[w * NSUM * HC + key_l];
#pragma unroll
                for (int c = 0; c < HC; ++c)
                    if (c == key_l) l = lsum[c];
                if constexpr (!FIX) mm = -neg[key_l];
                if (!whole) {
                    float* s = P.ws_s + (ws * R + r) * 4;
                    s[0] = mm;
                    s[1] = a;
                    s[2] = l;
                } else if (P.lse != nullptr) {
                    P.lse[static_cast<size_t>(2 * U.g + (r & 1)) * P.total_q + U.qrow + (r >> 1)] =
                        U.p0 + (r >> 1) >= 0 ? (mm + log2f(a)) * 0.69314718055994531f : -INFINITY;
                }
            }
            tc_fence_before();
            done += t_end - t_begin;
            ++unit;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::WARP_MMA) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Joins the partial results of units that more than one CTA worked on. Where
// the stretch of CTA blockIdx.x + 1 starts inside a unit, that CTA's record
// says which partials the unit has; the cuts of a unit share its rows (at d =
// 256, halves of rows): M = max m_i,
//   out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i
template <int D, int R>
__global__ void __launch_bounds__(256) extend_merge(const ExParams P) {
    constexpr int VW = D == 64 ? 2 : 4;           // columns per lane
    constexpr int BLK = D / (32 * VW);            // column blocks of a row
    constexpr int AHEAD = 4;                      // partials loaded ahead of the weights
    __shared__ float weight[8][EX_MAX_CTAS];
    __shared__ float part[8][32 * VW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 ra = P.ws_rec[2 * (blockIdx.x + 1)], rb = P.ws_rec[2 * (blockIdx.x + 1) + 1];
    if (ra.x < 0) return;
    const int qrow0 = ra.x, g = ra.y, rows = 2 * ra.z;
    const int c0 = rb.x, parts = rb.y - rb.x + 1, share = rb.z, shares = rb.w;
    // Few partials: a warp per row. Many (one long sequence): 8 warps share
    // the partials of a row, so that the loads of all of them are in flight.
    const int team = parts <= AHEAD ? 1 : (parts <= 2 * AHEAD ? 2 : (parts <= 4 * AHEAD ? 4 : 8));
    const int member = warp % team, teams = 8 / team;
    float* w = weight[warp];
    // partial i is slot 0 of CTA c0 + i, but for c0's own
    auto slot = [&](int i) -> size_t {
        return static_cast<size_t>(c0 + i) * 2 + (i == 0 ? ra.w : 0);
    };
    auto load = [&](int i, int r, int col, float (&v)[VW]) {
        const float* o = P.ws_o + (slot(i) * R + r) * D + col;
        if constexpr (VW == 4)
            *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
        else
            *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
    };
    // the whole CTA takes the same number of turns (there is a barrier inside)
    for (int e0 = share * teams; e0 < rows * BLK; e0 += shares * teams) {
        const int e = e0 + warp / team;
        const bool on = e < rows * BLK;
        const int r = on ? e / BLK : 0, col = (on ? e % BLK : 0) * 32 * VW + lane * VW;
        float v[AHEAD][VW];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (member + k * team < parts) load(member + k * team, r, col, v[k]);
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) {
            w[i] = P.ws_s[(slot(i) * R + r) * 4];
            M = fmaxf(M, w[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float a = 0.f, l = 0.f;
        for (int i = lane; i < parts; i += 32) {
            const float* st = P.ws_s + (slot(i) * R + r) * 4;
            w[i] = ex2_approx(w[i] - M);
            a = fmaf(w[i], st[1], a);
            l = fmaf(w[i], st[2], l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            l += __shfl_xor_sync(0xffffffffu, l, o);
        }
        __syncwarp();
        float acc[VW];
#pragma unroll
        for (int k = 0; k < VW; ++k) acc[k] = 0.f;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (member + k * team < parts) {
#pragma unroll
                for (int c = 0; c < VW; ++c) acc[c] = fmaf(w[member + k * team], v[k][c], acc[c]);
            }
        }
#pragma unroll 4
        for (int i = member + AHEAD * team; i < parts; i += team) {
            float u[VW];
            load(i, r, col, u);
#pragma unroll
            for (int c = 0; c < VW; ++c) acc[c] = fmaf(w[i], u[c], acc[c]);
        }
        if (team > 1) {  // in the order of the members
#pragma unroll
            for (int c = 0; c < VW; ++c) part[warp][c * 32 + lane] = acc[c];
            __syncthreads();
            if (member == 0) {
                for (int k = 1; k < team; ++k) {
#pragma unroll
                    for (int c = 0; c < VW; ++c) acc[c] += part[warp + k][c * 32 + lane];
                }
            }
            __syncthreads();
        } else {
            __syncwarp();  // w is written anew for the next row
        }
        if (!on || member != 0) continue;
        // (a unit with a query before the first key has one tile: none is cut, and
        // every row here sees a key)
        const float inv = 1.0f / l;
        const int qrow = qrow0 + (r >> 1), h = 2 * g + (r & 1);
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            P.out + (static_cast<size_t>(qrow) * P.H + h) * D + col);
#pragma unroll
        for (int k = 0; k < VW / 2; ++k)
            dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
        if (e % BLK == 0 && lane == 0 && P.lse != nullptr)
            P.lse[static_cast<size_t>(h) * P.total_q + qrow] =
                (M + log2f(a)) * 0.69314718055994531f;
    }
}

}  // namespace g2
