// pages.cuh -- management of the pages (blocks) of a paged KV cache on the
// device, for B200 / sm_100a: reserve, give back, fork, compact, copy.
//
// State: ref_counts[page] = number of block-table entries that name the page
// (0: free), block_table[seq][col] = page of rows col*bs .. of the sequence
// (-1 behind the last), seq_lens[seq]. Fresh pages are always the free ones of
// lowest index, handed out in sequence order, and counts change by integer
// additions only, so every result is determined by the inputs whatever the
// order of the threads.
//
// The bookkeeping is bound by latency: pages_assign and pages_plan run on one
// CTA of 1024 threads that ranks the free pages by block scans (16 pages per
// thread and step) and, where only the first few are wanted, stops at the step that has them.
#pragma once

#include "common.cuh"

namespace g2 {

constexpr int PG_THREADS = 1024;
constexpr int PG_PER = 16;                       // pages per thread and scan step
constexpr int PG_STEP = PG_THREADS * PG_PER;
constexpr int PG_REFUSED = -1;
constexpr int PG_BASES = 2048;                   // sequences whose ranks stay in shared memory
constexpr int PG_MAX_CACHES = 128;               // cache pointers per copy launch
constexpr int PG_COPY_THREADS = 256;
constexpr int PG_COPY_UNROLL = 8;                // 16-byte vectors in flight per thread
constexpr int PG_COPY_CHUNK = PG_COPY_THREADS * PG_COPY_UNROLL * 16;

struct PagesParams {
    int* table;            // grow, truncate, compact: in place; fork: the new table
    const int* table_in;   // fork
    int* lens;             // grow, truncate: in place; fork: the new lengths
    const int* lens_in;    // fork
    int* refs;
    const int* arg;        // grow: rows to add; truncate: rows to keep; fork: parents
    int* granted;          // grow, fork
    int* src;              // fork, compact, grow (may be NULL): pages to copy (-1: none)
    int* dst;
    int* num_live;         // compact
    int* ws_base;          // [num_seqs] rank of a sequence's first fresh page (past PG_BASES)
    int* ws_need;          // [num_seqs] fresh pages it asks for (past PG_BASES)
    int* ws_pages;         // [num_blocks] fresh pages by rank; compact: new page of a moved one
    int num_seqs, num_blocks, block_shift, max_blocks;
};

// Exclusive prefix of v over the CTA (1024 threads) and the total. `red` holds
// 33 values of shared memory; ends with a barrier after its last use.
template <typename T>
__device__ __forceinline__ T pg_scan(T v, T* red, T& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const T w = red[lane];
        T s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        red[lane] = s - w;
        if (lane == 31) red[32] = s;
    }
    __syncthreads();
    const T r = red[warp] + x - v;
    total = red[32];
    __syncthreads();
    return r;
}

// Bit j: page first + j exists and is free (free_ true) or in use (false).
__device__ __forceinline__ unsigned int pg_bits(const int* refs, int n, long long first, bool free_) {
    unsigned int m = 0;
    if (first + PG_PER <= n) {  // refs is 16-byte aligned and first a multiple of 16
        const int4* p = reinterpret_cast<const int4*>(refs + first);
        int4 v[PG_PER / 4];
#pragma unroll
        for (int j = 0; j < PG_PER / 4; ++j) v[j] = p[j];
#pragma unroll
        for (int j = 0; j < PG_PER / 4; ++j) {
            m |= static_cast<unsigned int>((v[j].x == 0) == free_) << (4 * j);
            m |= static_cast<unsigned int>((v[j].y == 0) == free_) << (4 * j + 1);
            m |= static_cast<unsigned int>((v[j].z == 0) == free_) << (4 * j + 2);
            m |= static_cast<unsigned int>((v[j].w == 0) == free_) << (4 * j + 3);
        }
    } else {
        for (int j = 0; j < PG_PER; ++j)
            if (first + j < n) m |= static_cast<unsigned int>((refs[first + j] == 0) == free_) << j;
    }
    return m;
}

__device__ __forceinline__ long long pg_pages(long long rows, int shift) {
    return (rows + (1ll << shift) - 1) >> shift;
}

__device__ __forceinline__ int pg_len(const PagesParams& P, const int* lens, int s) {
    return static_cast<int>(max(0ll, min(static_cast<long long>(lens[s]),
                                         static_cast<long long>(P.max_blocks) << P.block_shift)));
}

// Fresh pages that sequence s asks for; PG_REFUSED when the request cannot be
// met whatever is free (it then counts as none). Grow: a partly filled last page
// that other sequences share is replaced by a copy, one page more.
template <bool FORK>
__device__ __forceinline__ int pg_need(const PagesParams& P, int s) {
    if constexpr (FORK) {
        const int p = P.arg[s];
        if (p < 0 || p >= P.num_seqs || p == s) return 0;
        return (pg_len(P, P.lens_in, p) & ((1 << P.block_shift) - 1)) != 0;
    } else {
        const int add = max(0, P.arg[s]);
        const long long old = pg_len(P, P.lens, s);
        const long long have = pg_pages(old, P.block_shift);
        const long long want = pg_pages(old + add, P.block_shift);
        if (want > P.max_blocks) return PG_REFUSED;
        int need = static_cast<int>(want - have);
        if (add > 0 && (old & ((1 << P.block_shift) - 1)) != 0) {
            const int last = P.table[static_cast<size_t>(s) * P.max_blocks + have - 1];
            if (last >= 0 && last < P.num_blocks && P.refs[last] > 1) {
                if (P.src == nullptr) return PG_REFUSED;
                ++need;
            }
        }
        return need;
    }
}

// One CTA: ranks the requests, finds the free pages of lowest index and grants
// every request that its rank leaves room for. Grow: writes the new entries,
// counts and lengths. Fork: leaves the fresh page of each sequence in dst (-1:
// none).
template <bool FORK>
__global__ void __launch_bounds__(PG_THREADS) pages_assign(const PagesParams P) {
    __shared__ int red[33];
    __shared__ long long red64[33];
    __shared__ int s_base[PG_BASES], s_need[PG_BASES];
    const int tid = threadIdx.x;
    auto base_of = [&](int s) -> int& { return s < PG_BASES ? s_base[s] : P.ws_base[s]; };
    auto need_of = [&](int s) -> int& { return s < PG_BASES ? s_need[s] : P.ws_need[s]; };
    long long wanted = 0;  // requests can exceed 32 bits in sum
    for (int b = 0; b < P.num_seqs; b += PG_THREADS) {
        const int s = b + tid;
        const int need = s < P.num_seqs ? pg_need<FORK>(P, s) : 0;
        long long total;
        const long long r = wanted + pg_scan(static_cast<long long>(max(0, need)), red64, total);
        // a rank that no cache has is refused below, whatever it is exactly
        if (s < P.num_seqs) {
            base_of(s) = static_cast<int>(min(r, 0x7fffffffll));
            need_of(s) = need;
        }
        wanted += total;
    }
    int found = 0;
    for (long long b = 0; b < P.num_blocks && found < wanted; b += PG_STEP) {
        const long long first = b + static_cast<long long>(tid) * PG_PER;
        unsigned int m = first < P.num_blocks ? pg_bits(P.refs, P.num_blocks, first, true) : 0;
        int total;
        int r = found + pg_scan(__popc(m), red, total);
        while (m != 0 && r < wanted) {
            P.ws_pages[r++] = static_cast<int>(first) + __ffs(m) - 1;
            m &= m - 1;
        }
        found += total;
    }
    __syncthreads();  // ws_pages and what lies past PG_BASES, written by this CTA, are read below
    auto granted = [&](int base, int need) -> bool {
        return need == 0 || (need > 0 && static_cast<long long>(base) + need <= found);
    };
    for (int s = tid; s < P.num_seqs; s += PG_THREADS) {
        const int need = need_of(s);
        const bool ok = granted(base_of(s), need);
        P.granted[s] = ok;
        if (P.src != nullptr && (FORK ? !(ok && need > 0) : true)) P.src[s] = P.dst[s] = -1;
    }
    __syncthreads();  // (a copy's pair is written over that -1)
    // one thread per fresh page: its sequence is the last one whose rank is not
    // above the page's (of equal ranks the last asks for pages, the others do not)
    const int given = static_cast<int>(min(static_cast<long long>(found), wanted));
    for (int r = tid; r < given; r += PG_THREADS) {
        int lo = 0, hi = P.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (base_of(mid) <= r) lo = mid; else hi = mid - 1;
        }
        const int first = base_of(lo), need = need_of(lo);
        if (!granted(first, need)) continue;
        const int page = P.ws_pages[r];
        if constexpr (FORK) {
            P.dst[lo] = page;
        } else {
            const long long old = pg_len(P, P.lens, lo);
            const long long have = pg_pages(old, P.block_shift);
            // rank 0 of one page more than the new rows need: the copy
            const long long want = pg_pages(old + max(0, P.arg[lo]), P.block_shift);
            const int copies = need - static_cast<int>(want - have);
            int* e = P.table + static_cast<size_t>(lo) * P.max_blocks + have - copies + (r - first);
            if (r - first < copies) {
                P.src[lo] = *e;
                P.dst[lo] = page;
                atomicSub(P.refs + *e, 1);
            }
            *e = page;
            P.refs[page] = 1;
        }
    }
    if constexpr (!FORK) {
        __syncthreads();  // the lengths are overwritten only now
        for (int s = tid; s < P.num_seqs; s += PG_THREADS)
            if (granted(base_of(s), need_of(s)))
                P.lens[s] = pg_len(P, P.lens, s) + max(0, P.arg[s]);
    }
}

// One CTA per sequence: the new row, length and counts of a fork.
__global__ void __launch_bounds__(128) pages_fork_rows(const PagesParams P) {
    const int s = blockIdx.x;
    const int p = P.arg[s];
    const bool moves = p >= 0 && p < P.num_seqs && p != s && P.granted[s] != 0;
    const int* own = P.table_in + static_cast<size_t>(s) * P.max_blocks;
    int* out = P.table + static_cast<size_t>(s) * P.max_blocks;
    if (!moves) {
        for (int c = threadIdx.x; c < P.max_blocks; c += blockDim.x) out[c] = own[c];
        if (threadIdx.x == 0) {
            P.lens[s] = P.lens_in[s];
            P.src[s] = -1;  // dst already is
        }
        return;
    }
    const int* from = P.table_in + static_cast<size_t>(p) * P.max_blocks;
    const int L = pg_len(P, P.lens_in, p);
    const int full = L >> P.block_shift;
    const int fresh = P.dst[s];
    for (int c = threadIdx.x; c < P.max_blocks; c += blockDim.x) {
        const int had = own[c];
        const int gets = c < full ? from[c] : (c == full ? fresh : -1);
        if (had >= 0 && had < P.num_blocks) atomicSub(P.refs + had, 1);
        if (gets >= 0 && gets < P.num_blocks) atomicAdd(P.refs + gets, 1);
        out[c] = gets;
    }
    if (threadIdx.x == 0) {
        P.lens[s] = L;
        P.src[s] = fresh >= 0 ? from[full] : -1;
    }
}

// One CTA per sequence: pages behind the kept rows go back.
__global__ void __launch_bounds__(128) pages_truncate_rows(const PagesParams P) {
    const int s = blockIdx.x;
    const int keep = min(pg_len(P, P.lens, s), max(0, P.arg[s]));
    int* row = P.table + static_cast<size_t>(s) * P.max_blocks;
    for (long long c = pg_pages(keep, P.block_shift) + threadIdx.x; c < P.max_blocks; c += 4 * 128) {
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) page[u] = c + 128 * u < P.max_blocks ? row[c + 128 * u] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (page[u] < 0) continue;
            if (page[u] < P.num_blocks) atomicSub(P.refs + page[u], 1);
            row[c + 128 * u] = -1;
        }
    }
    __syncthreads();  // every thread has read the old length
    if (threadIdx.x == 0) P.lens[s] = keep;
}

// One CTA: counts the live pages, then pairs the i-th live page at or above
// that count with the i-th free page below it, moves the counts and leaves the
// new page of every moved one in ws_pages.
__global__ void __launch_bounds__(PG_THREADS) pages_plan(const PagesParams P) {
    __shared__ int red[33];
    const int tid = threadIdx.x;
    int mine = 0, live;
    for (long long b = static_cast<long long>(tid) * PG_PER; b < P.num_blocks; b += PG_STEP)
        mine += __popc(pg_bits(P.refs, P.num_blocks, b, false));
    pg_scan(mine, red, live);
    if (tid == 0) *P.num_live = live;
    const int cap = P.num_blocks / 2;
    int holes = 0, moves = 0;
    for (long long b = 0; b < P.num_blocks; b += PG_STEP) {
        const long long first = b + static_cast<long long>(tid) * PG_PER;
        const bool any = first < P.num_blocks;
        // bits of pages below `live`
        const long long k = live - first;
        const unsigned int below = k <= 0 ? 0u : (k >= PG_PER ? (1u << PG_PER) - 1u : (1u << k) - 1u);
        unsigned int h = any ? pg_bits(P.refs, P.num_blocks, first, true) & below : 0u;
        unsigned int m = any ? pg_bits(P.refs, P.num_blocks, first, false) & ~below : 0u;
        int th, tm;
        int rh = holes + pg_scan(__popc(h), red, th);
        int rm = moves + pg_scan(__popc(m), red, tm);
        while (h != 0) {
            P.dst[rh++] = static_cast<int>(first) + __ffs(h) - 1;
            h &= h - 1;
        }
        while (m != 0) {
            P.src[rm++] = static_cast<int>(first) + __ffs(m) - 1;
            m &= m - 1;
        }
        holes += th;
        moves += tm;
    }
    __syncthreads();
    for (int i = tid; i < cap; i += PG_THREADS) {
        if (i >= moves) {
            P.src[i] = P.dst[i] = -1;
            continue;
        }
        const int a = P.src[i], b = P.dst[i];
        P.refs[b] = P.refs[a];
        P.refs[a] = 0;
        P.ws_pages[a] = b;
    }
}

// The block table after a compaction (entries of pages that did not move stay).
__global__ void __launch_bounds__(256) pages_remap(const PagesParams P) {
    const long long n = static_cast<long long>(P.num_seqs) * P.max_blocks;
    const int live = *P.num_live;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * 256) {
        const int page = P.table[i];
        if (page >= live && page < P.num_blocks) P.table[i] = P.ws_pages[page];
    }
}

struct PagesCopyParams {
    void* caches[PG_MAX_CACHES];
    const int* src;
    const int* dst;
    int num_pairs, num_blocks;
    int chunks;                    // CTAs per page
    unsigned long long page_vecs;  // 16-byte vectors per page
};

// One CTA copies PG_COPY_CHUNK bytes of one page of one cache: reads and
// writes every byte once, bound by HBM bandwidth.
__global__ void __launch_bounds__(PG_COPY_THREADS) pages_copy(const __grid_constant__ PagesCopyParams P) {
    const int pair = blockIdx.x / P.chunks, chunk = blockIdx.x % P.chunks;
    const int a = P.src[pair], b = P.dst[pair];
    if (a < 0 || a >= P.num_blocks || b < 0 || b >= P.num_blocks || a == b) return;
    uint4* base = static_cast<uint4*>(P.caches[blockIdx.y]);
    const uint4* from = base + a * P.page_vecs;
    uint4* to = base + b * P.page_vecs;
    unsigned long long at = static_cast<unsigned long long>(chunk) * (PG_COPY_CHUNK / 16) + threadIdx.x;
    uint4 v[PG_COPY_UNROLL];
#pragma unroll
    for (int u = 0; u < PG_COPY_UNROLL; ++u)
        if (at + u * PG_COPY_THREADS < P.page_vecs) v[u] = from[at + u * PG_COPY_THREADS];
#pragma unroll
    for (int u = 0; u < PG_COPY_UNROLL; ++u)
        if (at + u * PG_COPY_THREADS < P.page_vecs) to[at + u * PG_COPY_THREADS] = v[u];
}

}  // namespace g2
