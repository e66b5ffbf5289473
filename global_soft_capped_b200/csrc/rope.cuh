// rope.cuh -- rotary positions of q and k, on their own (forward and gradient)
// and fused with writing k and v into a KV cache, for B200 / sm_100a.
//
// Operation, for a token at position p and pair i < rot/2 of a head, with w_i
// turns per position, a = 2 pi p w_i and a factor m on the rotation:
//   y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a)
// The pair is elements (i, i + rot/2) of the head (half layout) or (2i, 2i+1)
// (interleaved); elements rot .. d-1 pass through. The gradient is the
// transposed rotation: the same with sin a negated.
//
// Angles: w_i comes as 64-bit fixed point, the fraction of a turn times 2^64,
// so p * w_i mod 2^64 is the phase with whole turns dropped exactly, for any
// 32-bit position (the table's rounding, 2^-65 turns, grows to at most 2^-34
// turns). Its top 32 bits, as a signed number, are the angle in units of pi /
// 2^31 in [-pi, pi): one conversion and one sincospif. A float product p * w
// would be off by 0.06 rad at p = 2^20.
//
// Work split: a thread owns two 16-byte vectors ("slot") of a head, the same two in
// every head of its head group, so the 8 sines and cosines of a slot are
// computed once per group and used for all its heads. A group is a launch
// parameter: fewer heads per group where there are few tokens.
#pragma once

#include "common.cuh"
#include "decode.cuh"

namespace g2 {

// Bit 2 of the sticky device error word (bits 0 and 1: a wait that gave up, a
// decode split plan that was too short): a token to be appended had no row in
// its cache and was dropped.
constexpr unsigned int DEVERR_CACHE_ROW = 4u;

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_MIN_CTAS = 6;   // 768 threads of up to 85 registers per SM
constexpr int ROPE_UNROLL = 4;     // heads in flight per thread (128 bytes of loads)
constexpr int ROPE_MAX_HEADS = 8;  // heads per thread

// What happens to the rotated k (and to v).
enum RopeMode : int {
    ROPE_PLAIN = 0,          // k_out rows, no v; positions from an array
    ROPE_TO_LINEAR = 1,      // rows of a packed cache
    ROPE_TO_RING = 2,        // slots of a ring cache
    ROPE_TO_PAGED = 3,       // rows of paged blocks
};

struct RopeParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;   // cache modes
    __nv_bfloat16* q_out;
    __nv_bfloat16* k_out;     // k_out or the K cache
    __nv_bfloat16* v_out;     // the V cache
    long long q_stride, k_stride, v_stride;  // elements between tokens
    long long qo_stride, ko_stride;          // ROPE_PLAIN
    const unsigned long long* freqs;         // [rot/2] turns per position * 2^64
    const int* positions;                    // ROPE_PLAIN
    const int* cu_q;        // cache modes; NULL: one token per sequence
    const int* cu_k;        // ROPE_TO_LINEAR
    const int* seq_lens;    // ROPE_TO_RING, ROPE_TO_PAGED: length with the new tokens
    const int* block_table; // ROPE_TO_PAGED
    int tokens, H, Hkv, rot, num_seqs, total_k;
    int ring_mask, ring_shift, block_shift, max_blocks, num_blocks;
    int heads_per_group, groups;
    float mscale, sign;     // sign: +1 forward, -1 gradient
};

// Sequence of packed token t: the last s with cu[s] <= t, or -1 when t lies
// behind the last sequence.
__device__ __forceinline__ int rope_seq(const int* cu, int num_seqs, int t) {
    if (t >= cu[num_seqs]) return -1;
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Cache row of position p of sequence s (L its length with the new tokens), or
// -1 when the token is not stored; `lost` when that is because the cache has
// no such row (a ring drops what the same chunk overwrites without loss).
template <int MODE>
__device__ __forceinline__ int rope_row(const RopeParams& P, int s, int p, int L, bool& lost) {
    int row = -1;
    lost = true;
    if (p < 0) return row;
    if constexpr (MODE == ROPE_TO_LINEAR) {
        const long long r = static_cast<long long>(P.cu_k[s]) + p;
        if (r >= 0 && r < P.total_k) row = static_cast<int>(r);
    } else if constexpr (MODE == ROPE_TO_RING) {
        if (p < L - (P.ring_mask + 1))
            lost = false;
        else
            row = (s << P.ring_shift) + (p & P.ring_mask);
    } else {
        const int col = p >> P.block_shift;
        if (col < P.max_blocks) {
            const int b = P.block_table[static_cast<size_t>(s) * P.max_blocks + col];
            if (b >= 0 && b < P.num_blocks)
                row = (b << P.block_shift) + (p & ((1 << P.block_shift) - 1));
        }
    }
    if (row >= 0) lost = false;
    return row;
}

// Streaming 16-byte load (not .nc: in place, the thread writes it later).
__device__ __forceinline__ uint4 rope_ld(const __nv_bfloat16* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

template <int D, int MODE, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_MIN_CTAS) rope_kernel(const RopeParams P) {
    constexpr int SL = D / 16;  // slots of a head
    const long long t = static_cast<long long>(blockIdx.x) * ROPE_THREADS + threadIdx.x;
    const int slot = static_cast<int>(t % SL);
    if (t / SL >= static_cast<long long>(P.tokens) * P.groups) return;
    const unsigned int unit = static_cast<unsigned int>(t / SL);  // tokens * groups fits 31 bits
    const int token = static_cast<int>(unit / static_cast<unsigned int>(P.groups));
    const int h0 = static_cast<int>(unit % static_cast<unsigned int>(P.groups)) * P.heads_per_group;
    const int HK = P.H + P.Hkv;                          // heads that turn
    const int NH = MODE == ROPE_PLAIN ? HK : HK + P.Hkv;  // with the heads of v
    const int h1 = min(NH, h0 + P.heads_per_group);

    int pos, row = -1;
    if constexpr (MODE == ROPE_PLAIN) {
        pos = P.positions[token];
    } else {
        int s = token, i = 0, T = 1;
        if (P.cu_q != nullptr) {
            s = rope_seq(P.cu_q, P.num_seqs, token);
            if (s < 0) return;  // behind the last sequence: left as it is
            i = token - P.cu_q[s];
            T = P.cu_q[s + 1] - P.cu_q[s];
        }
        int L;
        if constexpr (MODE == ROPE_TO_LINEAR)
            L = P.cu_k[s + 1] - P.cu_k[s];
        else
            L = P.seq_lens[s];
        if (P.cu_q == nullptr && L <= 0) return;  // an empty slot of the batch
        pos = L - T + i;
        bool lost;
        row = rope_row<MODE>(P, s, pos, L, lost);
        if (lost && slot == 0 && h0 == 0) atomicOr(&g_device_error, DEVERR_CACHE_ROW);
    }

    // the slot's two vectors: elements e0 .. e0+7 and e1 .. e1+7 of the head
    const bool turns = slot < P.rot / 16;
    int e0, e1;
    if (turns) {
        e0 = slot * 8;
        e1 = P.rot / 2 + slot * 8;
    } else {
        e0 = P.rot + (slot - P.rot / 16) * 8;
        e1 = e0 + (D - P.rot) / 2;
    }
    float c[8], s[8];
    if (turns && h0 < HK) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // interleaved: the two vectors hold 4 whole pairs each
            const int i = INTER ? (j < 4 ? slot * 4 + j : P.rot / 4 + slot * 4 + j - 4)
                                : slot * 8 + j;
            const unsigned long long ph = P.freqs[i] * static_cast<unsigned long long>(
                                              static_cast<long long>(pos));
            const float x = static_cast<float>(static_cast<int>(ph >> 32)) * 0x1p-31f;
            sincospif(x, &s[j], &c[j]);
            c[j] *= P.mscale;
            s[j] *= P.mscale * P.sign;
        }
    }

    for (int hb = h0; hb < h1; hb += ROPE_UNROLL) {
        uint4 a[ROPE_UNROLL], b[ROPE_UNROLL];
        __nv_bfloat16* dst[ROPE_UNROLL];
        bool same[ROPE_UNROLL];  // v heads: copied whole
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            const int h = hb + u;
            dst[u] = nullptr;
            same[u] = !turns;
            if (h >= h1) continue;
            const __nv_bfloat16* src;
            if (h < P.H) {
                src = P.q + token * P.q_stride + h * D;
                dst[u] = P.q_out + token * P.qo_stride + h * D;
            } else if (h < HK) {
                src = P.k + token * P.k_stride + (h - P.H) * D;
                if constexpr (MODE == ROPE_PLAIN)
                    dst[u] = P.k_out + token * P.ko_stride + (h - P.H) * D;
                else if (row >= 0)
                    dst[u] = P.k_out + static_cast<size_t>(row) * P.Hkv * D + (h - P.H) * D;
            } else {
                src = P.v + token * P.v_stride + (h - HK) * D;
                if (row >= 0)
                    dst[u] = P.v_out + static_cast<size_t>(row) * P.Hkv * D + (h - HK) * D;
                same[u] = true;
            }
            if (dst[u] == nullptr) continue;
            a[u] = rope_ld(src + e0);
            b[u] = rope_ld(src + e1);
        }
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            if (dst[u] == nullptr) continue;
            if (!same[u]) {
                float x[8], y[8], z[8], w[8];
                bf16x8_to_f32(a[u], x);
                bf16x8_to_f32(b[u], y);
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        z[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
                        z[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
                        w[2 * j] = y[2 * j] * c[4 + j] - y[2 * j + 1] * s[4 + j];
                        w[2 * j + 1] = y[2 * j + 1] * c[4 + j] + y[2 * j] * s[4 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        z[j] = x[j] * c[j] - y[j] * s[j];
                        w[j] = y[j] * c[j] + x[j] * s[j];
                    }
                }
                // one rounding to bf16 per element
                a[u] = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]),
                                  pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
                b[u] = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]),
                                  pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
            }
            __stcs(reinterpret_cast<uint4*>(dst[u] + e0), a[u]);
            __stcs(reinterpret_cast<uint4*>(dst[u] + e1), b[u]);
        }
    }
}

}  // namespace g2
