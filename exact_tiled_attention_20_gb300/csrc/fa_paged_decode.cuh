// fa_paged_decode.cuh -- split-KV attention of a few query tokens over the 16-bit paged cache,
// under the mask of a draft tree or of a causal window with sinks (tcgen05 + TMA).
//
// For sequence b of n keys, its query tokens being its last Sq keys, token i and query head h:
//     s_j = scale * (q . k_j),  o = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
// over the keys j that token i sees:
//     tree:    j < n - Sq, and n - Sq + t where bit t of the token's mask is set;
//     window:  j <= p = n - Sq + i, and j >= p - window_left or j < sinks.
//
// A sub-tile holds the query rows of T tokens of one kv head (row = token * group + head, at most
// 128), a row block NQ sub-tiles.  One CTA streams key tiles through shared memory for a row
// block: a TMA warp, an MMA warp (S = Q K^T with A and B from shared memory, O += P V with P from
// TMEM), and a softmax warpgroup per sub-tile, thread = row = TMEM lane, as in the forward.
//
// Why tcgen05 although few rows may be in use: an M = 128 product costs the same for 1 row as for
// 128, and that is less than the tile's way from HBM (D = 128, 128 keys: 1100 cycles of products
// against some 2800 for 64 KB at an SM's share of the bandwidth), so it is the bytes that bound
// the kernel for anything up to about 256 rows.
//
// A tile is BN keys of the sequence's visible ones, in strips of 32: the strips of the sinks, then
// those from the first token's window on.  Strips that hold no visible key are not read.
//
// Plan: a sequence's tiles are counted as units; the units of all entries (sequence, group of kv
// heads), each led by C::Lead units for what starting and finishing one costs, lie end to end
// and are cut into equal ranges.  A range is worked on by G CTAs, one for each head of the group
// (and for each row block, where there are few): they read the same keys at about the same time,
// whose rows lie side by side in a page.  A cut entry leaves a partial output and log-sum-exp in
// each range, at most two per CTA, which the merge kernel joins.
//
// Infinities and NaNs: the scores of hidden keys are replaced, not added to.  In tiles that hide a
// key from some row, V's values that are not finite are taken out before the product (0 * inf is
// NaN) and added to the rows that see them in the epilogue, from memory.
#pragma once

#include <algorithm>

#include "fa_kv8_decode.cuh"  // shared-memory loads, 16-bit conversions, prefer_shared
#include "fa_paged.cuh"

namespace fa {

// 4-D map over [dim3][dim2][dim1][dim0] in 16 bits, box (64, box1, box2, 1), 128-byte swizzle.
bool encode_paged_tmap(CUtensorMap* map, const void* base, bool bf16, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                       uint64_t dim3, uint32_t box1, uint32_t box2);

struct PagedDecParams {
    int B, Sq, Hq, Hkv, group;
    int T;               // query tokens of a sub-tile
    int row_blocks;      // of a (sequence, kv head)
    int g, rg;           // heads and row blocks of an entry: G = g * rg CTAs work on a range
    int groups, blocks;  // entries of a sequence: groups of heads, by row blocks over rg
    int merge_ctas;      // of a range and member
    int ranges, whole;   // whole: entries are not cut, a range has those that begin in it
    int capacity, page_size, num_pages, max_pages, box_rows;
    int nb_log;           // log2 of the boxes of a tile, BN / box_rows
    unsigned page_recip;  // floor(2^32 / page_size) + 1
    int window_left, sinks;
    int words;            // of a token's tree mask
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* tree;
    float scale_log2;
    const uint16_t* v_pages;
    void* o;
    float* lse;
    float* o_part;    // [G, 2 * ranges, block rows, D]
    float* lse_part;  // [G, 2 * ranges, block rows]
    int* status;
};

constexpr int kPagedMaxB = 1024;
constexpr float kPagedLn2 = 0.69314718055994531f;

template <int D_, int NQ_>
struct PagedCfg {
    static constexpr int D = D_, NQ = NQ_;
    static constexpr int NR = 0;  // rows are TMEM lanes
    static constexpr int BM = 128;
    static constexpr int BN = D == 256 ? 64 : 128;  // keys of a tile
    static constexpr int DA = (D + 63) / 64;        // 128-byte column atoms per row
    static constexpr int kQRows = BM;
    static constexpr int kQBytes = BM * DA * 128;
    static constexpr int kTileBytes = BN * DA * 128;
    // K and V tiles take turns in one ring of NB buffers.  (NB is even, so that a buffer is one producer's, or 5
    // or more: a producer that waits for a buffer knows only the parity of its uses, and must be sure that the
    // use before the last is over.  That is so where the buffer two loads back, which it has waited for, was
    // freed behind it: K of a tile is freed behind V of the tile two before.  Of 3 it is not.)  As many as fit
    // are not better: 26 drafts of 4 heads took 93.3 us with 5 and 92.1 with 4, 24 drafts at D = 64 57.2, 56.8
    // and 56.3 with 10, 8 and 6.
    static constexpr int NB = D == 64 ? 6 : 4;
    // Units charged to each entry beside its tiles, and the least units of a range, since a cut costs the
    // merge kernel.  Measured (us) with leads of 1, 2, 3, 4, 6: 64 drafts of 4 heads 107.5, 105.0,
    // 102.7, 98.4, 96.4; window steps at D = 128 53.6, 53.2, 54.2, 53.4, 54.6 and at D = 96 20.3, 19.3, 18.5,
    // 18.9, 19.2; D = 256 31.8, 31.1, 31.0, 30.6, 30.4.
    static constexpr int Lead = NQ == 1 ? 4 : 6;
    static constexpr int MinWidth = Lead + 4;
    static constexpr int kSlots = 2;  // S buffers in TMEM: two of one sub-tile, or one of each
    static constexpr int kOCol0 = kSlots * BN;
    static constexpr int kTmemCols = 512;
    static_assert(kOCol0 + NQ * D <= kTmemCols, "TMEM budget");
    static_assert(NB % 2 == 0, "two producers of one ring");
    static constexpr int kThreads = 128 * NQ + 96;
    static constexpr int kProducerWarp = 4 * NQ;  // Q and K; the next warp: V
    static constexpr int kMmaWarp = 4 * NQ + 2;
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQEmpty = kBarQFull + NQ;
    static constexpr int kBarFull = kBarQEmpty + NQ;
    static constexpr int kBarEmpty = kBarFull + NB;
    static constexpr int kBarSFull = kBarEmpty + NB;
    static constexpr int kBarPFull = kBarSFull + kSlots;
    static constexpr int kPFulls = NQ;
    static constexpr int kBarODone = kBarPFull + kPFulls;
    static constexpr int kODones = NQ;
    static constexpr int kBarODrained = kBarODone + kODones;
    static constexpr int kBarFinal = kBarODrained + NQ;
    static constexpr int kBarJoin = kBarFinal;  // (none)
    static constexpr int kNumBars = kBarFinal + 1;
    // Results leave through shared memory, OC columns of a warp's 32 rows at a time, so that lanes side by
    // side write memory side by side (a lane that wrote its own row took 32 lines for each instruction:
    // 256 rows of D = 128 8800 cycles).  Rows are 4 words more than OC apart: no bank is met twice.
    static constexpr int OC = NQ == 1 ? 32 : 16;
    static constexpr int kOutBytes = 4 * NQ * 32 * (OC + 4) * 4;
    // Offsets in shared memory.
    static constexpr int kQOff = 0, kRingOff = NQ * kQBytes, kOutOff = kRingOff + NB * kTileBytes;
    static constexpr int kBarOff = kOutOff + kOutBytes;
    static constexpr int kFixedBytes = 1024 + kBarOff + 8 * kNumBars + 32;
    static constexpr int plan_bytes(int B) { return (2 * B + 1) * 4; }
    static_assert(kFixedBytes + (2 * kPagedMaxB + 1) * 4 + 256 <= 232448, "shared memory of a CTA");
};

// Few rows, at most 16 of a (sequence, kv head): the products are turned round, S^T = K Q^T with the keys
// in TMEM's lanes and O^T = V^T P^T with the dims there.  All four softmax warps then have a share of a
// tile's scores, 32 keys of 16 rows each, where else one warp takes the 128 of each row one after the
// other, which is most of what a tile takes (1300 cycles of 1650).  P^T goes through shared memory.
// Measured (us) against rows in lanes: 64 window steps of 4 heads at D = 128 48.9 : 52.5, 13 of three
// tokens at D = 96 14.6 : 17.2, 32 of two tokens of 8 heads at D = 64 21.4 : 24.0, one sequence of 16384 keys
// 15.5 : 17.5, 32 of 4096 to 16384 keys 191 : 192.  With 32 rows there was nothing in it (28 drafts'
// rows of a short chat 7.7 : 7.4, 16 trees of 8 drafts and 4 heads 50.8 : 50.8, 24 drafts at D = 64 58.8 : 57.0),
// so that rows from 17 on stay in lanes; at D = 256 the ring would hold 3 tiles of 128 keys.
template <int D_>
struct PagedFewCfg {
    static constexpr int D = D_, NQ = 1, NR = 16;
    static constexpr int BM = 128, BN = 128;
    static constexpr int DA = (D + 63) / 64;
    static constexpr int kQRows = NR;
    static constexpr int kQBytes = NR * DA * 128;
    static constexpr int kTileBytes = BN * DA * 128;
    static constexpr int NB = D == 64 ? 6 : 5;  // (of 6 the 32 long sequences took 200 us, of 4 189 and D = 96 15.0)
    static_assert(D <= 128 && (NB % 2 == 0 || NB >= 5), "O^T has 128 lanes; two producers of one ring");
    // (With leads of 2, 3, 4, 5 the window steps took 48.9, 49.1, 48.8, 49.3, at D = 96 15.7, 14.5, 14.6, 15.2.)
    static constexpr int Lead = 3, MinWidth = Lead + 4;
    static constexpr int kSlots = 2;
    static constexpr int kOCol0 = kSlots * NR;
    static constexpr int kTmemCols = 64;
    static_assert(kOCol0 + NR <= kTmemCols, "TMEM budget");
    static constexpr int kThreads = 128 + 96;
    static constexpr int kProducerWarp = 4, kMmaWarp = 6;
    static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarFull = 2, kBarEmpty = kBarFull + NB;
    static constexpr int kBarSFull = kBarEmpty + NB, kBarPFull = kBarSFull + kSlots;
    static constexpr int kODones = 2;  // of even and odd tiles
    static constexpr int kPFulls = 2;  // too: P of a tile may be complete before the product of the tile before starts
    static constexpr int kBarODone = kBarPFull + kPFulls, kBarODrained = kBarODone + kODones;
    static constexpr int kBarFinal = kBarODrained + 1, kBarJoin = kBarFinal + 1, kNumBars = kBarJoin + 1;
    // The ring comes first: at D = 64 the second half of O^T's 128 rows is made of what lies behind a tile
    // of V, which has to be there and is not used.
    static constexpr int kRingOff = 0, kQOff = NB * kTileBytes, kPOff = kQOff + kQBytes;
    static constexpr int kPBytes = NR * 256;  // [NR rows][128 keys], as the products want it; two of them
    static constexpr int kRedOff = kPOff + 2 * kPBytes;  // floats [2][4][32], [4][32]; ints [32], [2]
    static constexpr int kOutOff = kRedOff;
    static constexpr int kBarOff = kRedOff + 2048 + (D == 64 ? 16384 : 0);
    static constexpr int kFixedBytes = 1024 + kBarOff + 8 * kNumBars + 32;
    static constexpr int plan_bytes(int B) { return (2 * B + 1) * 4; }
    static_assert(kFixedBytes + (2 * kPagedMaxB + 1) * 4 + 256 <= 232448, "shared memory of a CTA");
};

template <bool kSum>
__device__ __forceinline__ float paged_op(float a, float b) {
    return kSum ? a + b : fmaxf(a, b);
}

// Lanes n and n + 16 of the warp get the maximum, or sum, of its lanes' v[n].
template <bool kSum>
__device__ __forceinline__ float paged_transposed(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = paged_op<kSum>(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const bool upper = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = upper ? v[i] : v[i + w], keep = upper ? v[i + w] : v[i];
            v[i] = paged_op<kSum>(keep, __shfl_xor_sync(0xffffffffu, give, w));
        }
    }
    return v[0];
}

__device__ __forceinline__ int paged_len(const PagedDecParams& p, int b) {
    return min(max(__ldcg(p.kv_lens + b), 0), p.capacity);
}

// The strips of 32 keys of a sequence that may be visible: 0 .. sinks - 1 and first, first + 1, ...
struct PagedStrips {
    int sinks, first;
    // First key of strip i of the tiles; behind the last visible one it is past the sequence's keys.
    __device__ __forceinline__ int key(int i) const { return (i < sinks ? i : first + i - sinks) * 32; }
};

__device__ __forceinline__ PagedStrips paged_strips(const PagedDecParams& p, int len) {
    PagedStrips t;
    t.first = p.window_left >= 0 ? max(len - p.Sq - p.window_left, 0) / 32 : 0;
    t.sinks = min((min(p.sinks, len) + 31) / 32, t.first);
    return t;
}

template <class C>
__device__ __forceinline__ int paged_units(const PagedDecParams& p, int len) {
    if (len <= 0) return 0;
    const PagedStrips t = paged_strips(p, len);
    return (t.sinks + (len + 31) / 32 - t.first + C::BN / 32 - 1) / (C::BN / 32) + C::Lead;
}

// Units of a range, from the units of one entry of each sequence summed.
template <class C>
__device__ __forceinline__ int paged_width(const PagedDecParams& p, int sum_units) {
    const unsigned total = (unsigned)sum_units * (unsigned)(p.groups * p.blocks);
    return max((int)((total + (unsigned)p.ranges - 1u) / (unsigned)p.ranges), C::MinWidth);
}

// The pieces of an entry of `units` units from unit `start` on: the first range that holds keys of
// it, and how many ranges do.
template <class C>
__device__ __forceinline__ int paged_first_piece(int start, int w) {
    return (start + C::Lead) / w;
}
template <class C>
__device__ __forceinline__ int paged_pieces(int start, int units, int w) {
    return units > 0 ? (start + units - 1) / w - paged_first_piece<C>(start, w) + 1 : 0;
}
// The slot of an entry's piece in range r: a range has at most one piece of an entry that began
// before it, and one that goes on behind it.
__device__ __forceinline__ int paged_slot(const PagedDecParams& p, int r, bool first) {
    return first ? p.ranges + r : r;
}

struct PagedSeg {
    int b, hk, rb, len;
    int u0, u1;  // its tiles u0 .. u1 - 1
    PagedStrips strips;
    int slot;
    bool cut;
};

// Walks the segments of one range; no division but at its start.
template <class C>
struct PagedWalk {
    const int* len;     // [B]
    const int* prefix;  // [B + 1], of the units of one entry
    int x0, W, x, x_end, rng;
    int b, group, block, start, units;  // the entry that holds unit x, or ends there
    int head, sub;                      // this CTA's head of the group and row block of the entry

    __device__ __forceinline__ void init(const PagedDecParams& p, const int* len_, const int* prefix_, int rng_,
                                         int member) {
        len = len_;
        prefix = prefix_;
        rng = rng_;
        head = member & (p.g - 1);
        sub = member / p.g;
        const int entries = p.groups * p.blocks, total = prefix[p.B] * entries;
        W = paged_width<C>(p, prefix[p.B]);
        x = x0 = (int)min((long long)rng * W, (long long)total);
        x_end = (int)min((long long)x + W, (long long)total);
        if (x >= x_end) return;
        int lo = 0, hi = p.B;  // largest b with entries * prefix[b] <= x: it has keys
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (entries * prefix[mid] <= x) lo = mid; else hi = mid;
        }
        b = lo;
        units = prefix[lo + 1] - prefix[lo];
        const int e = entries == 1 ? 0 : (int)((unsigned)(x - entries * prefix[lo]) / (unsigned)units);
        start = entries * prefix[lo] + e * units;
        group = p.blocks == 1 ? e : e / p.blocks;
        block = e - group * p.blocks;
    }

    __device__ __forceinline__ bool next(const PagedDecParams& p, PagedSeg& s) {
        while (x < x_end) {
            if (x >= start + units) {
                start += units;
                if (++block == p.blocks) {
                    block = 0;
                    if (++group == p.groups) {
                        group = 0;
                        do {
                            ++b;
                            units = prefix[b + 1] - prefix[b];
                        } while (units == 0);
                    }
                }
            }
            if (p.whole && x > start) {  // the range before has it
                x = start + units;
                continue;
            }
            const int end = p.whole ? start + units : min(x_end, start + units);
            const bool first = start + C::Lead >= x0;  // its first keys are this range's
            s.b = b;
            s.hk = group * p.g + head;
            s.rb = block * p.rg + sub;
            s.len = len[b];
            s.strips = paged_strips(p, s.len);
            s.u0 = max(x - start - C::Lead, 0);
            s.u1 = end - start - C::Lead;
            s.slot = paged_slot(p, rng, first);
            s.cut = !p.whole && !(first && start + units <= x0 + W);
            x = end;
            if (s.u1 > s.u0) return true;  // else the range ends within the lead
        }
        return false;
    }
};

// Bits i of a word with a <= i <= b.
__device__ __forceinline__ uint32_t paged_bits(int a, int b) {
    a = max(a, 0);
    b = min(b, 31);
    return a > b ? 0u : (0xffffffffu >> (31 - b)) & (0xffffffffu << a);
}

// The keys that token `tok` of a sequence of `len` keys sees: lo .. hi and those before sink (of a
// tree: those before the drafts).
__device__ __forceinline__ void paged_row(const PagedDecParams& p, int len, int tok, int& lo, int& hi, int& sink) {
    const int ctx = len - p.Sq;
    hi = p.tree ? ctx - 1 : ctx + tok;
    lo = p.window_left >= 0 ? max(hi, 0) - p.window_left : 0;
    sink = min(p.sinks, hi + 1);
}

// Bit i: whether key k + i is a draft that token `tok` sees.
static __device__ __noinline__ uint32_t paged_drafts(const PagedDecParams& p, int b, int tok, int len, int k) {
    const int t = k - (len - p.Sq);  // bit i is draft t + i
    if (t <= -32 || t >= p.Sq) return 0u;
    const int32_t* m = p.tree + ((size_t)b * p.Sq + tok) * p.words;
    uint32_t d;
    if (t < 0) {
        d = (uint32_t)__ldg(m) << -t;
    } else {
        const int i = t >> 5;
        d = __funnelshift_r((uint32_t)__ldg(m + i), i + 1 < p.words ? (uint32_t)__ldg(m + i + 1) : 0u, t & 31);
    }
    return d & paged_bits(-t, len - 1 - k);
}

// The strips of a sequence's tiles that hide no key from any token: lo .. hi - 1, and the first `sinks`,
// which are all sinks.  The others are few whatever the lengths: the one that the last sinks are in, those
// where the tokens' windows begin, and those with the tokens' own keys.
struct PagedClear {
    int lo, hi, sinks;
    __device__ __forceinline__ bool has(int i) const { return (i >= lo && i < hi) || i < sinks; }
};

__device__ __forceinline__ PagedClear paged_clear(const PagedDecParams& p, int len, const PagedStrips& t) {
    const int ctx = len - p.Sq;  // keys up to ctx (of a tree: before it) are seen by all, windows aside
    PagedClear c;
    c.lo = p.window_left >= 0 ? (max(len - 1 - p.window_left, 0) + 31) / 32 - t.first + t.sinks : 0;
    c.hi = max(p.tree ? ctx : ctx + 1, 0) / 32 - t.first + t.sinks;
    c.sinks = min(t.sinks, p.sinks / 32);  // (before t.first: before the first token)
    return c;
}

// Whether one of a word's 16-bit values is an infinity or NaN.
template <bool kBF16>
__device__ __forceinline__ bool paged_nonfinite(uint32_t w) {
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    return (((w & 0x7fff7fffu) + (0x8000u - kInf) * 0x10001u) & 0x80008000u) != 0;
}

template <bool kBF16>
__device__ __forceinline__ float paged_from16(uint32_t x) {
    if constexpr (kBF16) {
        return __uint_as_float(x << 16);
    } else {
        float f;
        asm("{\n.reg .b16 a;\ncvt.u16.u32 a, %1;\ncvt.f32.f16 %0, a;\n}" : "=f"(f) : "r"(x));
        return f;
    }
}

// Sends for a tensor map's box to L2.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// Page and row within it of key `key` of sequence b; page -1: none.
__device__ __forceinline__ int2 paged_place(const PagedDecParams& p, int b, int key) {
    unsigned pi = __umulhi((unsigned)key, p.page_recip);  // the quotient, or one more
    int row = (int)((unsigned)key - pi * (unsigned)p.page_size);
    if (row < 0) {
        --pi;
        row += p.page_size;
    }
    const int page = __ldcg(p.table + (size_t)b * p.max_pages + pi);  // (past L1: it may be read before the wait)
    return make_int2(page >= 0 && page < p.num_pages ? page : -1, row);
}

// Fills len[B] and prefix[B + 1] (all threads; ends with a barrier).
template <class C, int kThreads>
__device__ __forceinline__ void paged_make_plan(const PagedDecParams& p, int* len, int* prefix, int* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            const int n = paged_len(p, b);
            len[b] = n;
            sum += prefix[b] = paged_units<C>(p, n);
        }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_sum[w];
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            const int units = prefix[b];
            prefix[b] = run;
            run += units;
        }
    }
    if (threadIdx.x == kThreads - 1) prefix[p.B] = run;
    __syncthreads();
}

// Of a tile of V, the strips that hide a key: values that are not finite give way to zeros.  128
// threads take 16 bytes each in turn; returns whether this one found any.
template <int DA, int BN, bool kBF16>
__device__ __forceinline__ bool paged_finite_v(uint32_t at, int r, const PagedClear& clear, int strip0) {
    bool odd = false;
#pragma unroll 1
    for (int ch = 0; ch < BN / 32; ++ch) {
        if (clear.has(strip0 + ch)) continue;
#pragma unroll
        for (int i = 0; i < 2 * DA; ++i) {  // 32 rows of an atom are 4096 bytes
            const uint32_t a = at + (i >> 1) * (BN * 128) + ch * 4096 + (i & 1) * 2048 + r * 16;
            uint32_t w[4];
            lds128(a, w);
            if (paged_nonfinite<kBF16>(w[0]) | paged_nonfinite<kBF16>(w[1]) | paged_nonfinite<kBF16>(w[2]) |
                paged_nonfinite<kBF16>(w[3])) {
                odd = true;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] &= (paged_nonfinite<kBF16>(w[k] & 0xffffu) ? 0u : 0xffffu) |
                            (paged_nonfinite<kBF16>(w[k] & 0xffff0000u) ? 0u : 0xffff0000u);
                st_shared_v4(a, w[0], w[1], w[2], w[3]);
            }
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    return odd;
}

// Adds V's values that were taken out of a segment's product to a row that it was written to, where
// the row's token sees them.  (An infinity or NaN is the sum that it is in, whatever its weight.)
template <int D, int BN, bool kBF16>
__device__ __noinline__ void paged_add_odd(const PagedDecParams& p, int b, int hk, int len, int tok, int u0, int u1,
                                           float* part, uint16_t* out) {
    const PagedStrips strips = paged_strips(p, len);
    const PagedClear clear = paged_clear(p, len, strips);
    int lo, hi, sink;
    paged_row(p, len, tok, lo, hi, sink);
    for (int i = u0 * (BN / 32); i < u1 * (BN / 32); ++i) {
        if (clear.has(i)) continue;
        const int k = strips.key(i);
        uint32_t sees = paged_bits(lo - k, hi - k) | paged_bits(0, sink - 1 - k);
        if (p.tree) sees |= paged_drafts(p, b, tok, len, k);
        for (int c = 0; c < 32; ++c) {
            if (!(sees >> c & 1u)) continue;
            const int2 at = paged_place(p, b, k + c);
            if (at.x < 0) continue;
            const uint16_t* v = p.v_pages + (((size_t)at.x * p.page_size + at.y) * p.Hkv + hk) * D;
            for (int d = 0; d < D; ++d) {
                const uint32_t y = v[d];
                if (!paged_nonfinite<kBF16>(y)) continue;
                if (part)
                    part[d] += paged_from16<kBF16>(y);
                else
                    out[d] = float_to16<kBF16>(paged_from16<kBF16>(out[d]) + paged_from16<kBF16>(y));
            }
        }
    }
}

template <class C, bool kBF16>
__global__ void __launch_bounds__(C::kThreads, 1)
    paged_split_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedDecParams p) {
    constexpr int D = C::D, NQ = C::NQ, NR = C::NR, BN = C::BN, DA = C::DA, NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_warp_sum[C::kThreads / 32];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t sQ = base + C::kQOff, sRing = base + C::kRingOff, sOut = base + C::kOutOff, sBar = base + C::kBarOff;
    uint32_t* tmem_slot =
        reinterpret_cast<uint32_t*>(smem_raw + (sBar - raw) + 8 * C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // Of the last segments those (counted from 1) whose V held a value that is not finite in a tile with
    // hidden keys.  Sub-tile 0 writes; it may be scanning the tile two segments ahead of the one whose flag
    // sub-tile 1 has yet to read, and no further: it needs a product behind sub-tile 1's P.
    constexpr int kOddSlots = 4;
    volatile int* odd_seg = reinterpret_cast<volatile int*>(tmem_slot + 2);
    int* plan_len = reinterpret_cast<int*>(tmem_slot + 8);
    int* plan_prefix = plan_len + p.B;
    auto bar = [&](int i) -> uint32_t { return sBar + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtx wc{abort_flag, p.status};
    const float kNegInf = -__int_as_float(0x7f800000);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            const bool by_warpgroup = (i >= C::kBarPFull && i < C::kBarPFull + C::kPFulls) ||
                                      (i >= C::kBarODrained && i < C::kBarODrained + NQ) || (NR > 0 && i == C::kBarJoin);
            mbar_init(bar(i), by_warpgroup ? 4u : 1u);  // one arrive per warp
        }
        *abort_flag = 0;
        for (int i = 0; i < kOddSlots; ++i) odd_seg[i] = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == C::kProducerWarp && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    // While the kernel before may still be running: the plan, of lengths that may yet change.  If one
    // has, it is made again.
    const int G = p.g * p.rg, rng = (int)blockIdx.x / G, member = (int)blockIdx.x - rng * G;
    PagedWalk<C> walk;
    PagedSeg s;
    const bool producer = warp == C::kProducerWarp || warp == C::kProducerWarp + 1;
    bool more = false;
    // The producer: a tile is nb boxes of box_rows keys and DA column atoms; lane i issues box i % nb
    // of atom i / nb.  Table entries are loaded for 32 / nb tiles at a time, one such window ahead.
    const int nb_log = p.nb_log, box = lane & ((1 << nb_log) - 1), ahead = lane >> nb_log;
    auto fetch = [&](const PagedSeg& sg, int u) -> int2 {
        u += ahead;
        const int row = box * p.box_rows;
        const int key = u < sg.u1 ? sg.strips.key(u * (BN / 32) + row / 32) + row % 32 : sg.len;
        return key < sg.len ? paged_place(p, sg.b, key) : make_int2(-1, 0);
    };
    int2 ids = make_int2(-1, 0);
    tc_fence_before();
    for (bool first = true;; first = false) {
        paged_make_plan<C, C::kThreads>(p, plan_len, plan_prefix, s_warp_sum);
        walk.init(p, plan_len, plan_prefix, rng, member);
        if (producer) more = walk.next(p, s);
        if (first) {
            // The first tile is sent for to L2, by a table that may yet change too: a guess, which decides
            // nothing but the lines that go there.
            if (more) {
                const int2 guess = fetch(s, s.u0);
                const int page = __shfl_sync(0xffffffffu, guess.x, box), row = __shfl_sync(0xffffffffu, guess.y, box);
                if (ahead < DA && page >= 0)
                    tma_prefetch_4d(warp == C::kProducerWarp ? &tm_k : &tm_v, ahead * 64, s.hk, row, page);
            }
            grid_dependency_wait();
        }
        // (every warp by itself: after the wait all see the same lengths; the first are on their way with the
        // first table entries)
        const int now = __ldcg(p.kv_lens + min(lane, p.B - 1));
        if (more) ids = fetch(s, s.u0);
        bool stale = min(max(now, 0), p.capacity) != plan_len[min(lane, p.B - 1)];
        for (int b = lane + 32; b < p.B; b += 32) stale |= paged_len(p, b) != plan_len[b];
        if (!__any_sync(0xffffffffu, stale)) break;
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

    if (producer) {
        // ----------------------------------------------------------- TMA producers --
        // One for Q and K, one for V: a copy takes a warp some 70 cycles, and a tile of 16-key pages is 16
        // copies of K and as many of V.
        const int nb = 1 << nb_log, per_window = 32 >> nb_log, atom = ahead;
        const int is_v = warp - C::kProducerWarp;
        const CUtensorMap* map = is_v ? &tm_v : &tm_k;
        uint32_t load = is_v, tcount = 0;  // the ring's loads: K of tile n is load 2 n, V is load 2 n + 1; segments
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(b, parity, wc));
        };
        const uint32_t q_bytes = (uint32_t)(DA * p.T * p.group * 128);
        auto load_q = [&](const PagedSeg& sg) -> bool {
            for (int q = 0; q < NQ; ++q) {
                if (!wait(bar(C::kBarQEmpty + q), (tcount & 1u) ^ 1u)) return false;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarQFull + q), q_bytes);
                __syncwarp();
                if (lane < DA)
                    tma_load_4d(sQ + q * C::kQBytes + lane * (C::kQRows * 128), &tm_q, bar(C::kBarQFull + q), lane * 64,
                                sg.hk * p.group, (sg.rb * NQ + q) * p.T, sg.b);
            }
            ++tcount;
            return true;
        };
        while (more && ok) {
            PagedSeg nxt;
            bool again = false, first = true;
            for (int u = s.u0; u < s.u1 && ok; u += per_window) {
                const int2 use = ids;
                const int n = min(per_window, s.u1 - u);
                for (int k = 0; k < n && ok; ++k) {
                    const int page = __shfl_sync(0xffffffffu, use.x, k * nb + box);
                    const int row = __shfl_sync(0xffffffffu, use.y, k * nb + box);
                    const uint32_t st = load % NB;
                    ok = wait(bar(C::kBarEmpty + st), ((load / NB) & 1u) ^ 1u);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarFull + st), C::kTileBytes);
                    __syncwarp();
                    if (atom < DA)  // keys on no page read as zeros: a page past the last one
                        tma_load_4d(sRing + st * C::kTileBytes + atom * (BN * 128) + box * p.box_rows * 128, map,
                                    bar(C::kBarFull + st), atom * 64, s.hk, row, page < 0 ? p.num_pages : page);
                    load += 2;
                    if (first) {
                        // Behind the first tile: the queries, which may have to wait for the products of the
                        // segment before, and what comes after this segment.
                        if (!is_v) ok = load_q(s);
                        again = walk.next(p, nxt);
                        first = false;
                    }
                    if (k == 0) {  // the next window's table entries
                        if (u + per_window < s.u1)
                            ids = fetch(s, u + per_window);
                        else if (again)
                            ids = fetch(nxt, nxt.u0);
                    }
                }
            }
            s = nxt;
            more = again;
        }
        grid_launch_dependents();  // only now: the merge kernel's CTAs share the SM with this one
        __syncwarp();
        // Every copy this warp started has landed before shared memory goes.
        if (lane == 0) {
            // (the last use of each buffer: an earlier one's phase may have passed twice)
            const uint32_t end = load - is_v;
            for (uint32_t l = load; l >= 2 + (uint32_t)is_v && l - 2 + NB >= end; l -= 2)
                mbar_wait_drain(bar(C::kBarFull + (l - 2) % NB), ((l - 2) / NB) & 1u);
            if (tcount > 0)
                for (int q = 0; q < NQ; ++q) mbar_wait_drain(bar(C::kBarQFull + q), (tcount - 1) & 1u);
        }
        __syncwarp();
    } else if (NR > 0 && warp == C::kMmaWarp) {
        // ----------------------------------------------------- MMA issuer, few rows ----
        // S^T of the next tile is issued ahead of O^T += V^T P^T of this one.
        if constexpr (NR > 0) {
            constexpr uint32_t idesc_s = make_idesc_f16(128, NR, kBF16, false, false);
            constexpr uint32_t idesc_o = make_idesc_f16(128, NR, kBF16, true, false);
            uint32_t it = 0, tcount = 0;
            bool ok = true;
            auto wait = [&](uint32_t b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(b, parity, wc));
            };
            auto wait_load = [&](uint32_t load) -> bool { return wait(bar(C::kBarFull + load % NB), (load / NB) & 1u); };
            auto free_load = [&](uint32_t load) { umma_commit_elect(bar(C::kBarEmpty + load % NB)); };
            const uint64_t dq = make_sdesc_sw128(sQ, 16, 1024), dk = make_sdesc_sw128(sRing, 16, 1024);
            const uint64_t dv = make_sdesc_sw128(sRing, BN * 128, 1024), dp = make_sdesc_sw128(base + C::kPOff, 16, 1024);
            const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32), k_lo = (uint32_t)dk;
            const uint32_t k_hi = (uint32_t)(dk >> 32), v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
            const uint32_t p_lo = (uint32_t)dp, p_hi = (uint32_t)(dp >> 32);
            auto issue_s = [&](uint32_t tile) {
                const uint32_t d = tmem + (tile & 1u) * NR;
                const uint32_t a = k_lo + (((2 * tile % NB) * C::kTileBytes) >> 4);
                umma_ss_elect<false>(d, a, k_hi, q_lo, q_hi, idesc_s);
#pragma unroll
                for (int kk = 1; kk < D / 16; ++kk)
                    umma_ss_elect<true>(d, a + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), k_hi,
                                        q_lo + (((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4), q_hi, idesc_s);
                umma_commit_elect(bar(C::kBarSFull + (tile & 1u)));
                free_load(2 * tile);
            };
            auto issue_pv = [&](uint32_t tile, bool acc) {
                const uint32_t b = p_lo + (((tile & 1u) * C::kPBytes) >> 4);
                const uint32_t d = tmem + C::kOCol0, a = v_lo + ((((2 * tile + 1) % NB) * C::kTileBytes) >> 4);
                if (acc)
                    umma_ss_elect<true>(d, a, v_hi, b, p_hi, idesc_o);
                else
                    umma_ss_elect<false>(d, a, v_hi, b, p_hi, idesc_o);
#pragma unroll
                for (int kk = 1; kk < BN / 16; ++kk)
                    umma_ss_elect<true>(d, a + ((kk * (16 * 128)) >> 4), v_hi,
                                        b + (((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4), p_hi, idesc_o);
                umma_commit_elect(bar(C::kBarODone + (tile & 1u)));
                free_load(2 * tile + 1);
            };
            while (ok && walk.next(p, s)) {
                const int n = s.u1 - s.u0;
                ok = wait(bar(C::kBarQFull), tcount & 1u) && wait_load(2 * it);
                if (!ok) break;
                tc_fence_after();
                issue_s(it);
                if (n == 1) umma_commit_elect(bar(C::kBarQEmpty));
                for (int j = 0; j < n && ok; ++j) {
                    if (j + 1 < n) {
                        ok = wait_load(2 * it + 2);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(it + 1);
                        if (j + 2 == n) umma_commit_elect(bar(C::kBarQEmpty));
                    }
                    ok = wait_load(2 * it + 1) && wait(bar(C::kBarPFull + (it & 1u)), (it >> 1) & 1u);
                    if (ok && j == 0 && tcount > 0) ok = wait(bar(C::kBarODrained), (tcount - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(it, j > 0);
                    ++it;
                }
                ++tcount;
            }
            umma_commit_elect(bar(C::kBarFinal));
            mbar_wait_drain(bar(C::kBarFinal), 0);
            __syncwarp();
        }
    } else if (NR > 0) {
        // --------------------------------------------- softmax warpgroup, few rows ----
        if constexpr (NR > 0) {
            const int t = threadIdx.x;  // the key within a tile, and the row of O^T
            const int R = p.Sq * p.group;
            const uint32_t all = paged_bits(0, R - 1), of_token = paged_bits(0, p.group - 1);
            const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
            constexpr float kRescaleLog2 = 8.0f;  // the reference lags a row's maximum by less than 2^8
            float* red = reinterpret_cast<float*>(smem_raw + (base - raw) + C::kRedOff);  // [2][4][32]
            float* own = red + 256 + warp * 32;                                           // this warp's [32]
            int* rel = reinterpret_cast<int*>(red + 384);                                 // [32]
            volatile int* grown = rel + 32;                                               // [2]
            uint16_t* o16 = static_cast<uint16_t*>(p.o);
            uint32_t it = 0, tcount = 0, joins = 0, reds = 0;
            bool ok = true;
            // A barrier of the four warps whose wait is bounded like any other: arrive, then wait.
            auto arrive = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarJoin));
            };
            auto joined = [&]() -> bool { return mbar_wait(bar(C::kBarJoin), joins++ & 1u, wc); };
            auto load_row = [&](uint32_t col, uint32_t (&x)[NR]) {
                tmem_ld_32x32b_x16(lane_base + col, x);
                tmem_wait_ld(x);
            };
            // What the warps' lanes n hold, to all of them: four values each.
            auto gather = [&](float x, float (&y)[4]) -> bool {
                float* to = red + (reds++ & 1u) * 128;
                to[warp * 32 + lane] = x;
                arrive();
                if (!joined()) return false;
                for (int w = 0; w < 4; ++w) y[w] = to[w * 32 + lane];
                return true;
            };
            // All lanes get all lanes' x.
            auto spread = [&](float x, float (&v)[NR]) {
                __syncwarp();
                own[lane] = x;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NR; i += 4) load_vec<4>(v + i, own + i);
            };
            if (t < 32) {
                const int tok = t / p.group;
                rel[t] = tok * p.Hq + t - tok * p.group;  // a row's place behind the pair's first
                if (t < 2) grown[t] = 0;
            }
            arrive();
            ok = joined();

            for (int b = blockIdx.x; ok && b < p.B; b += gridDim.x) {  // sequences without keys
                if (plan_len[b] > 0) continue;
                const long long vals = (long long)p.Sq * p.Hq * D, rows = (long long)p.Sq * p.Hq;
                for (long long i = (long long)t * 8; i < vals; i += 128 * 8)
                    st_global_v4(o16 + b * vals + i, 0u, 0u, 0u, 0u);
                if (p.lse)
                    for (long long i = t; i < rows; i += 128) p.lse[b * rows + i] = kNegInf;
            }

            while (ok && walk.next(p, s)) {
                const int n = s.u1 - s.u0, ctx = s.len - p.Sq;
                const PagedClear clear = paged_clear(p, s.len, s.strips);
                // Lane i has the mask of token i; a draft's rows are one of its columns.
                const uint32_t tree = p.tree && lane < p.Sq ? (uint32_t)__ldg(p.tree + (size_t)s.b * p.Sq + lane) : 0u;
                float mref[NR], l[NR];  // the rows' references, in the exponent; this thread's part of their sums
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    mref[i] = kNegInf;
                    l[i] = 0.f;
                }
                for (int j = 0; j < n; ++j) {
                    const int strip0 = (s.u0 + j) * 4;
                    const bool masked = strip0 < clear.lo || strip0 + 4 > clear.hi;
                    uint32_t vis = all;  // the rows that see this thread's key
                    if (masked) {
                        if (!clear.has(strip0 + warp)) {
                            const int key = s.strips.key(strip0 + warp) + lane, d = key - ctx;
                            uint32_t seen = 0;  // of a draft: by the rows of the tokens whose bit is set
                            for (int i = 0; p.tree && i < p.Sq; ++i) {
                                const uint32_t w = __shfl_sync(0xffffffffu, tree, i);
                                if (d >= 0 && w >> (d & 31) & 1u) seen |= of_token << (i * p.group);
                            }
                            if (key >= s.len) {
                                vis = 0;
                            } else if (p.tree) {
                                if (d >= 0) vis = seen;
                            } else {
                                // tokens d .. d + window see it, or d .. of a sink
                                const int last = p.window_left < 0 || key < p.sinks ? p.Sq - 1
                                                                                    : min(d + p.window_left, p.Sq - 1);
                                vis = last < 0 ? 0u : paged_bits(max(d, 0) * p.group, (last + 1) * p.group - 1);
                                if (max(d, 0) >= p.Sq) vis = 0;
                            }
                        }
                        __syncwarp();
                        const uint32_t load = 2 * it + 1, at = sRing + (load % NB) * C::kTileBytes;
                        ok = mbar_wait(bar(C::kBarFull + load % NB), (load / NB) & 1u, wc);
                        if (!ok) break;
                        if (paged_finite_v<DA, BN, kBF16>(at, t, clear, strip0)) odd_seg[tcount % kOddSlots] = (int)tcount + 1;
                    }
                    ok = mbar_wait(bar(C::kBarSFull + (it & 1u)), (it >> 1) & 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t u[NR];
                    load_row((it & 1u) * NR, u);
                    float x[NR];
                    bool grow = j == 0;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        x[i] = (vis >> i) & 1u ? __uint_as_float(u[i]) * p.scale_log2 : kNegInf;
                        grow |= x[i] > mref[i] + kRescaleLog2;
                    }
                    if (j > 0) {
                        if (__any_sync(0xffffffffu, grow) && lane == 0) grown[it & 1u] = (int)it + 1;
                        arrive();
                        ok = joined();
                        if (!ok) break;
                        grow = grown[it & 1u] == (int)it + 1;
                    }
                    // P's buffer is that of the tile before the last: its products are done.
                    if (it >= 2) {
                        ok = mbar_wait(bar(C::kBarODone + (it & 1u)), ((it >> 1) - 1) & 1u, wc);
                        if (!ok) break;
                    }
                    if (grow) {  // the same in all warps: new references
                        float v[NR], y[4];
#pragma unroll
                        for (int i = 0; i < NR; ++i) v[i] = x[i];
                        ok = gather(paged_transposed<false>(v), y);
                        if (!ok) break;
                        spread(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), v);
#pragma unroll
                        for (int i = 0; i < NR; ++i) {
                            const float to = fmaxf(mref[i], v[i]);
                            v[i] = to == mref[i] ? 1.f : ex2_approx(mref[i] - to);
                            mref[i] = to;
                            l[i] *= v[i];
                        }
                        if (j > 0) {
                            ok = mbar_wait(bar(C::kBarODone + ((it - 1) & 1u)), ((it - 1) >> 1) & 1u, wc);
                            if (!ok) break;
                            tc_fence_after();
                            uint32_t o[NR];
                            load_row(C::kOCol0, o);
#pragma unroll
                            for (int i = 0; i < NR; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * v[i]);
                            tmem_st_32x32b_x16(lane_base + C::kOCol0, o);
                            tmem_wait_st();
                        }
                    }
                    // P = exp2(x - m), rounded to the inputs' 16 bits for the product; the sums l take it
                    // unrounded.  Row i's 128 keys are two runs of 64, 128 bytes each, in 16-byte units that are
                    // permuted as the products want them.
                    const uint32_t to = base + C::kPOff + (it & 1u) * C::kPBytes + (t >> 6) * (NR * 128) + (t & 7) * 2;
                    const uint32_t unit = (t & 63) >> 3;
#pragma unroll
                    for (int i = 0; i < NR; i += 2) {
                        const float p0 = ex2_approx(x[i] - (mref[i] == kNegInf ? 0.f : mref[i]));
                        const float p1 = ex2_approx(x[i + 1] - (mref[i + 1] == kNegInf ? 0.f : mref[i + 1]));
                        l[i] += p0;
                        l[i + 1] += p1;
                        const uint32_t w = pack2<kBF16>(p0, p1);
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + i * 128 + ((unit ^ (i & 7)) << 4)),
                                     "h"((uint16_t)w)
                                     : "memory");
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + (i + 1) * 128 +
                                                                     ((unit ^ ((i + 1) & 7)) << 4)),
                                     "h"((uint16_t)(w >> 16))
                                     : "memory");
                    }
                    fence_proxy_async_shared();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarPFull + (it & 1u)));
                    ++it;
                }
                if (!ok) break;

                // -------------------------------------------------------- epilogue ----
                float v[NR], y[4];
#pragma unroll
                for (int i = 0; i < NR; ++i) v[i] = l[i];
                ok = gather(paged_transposed<true>(v), y);
                if (!ok) break;
                const float sum = (y[0] + y[1]) + (y[2] + y[3]);
                spread(sum == 0.f ? 0.f : 1.0f / sum, v);  // 0: the row sees no key of the segment
                ok = mbar_wait(bar(C::kBarODone + ((it - 1) & 1u)), ((it - 1) >> 1) & 1u, wc);
                if (!ok) break;
                tc_fence_after();
                const bool odd = odd_seg[tcount % kOddSlots] == (int)tcount + 1;
                const size_t row0 = (size_t)s.b * p.Sq * p.Hq + s.hk * p.group;
                const size_t part0 = ((size_t)member * 2 * p.ranges + s.slot) * R;
                uint32_t o[NR];
                load_row(C::kOCol0, o);
                if (t < D) {  // lanes side by side have dims side by side
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        if (i >= R) break;
                        const float y = v[i] == 0.f ? 0.f : __uint_as_float(o[i]) * v[i];
                        if (s.cut)
                            p.o_part[(part0 + i) * D + t] = y;
                        else
                            o16[(row0 + rel[i]) * D + t] = float_to16<kBF16>(y);
                    }
                }
                __syncwarp();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarODrained));
                if (warp == 0) {
                    float m = kNegInf;
#pragma unroll
                    for (int i = 0; i < NR; ++i) m = lane == i ? mref[i] : m;
                    const float lse = sum == 0.f ? kNegInf : (m + lg2_approx(sum)) * kPagedLn2;
                    if (lane < R) {
                        const int tok = lane / p.group;
                        if (s.cut)
                            p.lse_part[part0 + lane] = lse;
                        else if (p.lse)
                            p.lse[((size_t)s.b * p.Hq + s.hk * p.group + lane - tok * p.group) * p.Sq + tok] = lse;
                    }
                }
                if (odd) {  // (the same in all threads) behind all of the rows' writes
                    __threadfence_block();
                    arrive();
                    ok = joined();
                    if (!ok) break;
                    if (t < R)
                        paged_add_odd<D, BN, kBF16>(p, s.b, s.hk, s.len, t / p.group, s.u0, s.u1,
                                                    s.cut ? p.o_part + (part0 + t) * D : nullptr,
                                                    o16 + (row0 + rel[t]) * D);
                    __syncwarp();
                }
                ++tcount;
            }
        }
    } else if (warp == C::kMmaWarp) {
        if constexpr (NR == 0) {
            // ------------------------------------------------------------- MMA issuer ----
            // One sub-tile: S of the next tile is issued ahead of P.V of this one, S having two buffers.  Two
            // sub-tiles: P.V and the next S of one run while the other's softmax does.
            constexpr uint32_t idesc_s = make_idesc_f16(128, BN, kBF16, false, false);
            constexpr uint32_t idesc_o = make_idesc_f16(128, D, kBF16, false, true);
            uint32_t kv_it = 0, tcount = 0;  // tiles and segments done
            bool ok = true;
            auto wait = [&](uint32_t b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(b, parity, wc));
            };
            // K of tile n is load 2 n of the ring, V is load 2 n + 1.
            auto wait_load = [&](uint32_t load) -> bool { return wait(bar(C::kBarFull + load % NB), (load / NB) & 1u); };
            auto free_load = [&](uint32_t load) { umma_commit_elect(bar(C::kBarEmpty + load % NB)); };
            const uint64_t dq = make_sdesc_sw128(sQ, 16, 1024);
            const uint64_t dk = make_sdesc_sw128(sRing, 16, 1024);
            const uint64_t dv = make_sdesc_sw128(sRing, BN * 128, 1024);
            const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32);
            const uint32_t k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
            const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
            auto issue_s = [&](int q, uint32_t load, uint32_t slot) {
                const uint32_t d = tmem + slot * BN;
                const uint32_t a = q_lo + (uint32_t)((q * C::kQBytes) >> 4);
                const uint32_t b = k_lo + (((load % NB) * C::kTileBytes) >> 4);
                umma_ss_elect<false>(d, a, q_hi, b, k_hi, idesc_s);
#pragma unroll
                for (int kk = 1; kk < D / 16; ++kk)
                    umma_ss_elect<true>(d, a + (((kk >> 2) * (C::BM * 128) + (kk & 3) * 32) >> 4), q_hi,
                                        b + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), k_hi, idesc_s);
            };
            auto issue_pv = [&](int q, uint32_t load, uint32_t slot, bool acc) {
                const uint32_t d = tmem + C::kOCol0 + q * D;
                const uint32_t a = tmem + slot * BN;
                const uint32_t b = v_lo + (((load % NB) * C::kTileBytes) >> 4);
                if (acc)
                    umma_ts_elect<true>(d, a, b, v_hi, idesc_o);
                else
                    umma_ts_elect<false>(d, a, b, v_hi, idesc_o);
#pragma unroll
                for (int kk = 1; kk < BN / 16; ++kk)
                    umma_ts_elect<true>(d, a + kk * 8, b + ((kk * (16 * 128)) >> 4), v_hi, idesc_o);
            };
            while (ok && walk.next(p, s)) {
                const int n = s.u1 - s.u0;
                for (int q = 0; q < NQ && ok; ++q) ok = wait(bar(C::kBarQFull + q), tcount & 1u);
                ok = ok && wait_load(2 * kv_it);
                if (!ok) break;
                for (int q = 0; q < NQ; ++q) {
                    const uint32_t slot = NQ == 1 ? kv_it & 1u : (uint32_t)q;
                    issue_s(q, 2 * kv_it, slot);
                    umma_commit_elect(bar(C::kBarSFull + slot));
                    if (n == 1) umma_commit_elect(bar(C::kBarQEmpty + q));
                }
                free_load(2 * kv_it);
                for (int j = 0; j < n && ok; ++j) {
                    const bool next = j + 1 < n;
                    if (NQ == 1 && next) {
                        ok = wait_load(2 * kv_it + 2);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(0, 2 * kv_it + 2, (kv_it + 1) & 1u);
                        umma_commit_elect(bar(C::kBarSFull + ((kv_it + 1) & 1u)));
                        free_load(2 * kv_it + 2);
                        if (j + 2 == n) umma_commit_elect(bar(C::kBarQEmpty));
                    }
                    ok = wait_load(2 * kv_it + 1);
                    for (int q = 0; q < NQ && ok; ++q) {
                        ok = wait(bar(C::kBarPFull + q), kv_it & 1u);
                        if (ok && j == 0 && tcount > 0) ok = wait(bar(C::kBarODrained + q), (tcount - 1) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(q, 2 * kv_it + 1, NQ == 1 ? kv_it & 1u : (uint32_t)q, j > 0);
                        if (NQ == 1 || !next) umma_commit_elect(bar(C::kBarODone + q));
                        if (q == NQ - 1) free_load(2 * kv_it + 1);
                        if (NQ > 1 && next) {
                            if (q == 0) {
                                ok = wait_load(2 * kv_it + 2);
                                if (!ok) break;
                            }
                            issue_s(q, 2 * kv_it + 2, (uint32_t)q);
                            umma_commit_elect(bar(C::kBarSFull + q));
                            if (q == NQ - 1) free_load(2 * kv_it + 2);
                            if (j + 2 == n) umma_commit_elect(bar(C::kBarQEmpty + q));
                        }
                    }
                    ++kv_it;
                }
                ++tcount;
            }
            // Every product issued is done before TMEM and shared memory are released.
            umma_commit_elect(bar(C::kBarFinal));
            mbar_wait_drain(bar(C::kBarFinal), 0);
            __syncwarp();
        }
    } else {
        if constexpr (NR == 0) {
            // ------------------------------------------------------ softmax warpgroups ----
            const int q = warp >> 2, wq = warp & 3;
            const int r = wq * 32 + lane;  // row of the sub-tile's 128 = TMEM lane
            const int tok_l = r / p.group, h_l = r - tok_l * p.group;
            const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
            const uint32_t tO = lane_base + C::kOCol0 + q * D;
            constexpr int kSC = BN / 32;
            constexpr float kRescaleLog2 = 8.0f;  // O is rescaled only when a maximum grows by more than 2^8
            const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
            const int block_rows = min(NQ * p.T, p.Sq) * p.group;
            uint16_t* o16 = static_cast<uint16_t*>(p.o);
            uint32_t it = 0, tcount = 0;
            bool ok = true;

            // Sequences without keys.
            for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
                if (plan_len[b] > 0) continue;
                const long long vals = (long long)p.Sq * p.Hq * D, rows = (long long)p.Sq * p.Hq;
                for (long long i = (long long)threadIdx.x * 8; i < vals; i += 128 * NQ * 8)
                    st_global_v4(o16 + b * vals + i, 0u, 0u, 0u, 0u);
                if (p.lse)
                    for (long long i = threadIdx.x; i < rows; i += 128 * NQ) p.lse[b * rows + i] = kNegInf;
            }

            while (ok && walk.next(p, s)) {
                const int n = s.u1 - s.u0;
                const int tok = (s.rb * NQ + q) * p.T + tok_l;
                const bool live = tok_l < p.T && tok < p.Sq;
                const bool any = __any_sync(0xffffffffu, live);  // whether the warp has rows
                const PagedClear clear = paged_clear(p, s.len, s.strips);
                const int tok_in = live ? tok : 0;
                int lo, hi, sink;
                paged_row(p, s.len, tok_in, lo, hi, sink);
                float m_run = kNegInf;
                uint64_t l2 = f2_pack(0.f, 0.f);
                for (int j = 0; j < n; ++j) {
                    const int strip0 = (s.u0 + j) * kSC;
                    const bool masked = strip0 < clear.lo || strip0 + kSC > clear.hi;
                    if (masked && q == 0) {
                        const uint32_t load = 2 * it + 1, at = sRing + (load % NB) * C::kTileBytes;
                        ok = mbar_wait(bar(C::kBarFull + load % NB), (load / NB) & 1u, wc);
                        if (!ok) break;
                        if (paged_finite_v<DA, BN, kBF16>(at, r, clear, strip0)) odd_seg[tcount % kOddSlots] = (int)tcount + 1;
                    }
                    const uint32_t slot = NQ == 1 ? it & 1u : (uint32_t)q;
                    float alpha = 1.f;
                    ok = mbar_wait(bar(C::kBarSFull + slot), NQ == 1 ? (it >> 1) & 1u : it & 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tS = lane_base + slot * BN;  // P goes over S
                    // P = exp2(s * scale * log2 e - m), rounded to the inputs' 16 bits for the product (a relative
                    // error of half a step each, independent, so of a row's output about that of its own
                    // rounding); the sum l takes it unrounded.
                    uint64_t sum2 = f2_pack(0.f, 0.f), nm2 = 0;
                    auto new_max = [&](float raw_max) {
                        const float m_blk = raw_max == kNegInf ? kNegInf : raw_max * p.scale_log2;
                        const bool bump = live && m_blk > m_run + kRescaleLog2;  // (other rows hold anything)
                        const float m_new = bump ? m_blk : m_run;
                        alpha = bump ? ex2_approx(m_run - m_new) : 1.0f;
                        m_run = m_new;
                        const float m_sub = m_run == kNegInf ? 0.f : m_run;
                        nm2 = f2_pack(-m_sub, -m_sub);
                    };
                    auto put_p = [&](int ch, const uint32_t (&u)[32]) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint64_t a =
                                fma2(f2_pack(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), c2, nm2);
                            float a0, a1;
                            f2_unpack(a, a0, a1);
                            const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
                            sum2 = add2(sum2, f2_pack(p0, p1));
                            pk[i] = pack2<kBF16>(p0, p1);
                        }
                        tmem_st_32x32b_x16(tS + ch * 16, pk);
                    };
                    if (any) {
                        uint32_t u[kSC][32];
#pragma unroll
                        for (int ch = 0; ch < kSC; ++ch) tmem_ld_32x32b_x32(tS + ch * 32, u[ch]);
                        tmem_wait_ld(u[0]);
#pragma unroll
                        for (int ch = 1; ch < kSC; ++ch) reg_fence(u[ch]);
                        if (masked) {
#pragma unroll
                            for (int ch = 0; ch < kSC; ++ch) {
                                if (clear.has(strip0 + ch)) continue;
                                // The row sees the keys lo .. hi and those before sink, and what the tree's mask says.
                                const int k = s.strips.key(strip0 + ch);
                                uint32_t w = paged_bits(lo - k, hi - k) | paged_bits(0, sink - 1 - k);
                                if (p.tree) w |= paged_drafts(p, s.b, tok_in, s.len, k);
                                if (!live) w = 0;
#pragma unroll
                                for (int i = 0; i < 32; ++i) u[ch][i] = (w >> i) & 1u ? u[ch][i] : 0xff800000u;
                            }
                            __syncwarp();
                        }
                        auto sv = [&](int k) -> float { return __uint_as_float(u[k >> 5][k & 31]); };
                        float mx[4];  // four chains of 3-input maxima
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = sv(k);
#pragma unroll
                        for (int k = 4; k + 8 <= BN; k += 8)
#pragma unroll
                            for (int c4 = 0; c4 < 4; ++c4) mx[c4] = max3f(mx[c4], sv(k + c4), sv(k + c4 + 4));
#pragma unroll
                        for (int c4 = 0; c4 < 4; ++c4) mx[c4] = fmaxf(mx[c4], sv(BN - 4 + c4));
                        new_max(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
#pragma unroll
                        for (int ch = 0; ch < kSC; ++ch) put_p(ch, u[ch]);
                    }
                    l2 = fma2(l2, f2_pack(alpha, alpha), sum2);
                    if (NQ == 1 && j > 0) {
                        // the product before may still be adding to O (with two sub-tiles, S of this tile
                        // was issued behind it)
                        ok = mbar_wait(bar(C::kBarODone + q), (it - 1) & 1u, wc);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (any && j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
                        for (int ch = 0; ch < D / 32; ++ch) {
                            uint32_t ov[32];
                            tmem_ld_32x32b_x32(tO + ch * 32, ov);
                            tmem_wait_ld(ov);
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            tmem_st_32x32b_x32(tO + ch * 32, ov);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarPFull + q));
                    ++it;
                }
                if (!ok) break;

                // ------------------------------------------------------------ epilogue ----
                ok = mbar_wait(bar(C::kBarODone + q), NQ == 1 ? (it - 1) & 1u : tcount & 1u, wc);
                if (!ok) break;
                tc_fence_after();
                const bool odd = odd_seg[tcount % kOddSlots] == (int)tcount + 1;
                float l0, l1;
                f2_unpack(l2, l0, l1);
                const float l_run = l0 + l1;
                const bool none = l_run == 0.f;  // the row sees no key of the segment
                const float inv_l = 1.0f / l_run;
                const int h = s.hk * p.group + h_l;
                const size_t row = ((size_t)s.b * p.Sq + tok) * p.Hq + h;
                const size_t part = ((size_t)member * 2 * p.ranges + s.slot) * block_rows + q * p.T * p.group + r;
                // The warp's live rows are its first ones; in the partial result they are part or row + ... of the
                // first.
                const int rows = __popc(__ballot_sync(0xffffffffu, live));
                const uint32_t out = sOut + (uint32_t)warp * (32 * (C::OC + 4) * 4);
                // Lanes of a row and rows at a time, of 32-bit and of 16-bit results.
                constexpr int LF = C::OC / 4, RF = 32 / LF, LH = C::OC / 8, RH = 32 / LH;
                uint32_t at[LH];
#pragma unroll
                for (int i = 0; i < LH; ++i) at[i] = __shfl_sync(0xffffffffu, (uint32_t)row, i * RH + lane / LH);
                auto load_o = [&](int c0, uint32_t (&ov)[C::OC]) {
                    if constexpr (C::OC == 32)
                        tmem_ld_32x32b_x32(tO + c0, ov);
                    else
                        tmem_ld_32x32b_x16(tO + c0, ov);
                };
                auto put_o = [&](int c0, uint32_t (&ov)[C::OC]) {
#pragma unroll
                    for (int i = 0; i < C::OC; ++i) ov[i] = none ? 0u : __float_as_uint(__uint_as_float(ov[i]) * inv_l);
                    __syncwarp();  // the columns before have been read
#pragma unroll
                    for (int i = 0; i < C::OC; i += 4)
                        st_shared_v4(out + (lane * (C::OC + 4) + i) * 4, ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
                    __syncwarp();
                    if (s.cut) {
                        const int rr = lane / LF, cc = lane % LF * 4;
                        float* to = p.o_part + (part - lane + rr) * D + c0 + cc;
                        uint32_t w[LF][4];
#pragma unroll
                        for (int i = 0; i < LF; ++i) lds128(out + ((i * RF + rr) * (C::OC + 4) + cc) * 4, w[i]);
#pragma unroll
                        for (int i = 0; i < LF; ++i)
                            if (i * RF + rr < rows) st_global_v4(to + i * RF * D, w[i][0], w[i][1], w[i][2], w[i][3]);
                    } else {
                        const int rr = lane / LH, cc = lane % LH * 8;
                        uint32_t w[LH][4], x[LH][4];
#pragma unroll
                        for (int i = 0; i < LH; ++i) {
                            lds128(out + ((i * RH + rr) * (C::OC + 4) + cc) * 4, w[i]);
                            lds128(out + ((i * RH + rr) * (C::OC + 4) + cc + 4) * 4, x[i]);
                        }
                        auto f = [](uint32_t y) { return __uint_as_float(y); };
#pragma unroll
                        for (int i = 0; i < LH; ++i)
                            if (i * RH + rr < rows)
                                st_global_v4(o16 + (size_t)at[i] * D + c0 + cc, pack2<kBF16>(f(w[i][0]), f(w[i][1])),
                                             pack2<kBF16>(f(w[i][2]), f(w[i][3])), pack2<kBF16>(f(x[i][0]), f(x[i][1])),
                                             pack2<kBF16>(f(x[i][2]), f(x[i][3])));
                    }
                };
#pragma unroll 1
                for (int c0 = 0; any && c0 < D; c0 += C::OC) {
                    uint32_t ov[C::OC];
                    load_o(c0, ov);
                    tmem_wait_ld(ov);
                    put_o(c0, ov);
                }
                if (odd) {  // other lanes' writes to the row come first
                    __threadfence_block();
                    __syncwarp();
                }
                if (live) {
                    if (odd)
                        paged_add_odd<D, BN, kBF16>(p, s.b, s.hk, s.len, tok, s.u0, s.u1, s.cut ? p.o_part + part * D : nullptr,
                                                    o16 + row * D);
                    const float lse = none ? kNegInf : (m_run + lg2_approx(l_run)) * kPagedLn2;
                    if (s.cut)
                        p.lse_part[part] = lse;
                    else if (p.lse)
                        p.lse[((size_t)s.b * p.Hq + h) * p.Sq + tok] = lse;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarODrained + q));
                ++tcount;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the pieces of the entries that were cut: lse = log sum_c exp(lse_c), and the outputs weighted
// with exp(lse_c - lse).  p.merge_ctas CTAs for each of the split kernel's: they walk the same range,
// and of each cut entry that they meet they join the share of the rows that the CTAs of the entry's
// other pieces do not.
// Eight warps take a row each, or share one where there are few; a lane holds D / 32 dims.  The
// plan is made before the split kernel is done.
template <class C, bool kBF16>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedDecParams p) {
    constexpr int D = C::D, NQ = C::NQ, V = D / 32, NP = V <= 4 ? 2 : 4;  // NP: pieces loaded together
    constexpr int Vec = V % 4 == 0 ? 4 : V % 2 == 0 ? 2 : 1;  // values of a lane side by side
    __shared__ __align__(16) float s_acc[8][D];
    __shared__ float s_sum[8], s_max[8];
    __shared__ int s_warp_sum[8];
    extern __shared__ int s_plan[];  // as large as the batch: the CTA fits beside the split kernels'
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float kNegInf = -__int_as_float(0x7f800000);
    paged_make_plan<C, 256>(p, s_plan, s_plan + p.B, s_warp_sum);
    const int G = p.g * p.rg, k = p.merge_ctas, cta = (int)blockIdx.x / k, sub = (int)blockIdx.x - cta * k;
    const int rng = cta / G, member = cta - rng * G;
    const int block_rows = min(NQ * p.T, p.Sq) * p.group;
    PagedWalk<C> walk;
    walk.init(p, s_plan, s_plan + p.B, rng, member);
    PagedSeg seg;
    bool waited = false;
    grid_launch_dependents();
    while (walk.next(p, seg)) {
        if (!seg.cut) continue;
        const int n = paged_pieces<C>(walk.start, walk.units, walk.W);
        const int first = paged_first_piece<C>(walk.start, walk.W), piece = (rng - first) * k + sub;
        const int tok0 = seg.rb * NQ * p.T;
        const int rows = min(block_rows, (p.Sq - tok0) * p.group);  // of this row block
        const int lo = (int)((unsigned)(rows * piece) / (unsigned)(n * k));
        const int hi = (int)((unsigned)(rows * (piece + 1)) / (unsigned)(n * k));
        const int share = hi - lo > 4 ? 1 : hi - lo > 2 ? 2 : hi - lo > 1 ? 4 : 8;  // warps of a row
        const int part = warp & (share - 1);
        if (!waited) {
            grid_dependency_wait();
            waited = true;
        }
        for (int r0 = lo; r0 < hi; r0 += 8 / share) {
            const int r = r0 + warp / share;
            const bool in = r < hi;
            const size_t base = (size_t)member * 2 * p.ranges * block_rows + (in ? r : lo);
            float acc[V], s = 0.f, m = kNegInf;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            for (int c0 = part; c0 < n; c0 += share * NP) {
                float w[NP], v[NP][V], top = m;
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                    const int c = c0 + u * share;
                    w[u] = kNegInf;
#pragma unroll
                    for (int i = 0; i < V; ++i) v[u][i] = 0.f;
                    if (c >= n) continue;
                    const size_t at = base + (size_t)paged_slot(p, first + c, c == 0) * block_rows;
                    w[u] = p.lse_part[at];
#pragma unroll
                    for (int i = 0; i < V; i += Vec) load_vec<Vec>(v[u] + i, p.o_part + at * D + i * 32 + lane * Vec);
                }
#pragma unroll
                for (int u = 0; u < NP; ++u) top = fmaxf(top, w[u]);
                const float ref = top == kNegInf ? 0.f : top;
                const float f = ex2_approx((m - ref) * (1.f / kPagedLn2));
                m = top;
                s *= f;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                    const float x = ex2_approx((w[u] - ref) * (1.f / kPagedLn2));
                    s += x;
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = fmaf(x, v[u][i], acc[i]);
                }
            }
            if (share > 1) {
                __syncthreads();  // the rows before have been read
#pragma unroll
                for (int i = 0; i < V; ++i) s_acc[warp][i / Vec * Vec * 32 + lane * Vec + i % Vec] = acc[i];
                if (lane == 0) {
                    s_sum[warp] = s;
                    s_max[warp] = m;
                }
                __syncthreads();
                if (part != 0) continue;
                for (int w = 1; w < share; ++w) m = fmaxf(m, s_max[warp + w]);
                s = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = 0.f;
                const float ref = m == kNegInf ? 0.f : m;
                for (int w = 0; w < share; ++w) {
                    const float f = ex2_approx((s_max[warp + w] - ref) * (1.f / kPagedLn2));
                    s += f * s_sum[warp + w];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        acc[i] = fmaf(f, s_acc[warp + w][i / Vec * Vec * 32 + lane * Vec + i % Vec], acc[i]);
                }
            }
            if (!in) continue;
            const int tok_l = r / p.group, h = seg.hk * p.group + r - tok_l * p.group, tok = tok0 + tok_l;
            const float inv = 1.f / s;  // s == 0: no piece holds a visible key
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = s == 0.f ? 0.f : acc[i] * inv;
            uint16_t* out = static_cast<uint16_t*>(p.o) + (((size_t)seg.b * p.Sq + tok) * p.Hq + h) * D + lane * Vec;
#pragma unroll
            for (int i = 0; i < V; i += Vec) {
                if constexpr (Vec == 1)
                    out[i * 32] = float_to16<kBF16>(acc[i]);
                else if constexpr (Vec == 2)
                    *reinterpret_cast<uint32_t*>(out + i * 32) = pack2<kBF16>(acc[i], acc[i + 1]);
                else
                    *reinterpret_cast<uint2*>(out + i * 32) =
                        make_uint2(pack2<kBF16>(acc[i], acc[i + 1]), pack2<kBF16>(acc[i + 2], acc[i + 3]));
            }
            if (p.lse && lane == 0)
                p.lse[((size_t)seg.b * p.Hq + h) * p.Sq + tok] = s == 0.f ? kNegInf : m + lg2_approx(s) * kPagedLn2;
        }
    }
    // No CTA may be done before the split kernel is: the next kernel's wait is for this one.
    if (!waited) grid_dependency_wait();
}

template <class C>
fa_status launch_paged_merge(const PagedDecParams& p, bool bf16, cudaStream_t s) {
    static int attr[64] = {0};
    if (!prefer_shared((const void*)paged_merge_kernel<C, true>, (const void*)paged_merge_kernel<C, false>, attr))
        return FA_ERR_CUDA;
    const unsigned grid = (unsigned)(p.ranges * p.g * p.rg * p.merge_ctas);
    const size_t smem = C::plan_bytes(p.B);
    return bf16 ? launch_overlapped(paged_merge_kernel<C, true>, grid, 256, smem, s, p)
                : launch_overlapped(paged_merge_kernel<C, false>, grid, 256, smem, s, p);
}

template <class C, bool kBF16>
fa_status launch_paged_split(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedDecParams& p, cudaStream_t s) {
    static int attr[64] = {0};
    if (!ensure_smem_attr((const void*)paged_split_kernel<C, kBF16>, C::kFixedBytes + C::plan_bytes(kPagedMaxB), attr))
        return FA_ERR_CUDA;
    return launch_overlapped(paged_split_kernel<C, kBF16>, (unsigned)(p.ranges * p.g * p.rg), C::kThreads,
                             C::kFixedBytes + C::plan_bytes(p.B), s, tq, tk, tv, p);
}

template <class C>
fa_status launch_paged_cfg(const PagedDecodeArgs& a, cudaStream_t s) {
    constexpr int D = C::D, NQ = C::NQ;
    PagedDecParams p;
    p.B = a.B, p.Sq = a.Sq, p.Hq = a.Hq, p.Hkv = a.Hkv;
    p.group = a.Hq / a.Hkv;
    p.T = std::min(a.Sq, C::BM / p.group);
    p.row_blocks = (a.Sq + NQ * p.T - 1) / (NQ * p.T);
    p.g = a.Hkv % 8 == 0 ? 8 : a.Hkv % 4 == 0 ? 4 : a.Hkv % 2 == 0 ? 2 : 1;
    p.rg = p.g * p.row_blocks <= 16 ? p.row_blocks : 1;
    const int G = p.g * p.rg;
    if (G > a.num_sms) return FA_ERR_UNSUPPORTED;
    p.groups = a.Hkv / p.g;
    p.blocks = p.row_blocks / p.rg;
    p.capacity = a.page_size * a.max_pages;
    p.page_size = a.page_size, p.num_pages = a.num_pages, p.max_pages = a.max_pages;
    // Rows of a copy: a tile's where its keys lie side by side, a strip's where a window may begin with
    // any of them; and the power of two that a page is made of.
    p.box_rows = std::min(a.page_size & -a.page_size, a.window_left >= 0 ? 32 : C::BN);
    p.nb_log = 0;
    while (p.box_rows << p.nb_log < C::BN) ++p.nb_log;
    p.page_recip = (unsigned)((1ull << 32) / (unsigned)a.page_size) + 1u;
    p.window_left = a.window_left, p.sinks = a.sinks;
    p.words = (a.Sq + 31) / 32;
    p.table = a.table, p.kv_lens = a.kv_lens, p.tree = a.tree;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.o = a.o, p.lse = a.lse, p.o_part = a.o_part, p.lse_part = a.lse_part;
    p.v_pages = static_cast<const uint16_t*>(a.v_pages);
    p.status = a.dev_status;
    // The most tiles that a sequence can have.
    long long strips = ((long long)p.capacity + 31) / 32;
    if (a.window_left >= 0)
        strips = std::min(strips, ((long long)a.window_left + a.Sq + 31) / 32 + 1 + ((long long)a.sinks + 31) / 32);
    const long long most = (strips + C::BN / 32 - 1) / (C::BN / 32);
    const long long units = (most + C::Lead) * (p.groups * p.blocks) * a.B;  // of all entries at most
    if (units > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    p.whole = most + C::Lead <= C::MinWidth ? 1 : 0;
    p.ranges = (int)std::min((long long)(a.num_sms / G), (units + C::MinWidth - 1) / C::MinWidth);
    // A row takes a warp two trips to L2, so more rows are taken by more CTAs.  Measured (us) with at most 3, 4
    // and 8: 26 drafts of 4 heads 92.9, 92.2, 93.4, 64 drafts 91.5, 87.6, 89.0.
    p.merge_ctas = std::max(1, std::min(4, std::min(NQ * p.T, p.Sq) * p.group / 16));
    CUtensorMap tq, tk, tv;
    if (!encode_paged_tmap(&tq, a.q, a.bf16, D, a.Hq, a.Sq, a.B, p.group, p.T) ||
        !encode_paged_tmap(&tk, a.k_pages, a.bf16, D, a.Hkv, a.page_size, a.num_pages, 1, p.box_rows) ||
        !encode_paged_tmap(&tv, a.v_pages, a.bf16, D, a.Hkv, a.page_size, a.num_pages, 1, p.box_rows))
        return FA_ERR_CUDA;
    const fa_status st = a.bf16 ? launch_paged_split<C, true>(tq, tk, tv, p, s)
                                : launch_paged_split<C, false>(tq, tk, tv, p, s);
    if (st != FA_OK || p.whole) return st;
    return launch_paged_merge<C>(p, a.bf16, s);
}

// Rows that are few go with the products turned round.  Two sub-tiles share each key tile where one
// does not hold a kv head's rows (at D = 256 TMEM has room for one: row blocks then share the keys
// through L2).
template <int D>
fa_status launch_paged_decode_d(const PagedDecodeArgs& a, cudaStream_t s) {
    const int group = a.Hq / a.Hkv, rows = a.Sq * group;
    if constexpr (D != 256) {
        if (rows <= PagedFewCfg<D>::NR) return launch_paged_cfg<PagedFewCfg<D>>(a, s);
        if (a.Sq > 128 / group) return launch_paged_cfg<PagedCfg<D, 2>>(a, s);
    }
    return launch_paged_cfg<PagedCfg<D, 1>>(a, s);
}

}  // namespace fa
