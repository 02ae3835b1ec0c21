// fa_kv8_decode.cuh -- split-KV decode over the 8-bit paged cache.
//
// For sequence b, query token i of Sq and query head h (kv head hk = h / (Hq / Hkv)):
//     s_j = scale * 2^(ks_j - 127) * (q . kcode_j),   j visible: j < len_b, and with `causal`
//                                                     j <= len_b - Sq + i
//     o   = sum_j softmax(s)_j 2^(vs_j - 127) vcode_j,    lse = log sum_j exp(s_j)
//
// Plan: the keys of every (sequence, kv head) pair, in units of 64 keys, lie end to end in
// the order (b, hk), each pair led by kKv8Lead units that hold no keys and stand for what
// starting and finishing a pair costs.  CTA c takes the range of units [c W, (c + 1) W):
// every CTA gets the same work whatever the mix of lengths.  A pair whose keys lie in one
// range is finished by its CTA.  One that is cut leaves a partial output and its log-sum-exp
// in each range, which the merge kernel joins.  A range meets at most one pair that began
// before it and one that goes on behind it: the partial results fill a slot for each range
// and one more for each range or for each pair, whichever are fewer, whatever the number of
// pieces.  Without room for that (`whole`), a CTA takes the pairs that begin in its range, uncut.
// Where every sequence is short and there are many pairs (`solo`), each warp has a range of
// its own and takes whole pairs: a pair of a few tiles gives four warps little to share, and
// joining them costs as much as the tiles.
//
// What bounds it: each cached byte is read once and meets at most 16 query rows, so HBM does;
// the products are 16 % of the tensor pipe's time even as mma.sync, which takes its operands
// from registers.  That is why these are not tcgen05 products: codes have to become fp16 on
// the way (the probabilities and queries do not fit e4m3), and registers, where the
// conversion leaves them, are where mma.sync wants them, while tcgen05 would have them
// written back to shared memory first.  (K Q^T as e4m3 products, the queries in two or three
// e4m3 pieces, was right and needs no conversion of K, but slower: 62.7 -> 83.5 us for 8
// sequences of 700..16384 keys at D = 256 with 16 rows, 90 -> 107 us for the fp16 batch below.)
// So a warp works alone on a tile: it copies its own keys (cp.async, 98 KB in flight on an SM),
// and nothing but the end of a pair makes it wait for another warp.
//
// Measured (split and merge, back to back, inputs larger than L2): lengths 1024..32768 x 8
// sequences, 8 kv heads of 4 query heads, D = 128, 279 MB: 46.4 us, 6.0 TB/s, 89 % of a copy's
// rate; 64 sequences of 1..8192, 542 MB: 88.4 us, 6.1 TB/s, 90 %; 8 of U[1024, 32768] at D = 64, 96,
// 128, 256 with 158, 235, 313, 623 MB: 30.4, 44.5, 51.8, 99 us, 76, 78, 89, 92 %.  About 6.6 us of a
// call do not stream (one sequence of 32768: 16.6 us, 10.0 at a copy's rate).  A trace from before
// the plan came ahead of the wait (then 17.9) placed 7.9: 1.0 for the plan, 0.5 for the first table
// entries, 1.4 for the last join and about 1 of uneven ends, 2 for the merge kernel, 1 to pass
// from one kernel to the next and 1 to fill and drain the memory's queues.
#pragma once

#include <algorithm>

#include "fa_kv8.cuh"

namespace fa {

struct Kv8DecParams {
    Kv8Pool pool;
    const void* q;
    void* o;
    float* lse;
    const int32_t* kv_lens;
    float* o_part;    // [slots, group * Sq, D]
    float* lse_part;  // [slots, group * Sq]
    int B, Sq, Hq, group, capacity, causal, whole;
    int solo_keys;  // the longest sequence of a batch whose pairs warps take alone; 0: none
    int grid;  // ranges, and CTAs of the split kernel
    unsigned page_recip;  // floor(2^32 / page_size) + 1
    float scale_log2;
};

constexpr int kKv8Unit = 64;  // keys per unit of the plan
constexpr int kKv8Lead = 4;   // units charged to each pair beside its keys
constexpr int kKv8Threads = 128;
constexpr int kKv8Warps = kKv8Threads / 32;
constexpr int kKv8MaxB = 1024;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ int kv8_len(const Kv8DecParams& p, int b) {
    // Past L1: the merge reads it before the kernels before it are known to be done.
    return min(max(__ldcg(p.kv_lens + b), 0), p.capacity);
}

// Units of one pair of a sequence.
__device__ __forceinline__ int kv8_units(int len) {
    return len > 0 ? (len + kKv8Unit - 1) / kKv8Unit + kKv8Lead : 0;
}

// Whether warps take pairs alone, from the units of one pair of the longest sequence.
__device__ __forceinline__ bool kv8_solo(const Kv8DecParams& p, int max_units) {
    return p.solo_keys > 0 && max_units <= p.solo_keys / kKv8Unit + kKv8Lead;
}

// W for so many ranges, from the units of one pair of each sequence summed.
__device__ __forceinline__ int kv8_width(const Kv8DecParams& p, int sum_units, int ranges) {
    return max((int)(((unsigned)(p.pool.Hkv * sum_units) + (unsigned)ranges - 1u) / (unsigned)ranges), 1);
}

// The ranges that hold keys of the pair of `units` units beginning at unit `start`: the first
// of them, and how many.
__device__ __forceinline__ int kv8_first_piece(int start, int w) { return (start + kKv8Lead) / w; }
__device__ __forceinline__ int kv8_pieces(int start, int units, int w) {
    return units > 0 ? (start + units - 1) / w - kv8_first_piece(start, w) + 1 : 0;
}
// The slot of a pair's piece in range r, the first of its pieces or not.
__device__ __forceinline__ int kv8_slot(const Kv8DecParams& p, int r, bool first, int pair) {
    return !first ? r : p.grid + (p.grid <= p.B * p.pool.Hkv ? r : pair);
}

template <bool kBF16>
__device__ __forceinline__ uint16_t float_to16(float x) {
    return (uint16_t)(pack2<kBF16>(x, 0.f) & 0xffffu);
}

template <bool kBF16>
__device__ __forceinline__ float float_from16(uint16_t x) {
    if constexpr (kBF16) {
        return __uint_as_float((uint32_t)x << 16);
    } else {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(x));
        return f;
    }
}

// Sends for `bytes` bytes to L2 (a hint); both multiples of 16.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// The plan in shared memory: the units of one pair of each sequence summed over the
// sequences before b, and what the last unit of b lacks to be full, so that
// len = (units - kKv8Lead) * kKv8Unit - pad.
struct Kv8Plan {
    int* prefix;   // [B + 1]
    uint8_t* pad;  // [B]
    static __host__ __device__ constexpr int bytes(int B) { return (B + 1) * 4 + ((B + 15) & ~15); }
};

// Fills the plan from kv_lens (all threads; ends with a barrier); returns the units of one pair of
// the longest sequence.
__device__ __forceinline__ int kv8_make_plan(const Kv8DecParams& p, const Kv8Plan& t, int* warp_sum, int* warp_max) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.B + kKv8Threads - 1) / kKv8Threads;
    int sum = 0, most = 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            const int len = kv8_len(p, b), units = kv8_units(len);
            t.prefix[b] = units;
            t.pad[b] = (uint8_t)(len > 0 ? (units - kKv8Lead) * kKv8Unit - len : 0);
            sum += units;
            most = max(most, units);
        }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (lane == 31) {
        warp_sum[warp] = incl;
        warp_max[warp] = most;
    }
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < kKv8Warps; ++w) {
        if (w < warp) run += warp_sum[w];
        most = max(most, warp_max[w]);
    }
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            const int units = t.prefix[b];
            t.prefix[b] = run;
            run += units;
        }
    }
    if (threadIdx.x == kKv8Threads - 1) t.prefix[p.B] = run;
    __syncthreads();
    return most;
}

// Whether a length is no longer what the plan was made of (all threads; a barrier).
__device__ __forceinline__ bool kv8_plan_is_stale(const Kv8DecParams& p, const Kv8Plan& t) {
    bool stale = false;
    for (int b = threadIdx.x; b < p.B; b += kKv8Threads) {
        const int units = t.prefix[b + 1] - t.prefix[b];
        stale |= kv8_len(p, b) != (units > 0 ? (units - kKv8Lead) * kKv8Unit - t.pad[b] : 0);
    }
    return __syncthreads_or(stale);
}

// The part of one pair that lies in one range.
struct Kv8Seg {
    int b, hk, len, k0, k1;  // keys k0 .. k1 - 1 of `len`
    int slot;
    bool cut;
};

// Walks the segments of range `rng`, units x .. x_end - 1.
struct Kv8Walk {
    int x, x_end;
    int b, hk, start, units;  // the pair that holds unit x, or ends there
    bool whole;

    __device__ __forceinline__ void init(const Kv8DecParams& p, const Kv8Plan& t, int rng, int W, bool whole_) {
        whole = whole_;
        const int Hkv = p.pool.Hkv, total = Hkv * t.prefix[p.B];
        x = (int)min((long long)rng * W, (long long)total);
        x_end = (int)min((long long)x + W, (long long)total);
        if (x >= x_end) return;
        int lo = 0, hi = p.B;  // largest b with Hkv * prefix[b] <= x: it has keys
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (Hkv * t.prefix[mid] <= x) lo = mid; else hi = mid;
        }
        b = lo;
        units = t.prefix[lo + 1] - t.prefix[lo];
        hk = (x - Hkv * t.prefix[lo]) / units;
        start = Hkv * t.prefix[lo] + hk * units;
    }

    // The next segment; false where none is left.
    __device__ __forceinline__ bool next(const Kv8DecParams& p, const Kv8Plan& t, int rng, int W, Kv8Seg& s) {
        while (x < x_end) {
            if (x >= start + units) {
                start += units;
                if (++hk == p.pool.Hkv) {
                    hk = 0;
                    do {
                        ++b;
                        units = t.prefix[b + 1] - t.prefix[b];
                    } while (units == 0);
                }
            }
            if (whole && x > start) {  // the range before has it
                x = start + units;
                continue;
            }
            const int end = whole ? start + units : min(x_end, start + units);
            s.b = b;
            s.hk = hk;
            s.len = (units - kKv8Lead) * kKv8Unit - t.pad[b];
            s.k0 = max(x - start - kKv8Lead, 0) * kKv8Unit;
            s.k1 = min((end - start - kKv8Lead) * kKv8Unit, s.len);
            s.slot = kv8_slot(p, rng, rng == kv8_first_piece(start, W), b * p.pool.Hkv + hk);
            s.cut = !whole && kv8_pieces(start, units, W) > 1;
            x = end;
            if (s.k1 > s.k0) return true;  // else the range ends within the lead
        }
        return false;
    }
};

// What the warps of a CTA tell one another about each query row, and of the plan.
struct Kv8Small {
    float mo[kKv8Warps][16], ms[kKv8Warps][16], l[kKv8Warps][16];
    float f[16], finv[16], lse[16], qf[16];
    int warp_sum[kKv8Warps], warp_max[kKv8Warps];
};

// ------------------------------------------------------------------ shared layout ----
// Each warp streams its own tiles of KT keys through a ring of NST stages in shared memory:
// K codes and V codes, and the scales of both beside the ring.  A row is split into a part of
// WA bytes and, at D = 96, one of 32; each part's rows lie in 128-byte lines whose 16-byte
// units are permuted so that the reads below, K by (row g, unit t) and V by (row 2 t, unit g),
// meet no bank twice.
//
// HB: query rows in blocks of four (1, 2 or 4 blocks; a row is a (token, head) of one kv head).
//
// KT x NST x CTAS were measured (us): D = 128, two batches, 32 x 2 x 3 48.7 and 89.6, 16 x 4 x 3
// 51.0 and 91.6, 16 x 3 x 4 50.9 and 91.4, 32 x 3 x 2 49.2 and 98.3: three CTAs cover each other's
// joins.  D = 64: 32 x 3 20.6, 32 x 4 21.0, 64 x 2 20.9.  D = 96: 32 x 2 20.7, 16 x 5 21.8.  At D = 256 and
// with 16 query rows the registers allow two CTAs; three at D = 96 spill and take 41.9 for 37.3.
// A CTA more or less on an SM is worth more than a stage or a buffer: 5 to 8 rows at D = 256 (8 of
// 700..16384 keys) take 67.8 us with three stages in one CTA and 59.9 with two in two; at D = 128 (256 of
// 100..1000 keys, 8 kv heads) 95 with two buffers of the exchange and 70.5 with one.
template <int D_, int HB_>
struct Kv8Cfg {
    static constexpr int D = D_, HB = HB_;
    static constexpr int NT = (HB + 1) / 2;     // 8-column blocks of P
    static constexpr int E = HB == 1 ? 1 : 2;   // columns of a lane in use
    static constexpr int KT = D == 256 ? 16 : 32;
    static constexpr int NST = D == 64 || (D == 256 && HB == 1) ? 3 : 2;
    static constexpr int CTAS = D == 256 || NT == 2 ? 2 : 3;  // resident on an SM
    static constexpr int NSUB = KT / 16;  // runs of 16 keys
    static constexpr int TileBytes = KT * D;
    static constexpr int RingBytes = NST * 2 * TileBytes;  // a warp's
    static constexpr int ScaleBytes = NST * 2 * KT;
    // Row of the exchange in floats: pair (block k, row g) of dims at 2 (8 k + g); a half-warp's
    // 4 g and 4 t, one query row apart, then lie in 32 different banks.
    static constexpr int XD = D + 8;
    static constexpr int Bufs = D == 128 && HB == 2 ? 1 : 2;   // one where a third CTA fits with it
    static constexpr int ExchBytes = Bufs * HB * 4 * XD * 4;
    // Query fragments stay in registers or, where they are too many, in shared memory; they are
    // made there, in the exchange's room if they do not stay.
    static constexpr bool QRegs = D / 16 * NT <= 16;
    static constexpr int QLanes = 16 * E;  // lanes that hold a query fragment: with E = 1 those of even g
    static constexpr int QStage = D / 16 * NT * QLanes * 8;
    static constexpr int QBytes = QRegs ? 0 : QStage;
    static_assert(!QRegs || QStage <= ExchBytes, "queries fit the exchange");
    static constexpr int FixedBytes = 128 + kKv8Warps * (RingBytes + ScaleBytes) + ExchBytes + QBytes;
    // CTAs that are resident on an SM with the plan of B sequences: 228 KB, less 1 KB for each.
    static int resident(int B) {
        const int each = (FixedBytes + Kv8Plan::bytes(B) + (int)sizeof(Kv8Small) + 127) / 128 * 128;
        const int fit = 228 * 1024 / (each + 1024);
        return fit < CTAS ? fit : CTAS;
    }
    static constexpr int WA = D == 96 ? 64 : D;
    static constexpr int KS = D / 16;        // steps of 16 dims, and 16-dim blocks of O^T
    static constexpr int Copies = D / 32;    // 16-byte copies of a lane per run and tensor
    // Byte offset of 16-byte unit c of row `row` in a tile of codes.
    static __device__ __forceinline__ uint32_t unit(int row, int c) {
        if constexpr (WA == 64) {
            if (D == 96 && c >= 4) {
                const int line = row >> 2;
                return KT * 64 + line * 128 + ((((row & 3) * 2 + c - 4) ^ ((line & 1) * 2)) * 16);
            }
            const int line = row >> 1;
            return line * 128 + ((((row & 1) * 4 + c) ^ ((line & 3) * 2)) * 16);
        } else {
            return row * WA + (c >> 3) * 128 + (((c & 7) ^ ((row & 1) * 4) ^ (((row >> 1) & 3) * 2)) * 16);
        }
    }
    // What 16 rows add to it.
    static __device__ __forceinline__ uint32_t run_step(int c) {
        return D == 96 && c >= 4 ? 512 : 16 * WA;
    }
    // The first of the two dims whose sums a lane of row g holds in block k of O^T; it has them in
    // o[k][.][e] and o[k][.][2 + e].
    static __device__ __forceinline__ int dim(int k, int g) {
        if constexpr (WA == 64)
            return k < 4 ? g * 8 + k * 2 : 64 + g * 4 + (k - 4) * 2;
        else
            return (k >> 3) * 128 + g * 16 + (k & 7) * 2;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}

// The four codes of a word as two f16 pairs.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = e4m3x2_to_f16x2((uint16_t)(w & 0xffffu));
    hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
}

// Whether one of a word's codes is NaN: all seven bits below its sign.
__device__ __forceinline__ bool has_nan(uint32_t w) {
    return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// D(16 x 8) += A(16 x 16) B(16 x 8), f16 in, fp32 out.  Lane 4 g + t holds A rows g, g + 8 at
// columns 2 t, 2 t + 1 (a0, a1) and 2 t + 8, 2 t + 9 (a2, a3); B column g at the same rows (b0,
// b1); D rows g (c0, c1) and g + 8 (c2, c3) at columns 2 t, 2 t + 1.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held as above (row g, columns 2 t, 2 t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

// P is taken 2^kPShift times its value, and its reference may lag the true maximum by
// kPSlack: P <= 2^15 in fp16, and what falls below fp16's least subnormal, 2^-24, is 2^-35 of
// the largest weight.
constexpr float kPShift = 11.f, kPSlack = 4.f;
constexpr float kLowest = -3.402823466e38f;

// Query row c (token * group + head) of the kv head belongs to block c / 4; lane t of four has
// rows 4 hb + t of the blocks hb = 2 nt + e, e < E.
template <int D, int HB, bool kBF16>
__global__ void __launch_bounds__(kKv8Threads, Kv8Cfg<D, HB>::CTAS) kv8_split_kernel(const Kv8DecParams p) {
    using C = Kv8Cfg<D, HB>;
    constexpr int KT = C::KT, NSUB = C::NSUB, NST = C::NST, KS = C::KS, XD = C::XD, NT = C::NT, E = C::E;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Kv8Small sm;
    auto &s_mo = sm.mo, &s_ms = sm.ms, &s_l = sm.l;
    auto &s_f = sm.f, &s_finv = sm.finv, &s_lse = sm.lse, &s_qf = sm.qf;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const float kNegInf = -__int_as_float(0x7f800000);
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    const uint32_t ring = base + warp * C::RingBytes;
    const uint32_t scales = base + kKv8Warps * C::RingBytes + warp * C::ScaleBytes;
    uint8_t* rest = smem_raw + (base - raw) + kKv8Warps * (C::RingBytes + C::ScaleBytes);
    float* exch = reinterpret_cast<float*>(rest);
    Kv8Plan plan;
    plan.prefix = reinterpret_cast<int*>(rest + C::ExchBytes + C::QBytes);
    plan.pad = reinterpret_cast<uint8_t*>(plan.prefix + p.B + 1);

    const int Hkv = p.pool.Hkv, cols = p.group * p.Sq;
    // A group of gw warps works through a range; this is warp wi of it.
    bool solo;
    int gw, wi, rng, W;
    Kv8Walk lw, cw;  // the loader's and the products'
    auto make_plan = [&]() {
        const int most = kv8_make_plan(p, plan, sm.warp_sum, sm.warp_max);
        solo = C::QRegs && kv8_solo(p, most);
        gw = solo ? 1 : kKv8Warps;
        wi = solo ? 0 : warp;
        rng = solo ? (int)blockIdx.x * kKv8Warps + warp : (int)blockIdx.x;
        W = kv8_width(p, plan.prefix[p.B], solo ? p.grid * kKv8Warps : p.grid);
        lw.init(p, plan, rng, W, p.whole || solo);
    };
    // The 16-key run of the pool that holds keys key .. key + 15 of a segment: -1 where there is none
    // (behind k1, or a page outside the pool).
    auto run_of = [&](const Kv8Seg& s, int key, bool early) -> int {
        if (key >= s.k1) return -1;
        // key / page_size: the reciprocal, rounded up, gives the quotient or one more
        unsigned pi = __umulhi((unsigned)key, p.page_recip);
        int slot = (int)((unsigned)key - pi * (unsigned)p.pool.page_size);
        if (slot < 0) {
            --pi;
            slot += p.pool.page_size;
        }
        const int* at = p.pool.table + (size_t)s.b * p.pool.max_pages + pi;
        const int page = early ? __ldcg(at) : *at;
        if (page < 0 || page >= p.pool.num_pages) return -1;
        return (page * Hkv + s.hk) * (p.pool.page_size / 16) + slot / 16;
    };
    // While the kernel before may still be running and the memory idles: the plan, and the warps'
    // first tiles are sent for to L2.  The lengths and the table may change until that kernel is
    // done, so this is a guess: nothing but L2 lines depends on it, and the plan is made again if a
    // length is another afterwards.  Behind a kernel that lets this one start early (this library's;
    // others' are done by then) it saves 0.4 us by the plan and 0.9 by the tiles: one sequence of
    // 32768 17.9 -> 16.6 us, the lengths 1024..32768 47.9 -> 46.4, each behind a decode.  Behind an
    // append of one token a sequence, the pair takes 0.9 us more than append and decode do among
    // their own kind; behind a kernel that does not let this one start early, 1.8 (16.5 + 1.2 -> 19.5
    // us and 46.3 + 1.2 -> 49.9 for an elementwise kernel).  More tiles: 16.6 with 2, 17.5 with 4;
    // for warps alone 12.8 us without and 13.5 with (2048 pairs of 64 keys).
    make_plan();
    {
        Kv8Walk guess = lw;
        Kv8Seg s;
        if (!solo && guess.next(p, plan, rng, W, s) && lane < NSUB) {
            const int run = run_of(s, s.k0 + wi * KT + lane * 16, true);
            if (run >= 0) {
                prefetch_l2(p.pool.k + (size_t)run * (16 * D), 16 * D);
                prefetch_l2(p.pool.v + (size_t)run * (16 * D), 16 * D);
                prefetch_l2(p.pool.ks + (size_t)run * 16, 16);
                prefetch_l2(p.pool.vs + (size_t)run * 16, 16);
            }
        }
    }
    grid_dependency_wait();
    if (kv8_plan_is_stale(p, plan)) make_plan();
    cw = lw;
    uint2* s_q = reinterpret_cast<uint2*>(C::QRegs ? rest : rest + C::ExchBytes);
    uint16_t* o16 = static_cast<uint16_t*>(p.o);
    const uint16_t* q16 = static_cast<const uint16_t*>(p.q);
    // This lane's 16-byte units of a run of 16 rows: unit i * 32 + lane of the run's 16 D bytes.
    uint32_t dst[C::Copies], step[C::Copies];
#pragma unroll
    for (int i = 0; i < C::Copies; ++i) {
        const int u = i * 32 + lane, row = u / (D / 16), c = u % (D / 16);
        dst[i] = ring + C::unit(row, c);
        step[i] = C::run_step(c);
    }

    // The loader walks the warp's tiles (wi, wi + gw, ... of each segment) up to NST - 1
    // ahead of the products, across the ends of segments.
    Kv8Seg ls;
    int lj = 0, ltiles = 0, run = -1;
    // Steps to the next tile and looks up run lane % NSUB of it.
    auto next_tile = [&]() {
        lj += gw;
        while (lj >= ltiles) {
            if (!lw.next(p, plan, rng, W, ls)) {
                ltiles = 0;
                lj = 0;
                grid_launch_dependents();  // only now: the merge's CTAs would take room from this grid's
                return;
            }
            ltiles = (ls.k1 - ls.k0 + KT - 1) / KT;
            lj = wi;
        }
        run = run_of(ls, ls.k0 + lj * KT + lane % NSUB * 16, false);
    };
    // Starts the copies of the loader's tile into stage st; rows without a key become zeros.
    auto issue = [&](int st) {
        const uint32_t ok = st * 2 * C::TileBytes, ov = ok + C::TileBytes;
#pragma unroll
        for (int s = 0; s < NSUB; ++s) {
            const int r = NSUB > 1 ? __shfl_sync(0xffffffffu, run, s) : run;
            const int left = ls.k1 - (ls.k0 + lj * KT + s * 16);
            const size_t off = (size_t)max(r, 0) * (16 * D) + lane * 16;
            const uint8_t *k = p.pool.k + off, *v = p.pool.v + off;
            if (r >= 0 && left >= 16) {
#pragma unroll
                for (int i = 0; i < C::Copies; ++i) {
                    cp_async16(dst[i] + ok + s * step[i], k + i * 512, 16);
                    cp_async16(dst[i] + ov + s * step[i], v + i * 512, 16);
                }
            } else {
                const int valid = r < 0 ? 0 : left * D;
#pragma unroll
                for (int i = 0; i < C::Copies; ++i) {
                    const int n = i * 512 + lane * 16 < valid ? 16 : 0;
                    cp_async16(dst[i] + ok + s * step[i], k + i * 512, n);
                    cp_async16(dst[i] + ov + s * step[i], v + i * 512, n);
                }
            }
        }
        if (lane < 2 * NSUB) {
            const uint8_t* src = (lane < NSUB ? p.pool.ks : p.pool.vs) + (size_t)max(run, 0) * 16;
            cp_async16(scales + st * 2 * KT + lane * 16, src, run < 0 ? 0 : 16);
        }
    };
    next_tile();
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) {
        if (lj < ltiles) {
            issue(i);
            next_tile();
        }
        cp_async_commit();
    }

    const int rows = p.Sq * p.Hq;
    for (int b = blockIdx.x; b < p.B; b += p.grid) {  // sequences without keys
        if (plan.prefix[b + 1] > plan.prefix[b]) continue;
        for (int i = tid; i < rows * D; i += kKv8Threads) o16[(size_t)b * rows * D + i] = 0;
        if (p.lse)
            for (int i = tid; i < rows; i += kKv8Threads) p.lse[(size_t)b * rows + i] = kNegInf;
    }

    // Queries as f16 fragments, column 2 t + e of block nt being row (2 nt + e) * 4 + t.  A row is
    // multiplied by a power of two that brings its largest magnitude to [2^13, 2^14).  fp16 has all
    // its 11 bits from 2^-14 on and steps of 2^-24 below, so bf16 and fp16 queries enter exactly
    // but for values under 2^-27 of their row's largest, which are off by 2^-38 of it at most.
    struct Factor {
        float up, down;  // the power of two, and softmax scale * log2 e over it
    };
    auto factor = [&](float amax) -> Factor {
        // amax = f 2^x; the factor is 2^(13 - x), from the exponent field, kept normal
        int ex = (int)(__float_as_uint(amax) >> 23);
        ex = ex == 255 ? 127 + 13 : max(ex, 14);
        return {__uint_as_float((uint32_t)(254 + 13 - ex) << 23),
                p.scale_log2 * __uint_as_float((uint32_t)(ex - 13) << 23)};
    };
    // Four warps: warp w makes rows w, w + 4, ... of a segment, a lane four dims at a time, in shared
    // memory; they are loaded while the segment before is joined.
    constexpr int QU = (D / 4 + 31) / 32;
    uint2 raw_q[HB][QU];
    auto load_queries = [&](const Kv8Seg& s) {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const int c = i * 4 + warp, tok = c / p.group, h = s.hk * p.group + c - tok * p.group;
            const uint16_t* src = q16 + (((size_t)s.b * p.Sq + tok) * p.Hq + h) * D;
#pragma unroll
            for (int k = 0; k < QU; ++k) {
                const int d = (lane + 32 * k) * 4;
                raw_q[i][k] = c < cols && d < D ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
            }
        }
    };
    auto make_fragments = [&]() {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            float x[QU][4], amax = 0.f;
#pragma unroll
            for (int k = 0; k < QU; ++k) {
                const uint32_t r[2] = {raw_q[i][k].x, raw_q[i][k].y};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[k][2 * e] = float_from16<kBF16>((uint16_t)r[e]);
                    x[k][2 * e + 1] = float_from16<kBF16>((uint16_t)(r[e] >> 16));
                    amax = fmaxf(amax, fmaxf(fabsf(x[k][2 * e]), fabsf(x[k][2 * e + 1])));
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const Factor fac = factor(amax);
            const float up = fac.up;
            if (lane == 0) s_qf[i * 4 + warp] = fac.down;
#pragma unroll
            for (int k = 0; k < QU; ++k) {
                const int d = (lane + 32 * k) * 4;
                const int ks = d < C::WA ? (d >> 6) * 4 + ((d >> 2) & 3) : 4 + ((d >> 2) & 1);
                const int tt = d < C::WA ? (d >> 4) & 3 : ((d - 64) >> 3) & 3;
                if (d < D)  // of lane 4 g + tt, g = 2 warp + i % 2
                    s_q[(ks * NT + (i >> 1)) * C::QLanes + (E * warp + (i & 1)) * 4 + tt] =
                        make_uint2(pack_f16x2(x[k][0] * up, x[k][1] * up), pack_f16x2(x[k][2] * up, x[k][3] * up));
            }
        }
    };
    // This lane's fragment: step ks, block nt.
    auto fragment = [&](int ks, int nt) -> uint2 {
        if constexpr (E == 2)
            return s_q[(ks * NT + nt) * C::QLanes + lane];
        else
            return (g & 1) == 0 ? s_q[(ks * NT + nt) * C::QLanes + (g >> 1) * 4 + t] : make_uint2(0, 0);
    };

    int st = 0;
    Kv8Seg sg;
    bool more = cw.next(p, plan, rng, W, sg);
    if (more && !solo) load_queries(sg);
    while (more) {
        const int b = sg.b, hk = sg.hk, len = sg.len, k0 = sg.k0, k1 = sg.k1;
        const int tiles = (k1 - k0 + KT - 1) / KT;

        uint2 qr[C::QRegs ? KS * NT : 1];
        float qf[NT][E];
        if (!solo) {
            make_fragments();
            __syncthreads();
            if constexpr (C::QRegs) {
#pragma unroll
                for (int i = 0; i < KS * NT; ++i) qr[i] = fragment(i / NT, i % NT);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) qf[nt][e] = s_qf[(nt * 2 + e) * 4 + t];
        } else if constexpr (C::QRegs) {
            // A warp alone: each lane loads what its fragments are made of.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int c = (nt * 2 + (g & 1)) * 4 + (g >> 1), tok = c / p.group;
                const bool in = c < cols && (g & 1) < E;
                const uint16_t* src = q16 + (((size_t)b * p.Sq + tok) * p.Hq + hk * p.group + c - tok * p.group) * D;
                uint2 w[KS];
                float amax = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int d = ks * 16 < C::WA ? (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 : 64 + t * 8 + (ks - 4) * 4;
                    w[ks] = in ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
                }
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(float_from16<kBF16>((uint16_t)w[ks].x)),
                                                   fabsf(float_from16<kBF16>((uint16_t)(w[ks].x >> 16)))),
                                             fmaxf(fabsf(float_from16<kBF16>((uint16_t)w[ks].y)),
                                                   fabsf(float_from16<kBF16>((uint16_t)(w[ks].y >> 16))))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const Factor fac = factor(amax);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    qr[ks * NT + nt] = make_uint2(pack_f16x2(float_from16<kBF16>((uint16_t)w[ks].x) * fac.up,
                                                             float_from16<kBF16>((uint16_t)(w[ks].x >> 16)) * fac.up),
                                                  pack_f16x2(float_from16<kBF16>((uint16_t)w[ks].y) * fac.up,
                                                             float_from16<kBF16>((uint16_t)(w[ks].y >> 16)) * fac.up));
#pragma unroll
                for (int e = 0; e < E; ++e) qf[nt][e] = __shfl_sync(0xffffffffu, fac.down, (2 * t + e) * 4);
            }
        }
        int lim[NT][E];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < E; ++e)
                lim[nt][e] = p.causal ? min(k1, len - p.Sq + ((nt * 2 + e) * 4 + t) / p.group + 1) : k1;
        const int full = p.causal ? min(k1, len - p.Sq + 1) : k1;  // keys that every row sees

        float o[KS][NT][4], ms[NT][E], mo[NT][E], l[NT][E];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int m = 0; m < KS; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][nt][i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ms[nt][e] = mo[nt][e] = kLowest;
                l[nt][e] = 0.f;
            }
        }

        for (int j = wi; j < tiles; j += gw) {
            cp_async_wait<NST - 2>();
            __syncwarp();
            if (lj < ltiles) {
                issue(st == 0 ? NST - 1 : st - 1);
                next_tile();
            }
            cp_async_commit();
            const uint32_t sk = ring + st * 2 * C::TileBytes, sv = sk + C::TileBytes, ss = scales + st * 2 * KT;
            st = st == NST - 1 ? 0 : st + 1;

            // S^T = K Q^T: 16 keys x 8 query rows at a time, the dims in an order that gives each
            // lane whole 16-byte units of its rows.
            float sc[NSUB][2][NT][E];  // keys g, g + 8 of a run
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                float acc[2][NT][4];  // two chains of dependent products
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[c][nt][i] = 0.f;
                auto steps = [&](int ks, uint32_t w0, uint32_t w1) {
                    uint32_t a0, a1, a2, a3;
                    codes4(w0, a0, a2);
                    codes4(w1, a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint2 q;
                        if constexpr (C::QRegs)
                            q = qr[ks * NT + nt];
                        else
                            q = fragment(ks, nt);
                        mma_16816(acc[ks & 1][nt], a0, a1, a2, a3, q.x, q.y);
                    }
                };
#pragma unroll
                for (int c = 0; c < C::WA / 64; ++c) {
                    uint32_t r0[4], r1[4];
                    lds128(sk + C::unit(s * 16 + g, c * 4 + t), r0);
                    lds128(sk + C::unit(s * 16 + g + 8, c * 4 + t), r1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) steps(c * 4 + i, r0[i], r1[i]);
                }
                if constexpr (D == 96) {
                    uint32_t r0[2], r1[2];
                    lds64(sk + C::unit(s * 16 + g, 4 + (t >> 1)) + (t & 1) * 8, r0[0], r0[1]);
                    lds64(sk + C::unit(s * 16 + g + 8, 4 + (t >> 1)) + (t & 1) * 8, r1[0], r1[1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) steps(4 + i, r0[i], r1[i]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int i = 0; i < 2; ++i) sc[s][i][nt][e] = acc[0][nt][i * 2 + e] + acc[1][nt][i * 2 + e];
            }

            // Softmax in base 2.  l: this lane's own sum of exp2(s - ms) (joined at the end); mo: the
            // reference of P = exp2(s + log2 V scale - mo), one for all lanes.  Both references
            // move only when a score passes them by a margin: ms by 2^64, which fp32 has room for,
            // mo by kPSlack.
            float lv[NSUB][2];
            bool grow = false;
            const bool masked = k0 + j * KT + KT > full;
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = s * 16 + g + i * 8, key = k0 + j * KT + r;
                    const float kf = kv8_scale(lds8(ss + r));
                    lv[s][i] = (float)((int)lds8(ss + KT + r) - 127);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            float& v = sc[s][i][nt][e];
                            v *= kf * qf[nt][e];
                            if (masked && key >= lim[nt][e]) v = kNegInf;
                            grow |= v + lv[s][i] > mo[nt][e] + kPSlack || v > ms[nt][e] + 64.f;
                        }
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float m = ms[nt][e], r = mo[nt][e];
#pragma unroll
                        for (int s = 0; s < NSUB; ++s) {
                            m = fmaxf(m, fmaxf(sc[s][0][nt][e], sc[s][1][nt][e]));
                            r = fmaxf(r, fmaxf(sc[s][0][nt][e] + lv[s][0], sc[s][1][nt][e] + lv[s][1]));
                        }
                        l[nt][e] *= ex2_approx(ms[nt][e] - m);
                        ms[nt][e] = m;
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, w));
                        const float f = ex2_approx(mo[nt][e] - r);
                        mo[nt][e] = r;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[k][nt][e] *= f;
                            o[k][nt][2 + e] *= f;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int s = 0; s < NSUB; ++s)
                        l[nt][e] += ex2_approx(sc[s][0][nt][e] - ms[nt][e]) + ex2_approx(sc[s][1][nt][e] - ms[nt][e]);

            // Keys that the mask hides from some rows have P = 0 there, which a NaN code of V would not
            // respect.  So a NaN among them is brought to the rows that see it, and becomes a zero.
            const int hidden = max(full - k0 - j * KT, 0), last = min(k1 - k0 - j * KT, KT);
            if (hidden < last) {
                bool bad = false;
                for (int i = hidden * (D / 16) + lane; i < last * (D / 16); i += 32) {
                    uint32_t w[4];
                    lds128(sv + C::unit(i / (D / 16), i % (D / 16)), w);
                    bad |= has_nan(w[0]) || has_nan(w[1]) || has_nan(w[2]) || has_nan(w[3]);
                }
                if (__any_sync(0xffffffffu, bad)) {
                    for (int r = hidden; r < last; ++r)
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int d = C::dim(k, g) + i;
                                if ((lds8(sv + C::unit(r, d / 16) + d % 16) & 0x7f) != 0x7f) continue;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int e = 0; e < E; ++e)
                                        if (k0 + j * KT + r < lim[nt][e])
                                            o[k][nt][2 * i + e] = __int_as_float(0x7fffffff);
                            }
                    __syncwarp();
                    for (int i = hidden * D + lane; i < last * D; i += 32) {
                        const uint32_t at = sv + C::unit(i / D, i % D / 16) + i % 16;
                        if ((lds8(at) & 0x7f) == 0x7f) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(0) : "memory");
                    }
                    __syncwarp();
                }
            }

            // O^T += V^T P^T: 16 dims x 8 query rows over 16 keys.  A lane's units of keys 2 t,
            // 2 t + 1 (and + 8) are interleaved into pairs of keys.
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v[2] = {0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            v[e] = ex2_approx((sc[s][i][nt][e] + lv[s][i]) - (mo[nt][e] - kPShift));
                        pb[nt][i] = transpose8x8(pack_f16x2(v[0], v[1]));
                    }
                // words of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9: dims 4 i .. 4 i + 3 of the unit
                auto steps = [&](int m, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
                    uint32_t a[2][4];  // [16-dim block][a0..a3]
                    codes4(__byte_perm(r0, r1, 0x5140), a[0][0], a[0][1]);
                    codes4(__byte_perm(r0, r1, 0x7362), a[1][0], a[1][1]);
                    codes4(__byte_perm(r2, r3, 0x5140), a[0][2], a[0][3]);
                    codes4(__byte_perm(r2, r3, 0x7362), a[1][2], a[1][3]);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816(o[m + u][nt], a[u][0], a[u][1], a[u][2], a[u][3], pb[nt][0], pb[nt][1]);
                };
                const int r = s * 16 + 2 * t;
                if constexpr (C::WA == 64) {
                    uint32_t w[4][2];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        lds64(sv + C::unit(r + (i >> 1) * 8 + (i & 1), g >> 1) + (g & 1) * 8, w[i][0], w[i][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) steps(2 * i, w[0][i], w[1][i], w[2][i], w[3][i]);
                } else {
#pragma unroll
                    for (int c = 0; c < C::WA / 128; ++c) {
                        uint32_t w[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            lds128(sv + C::unit(r + (i >> 1) * 8 + (i & 1), c * 8 + g), w[i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) steps(c * 8 + 2 * i, w[0][i], w[1][i], w[2][i], w[3][i]);
                    }
                }
                if constexpr (D == 96) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = lds32(sv + C::unit(r + (i >> 1) * 8 + (i & 1), 4 + (g >> 2)) + (g & 3) * 4);
                    steps(4, w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();  // the stage may be overwritten
        }

        const Kv8Seg done = sg;
        more = cw.next(p, plan, rng, W, sg);
        if (more && !solo) load_queries(sg);

        // Per query row the maxima and sums over the lanes of one t.
        float m_all[NT][E], sum_all[NT][E];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float m = ms[nt][e];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                float sum = l[nt][e] * ex2_approx(ms[nt][e] - m);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                m_all[nt][e] = m;
                sum_all[nt][e] = sum;
            }
        // O = (sum of the outputs) 2^(Mo - kPShift - Ms) / L.  The power is taken in two halves, f and
        // f / L: V scales go down to 2^-127.  L = 0: no visible key, and O = 0.
        auto half_power = [](float Mo, float Ms) { return ex2_approx((Mo - kPShift - Ms) * 0.5f); };
        auto log_sum = [](float Ms, float L) {
            return L == 0.f ? -__int_as_float(0x7f800000) : (Ms + lg2_approx(L)) * kLn2;
        };
        if (solo) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int col = (nt * 2 + e) * 4 + t;
                    if (col >= cols) continue;
                    const float L = sum_all[nt][e], f = half_power(mo[nt][e], m_all[nt][e]);
                    const float finv = L == 0.f ? 0.f : f / L;
                    const int tok = col / p.group, h = hk * p.group + col % p.group;
                    const size_t row = ((size_t)b * p.Sq + tok) * p.Hq + h;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const int d = C::dim(k, g);
                        *reinterpret_cast<uint32_t*>(o16 + row * D + d) =
                            pack2<kBF16>(o[k][nt][e] * finv * f, o[k][nt][2 + e] * finv * f);
                    }
                    if (g == 0 && p.lse)
                        p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = log_sum(m_all[nt][e], L);
                }
            __syncwarp();  // before the next pair's queries
            continue;
        }
        // Join the four warps through shared memory; the outputs, brought to one reference, are added
        // up in a buffer or two, by one or two warps at a time.
        if (g == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int col = (nt * 2 + e) * 4 + t;
                    s_mo[warp][col] = mo[nt][e];
                    s_ms[warp][col] = m_all[nt][e];
                    s_l[warp][col] = sum_all[nt][e];
                }
        }
        __syncthreads();
        auto leave = [&](bool add) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int col = (nt * 2 + e) * 4 + t;
                    if (col >= cols) continue;
                    float m = s_mo[0][col];
#pragma unroll
                    for (int w = 1; w < kKv8Warps; ++w) m = fmaxf(m, s_mo[w][col]);
                    const float f = ex2_approx(mo[nt][e] - m);
                    float* row = exch + (warp % C::Bufs * HB * 4 + col) * XD;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        float2* at = reinterpret_cast<float2*>(row) + k * 8 + g;
                        float2 v = make_float2(o[k][nt][e] * f, o[k][nt][2 + e] * f);
                        if (add) {
                            const float2 u = *at;
                            v = make_float2(u.x + v.x, u.y + v.y);
                        }
                        *at = v;
                    }
                }
        };
        if (warp < C::Bufs && warp < tiles) leave(false);
        if (tid >= 64 && tid < 64 + cols) {
            const int col = tid - 64;
            float Mo = s_mo[0][col], Ms = s_ms[0][col], L = 0.f;
#pragma unroll
            for (int w = 1; w < kKv8Warps; ++w) {
                Mo = fmaxf(Mo, s_mo[w][col]);
                Ms = fmaxf(Ms, s_ms[w][col]);
            }
#pragma unroll
            for (int w = 0; w < kKv8Warps; ++w) L = fmaf(ex2_approx(s_ms[w][col] - Ms), s_l[w][col], L);
            const float f = half_power(Mo, Ms);
            s_f[col] = f;
            s_finv[col] = L == 0.f ? 0.f : f / L;
            s_lse[col] = log_sum(Ms, L);
        }
        __syncthreads();
#pragma unroll
        for (int w = C::Bufs; w < kKv8Warps; w += C::Bufs)
            if (tiles > w) {  // else warp w and those behind it had none
                if (warp >= w && warp < w + C::Bufs && warp < tiles) leave(true);
                __syncthreads();
            }
        for (int i = tid; i < cols * (D / 2); i += kKv8Threads) {
            // Pair u of dims is block k, row g of the products; four threads of one g take
            // neighbouring pairs.
            const int col = i / (D / 2), u = i % (D / 2);
            int k, gg;
            if constexpr (C::WA == 64) {
                k = u < 32 ? u & 3 : 4 + (u & 1);
                gg = u < 32 ? u >> 2 : (u - 32) >> 1;
            } else {
                k = (u & 3) + (u >> 5) * 4;
                gg = (u >> 2) & 7;
            }
            const int d = C::dim(k, gg);
            const float2 v0 = *reinterpret_cast<const float2*>(exch + col * XD + (k * 8 + gg) * 2);
            const float2 v1 = C::Bufs > 1 && tiles > 1
                                  ? *reinterpret_cast<const float2*>(exch + (HB * 4 + col) * XD + (k * 8 + gg) * 2)
                                  : make_float2(0.f, 0.f);
            const float f = s_f[col], finv = s_finv[col];
            const float a0 = (v0.x + v1.x) * finv * f, a1 = (v0.y + v1.y) * finv * f;
            const int tok = col / p.group, h = hk * p.group + col % p.group;
            const size_t row = ((size_t)b * p.Sq + tok) * p.Hq + h;
            if (!done.cut) {
                *reinterpret_cast<uint32_t*>(o16 + row * D + d) = pack2<kBF16>(a0, a1);
                if (d == 0 && p.lse) p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = s_lse[col];
            } else {
                const size_t part = (size_t)done.slot * cols + col;
                *reinterpret_cast<float2*>(p.o_part + part * D + d) = make_float2(a0, a1);
                if (d == 0) p.lse_part[part] = s_lse[col];
            }
        }
        __syncthreads();  // before the next segment's exchange
    }
}

template <int D, int HB, bool kBF16>
fa_status launch_kv8_split(const Kv8DecParams& p, cudaStream_t s) {
    using C = Kv8Cfg<D, HB>;
    static int attr[64] = {0};
    constexpr int most = C::FixedBytes + Kv8Plan::bytes(kKv8MaxB);
    static_assert(most <= 227 * 1024 - 1536, "shared memory of a CTA");
    if (!ensure_smem_attr((const void*)kv8_split_kernel<D, HB, kBF16>, most, attr)) return FA_ERR_CUDA;
    return launch_overlapped(kv8_split_kernel<D, HB, kBF16>, p.grid, kKv8Threads,
                             C::FixedBytes + Kv8Plan::bytes(p.B), s, p);
}

// An SM divides its memory into L1 and shared memory anew only when it is idle: a kernel that
// prefers L1, still resident, would keep the split kernel's CTAs from fitting beside it.
inline bool prefer_shared(const void* f, const void* g, int* done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) return true;
    for (const void* k : {f, g})
        if (cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
            return false;
    __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
    return true;
}

template <int N>
__device__ __forceinline__ void load_vec(float* v, const float* p) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else if constexpr (N == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x, v[1] = x.y;
    } else {
        v[0] = *p;
    }
}

// Joins the pieces of each row (b, token, head): lse = log sum_c exp(lse_c), and the outputs
// weighted with exp(lse_c - lse).  WPR warps share a row, each taking every WPR-th piece; a
// lane holds D / 32 dims.  It moves few bytes: its time is the launch and the dependent trips
// to L2.  So where the pieces lie is worked out before the split kernel is done (kv_lens is
// older than that kernel), and a warp then loads the log-sum-exps and outputs of NB pieces
// together.
template <int D, int WPR, bool kBF16>
__global__ void __launch_bounds__(256) kv8_merge_kernel(const Kv8DecParams p) {
    constexpr int V = D / 32, Rows = 8 / WPR, NB = V <= 4 ? 8 : 4;
    constexpr int Vec = V % 4 == 0 ? 4 : V % 2 == 0 ? 2 : 1;  // values of a lane side by side
    __shared__ __align__(16) float s_acc[WPR > 1 ? 8 : 1][D];
    __shared__ float s_sum[8], s_max[8];
    __shared__ int s_units[kKv8MaxB];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * Rows + warp / WPR, part = warp % WPR;
    const float kNegInf = -__int_as_float(0x7f800000);
    const int b = row / (p.Sq * p.Hq), tok = row / p.Hq % p.Sq, h = row % p.Hq;
    for (int i = threadIdx.x; i < p.B; i += 256) s_units[i] = kv8_units(kv8_len(p, i));
    __syncthreads();
    int before = 0, sum = 0, units = 0, most = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int t = s_units[i];
        before += i < b ? t : 0;
        units += i == b ? t : 0;
        sum += t;
        most = max(most, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        before += __shfl_xor_sync(0xffffffffu, before, o);
        units += __shfl_xor_sync(0xffffffffu, units, o);
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const int W = kv8_width(p, sum, p.grid), start = p.pool.Hkv * before + h / p.group * units;
    const int n = kv8_solo(p, most) ? 1 : kv8_pieces(start, units, W), first = kv8_first_piece(start, W);
    const int cols = p.group * p.Sq, col = tok * p.group + h % p.group;
    const int pair = b * p.pool.Hkv + h / p.group;
    grid_launch_dependents();
    grid_dependency_wait();
    // Rows with one piece or none have been written by the split kernel.  n is the same in all of
    // a row's warps.
    if (row >= p.B * p.Sq * p.Hq || n < 2) return;
    float acc[V], s = 0.f, m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int c0 = part; c0 < n; c0 += WPR * NB) {
        float w[NB], v[NB][V], top = m;
#pragma unroll
        for (int u = 0; u < NB; ++u) {  // pieces past n: the last one, with weight 0
            const int c = min(c0 + u * WPR, n - 1);
            const size_t at = (size_t)kv8_slot(p, first + c, c == 0, pair) * cols + col;
            w[u] = p.lse_part[at];
#pragma unroll
            for (int i = 0; i < V; i += Vec) load_vec<Vec>(v[u] + i, p.o_part + at * D + i * 32 + lane * Vec);
        }
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            if (c0 + u * WPR >= n) w[u] = kNegInf;
            top = fmaxf(top, w[u]);
        }
        const float ref = top == kNegInf ? 0.f : top;
        const float f = ex2_approx((m - ref) * (1.f / kLn2));
        m = top;
        s *= f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            const float e = ex2_approx((w[u] - ref) * (1.f / kLn2));
            s += e;
            // a weight of 0 must not meet a NaN or an infinity of a piece read twice
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(e, w[u] == kNegInf ? 0.f : v[u][i], acc[i]);
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[warp][i / Vec * Vec * 32 + lane * Vec + i % Vec] = acc[i];
        if (lane == 0) {
            s_sum[warp] = s;
            s_max[warp] = m;
        }
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int w = 1; w < WPR; ++w) m = fmaxf(m, s_max[w]);
        s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        const float ref = m == kNegInf ? 0.f : m;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float f = ex2_approx((s_max[w] - ref) * (1.f / kLn2));
            s += f * s_sum[w];
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] = fmaf(f, s_acc[w][i / Vec * Vec * 32 + lane * Vec + i % Vec], acc[i]);
        }
    }
    const float inv = 1.f / s;  // s == 0: no piece holds a visible key
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = s == 0.f ? 0.f : acc[i] * inv;
    uint16_t* out = static_cast<uint16_t*>(p.o) + (size_t)row * D + lane * Vec;
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
        p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = s == 0.f ? kNegInf : m + lg2_approx(s) * kLn2;
}

template <int D, int WPR>
fa_status launch_kv8_merge(const Kv8DecParams& p, bool bf16, cudaStream_t s) {
    static int attr[64] = {0};
    if (!prefer_shared((const void*)kv8_merge_kernel<D, WPR, true>, (const void*)kv8_merge_kernel<D, WPR, false>, attr))
        return FA_ERR_CUDA;
    const unsigned rows = (unsigned)(p.B * p.Sq * p.Hq), grid = (rows + 8 / WPR - 1) / (8 / WPR);
    return bf16 ? launch_overlapped(kv8_merge_kernel<D, WPR, true>, grid, 256, 0, s, p)
                : launch_overlapped(kv8_merge_kernel<D, WPR, false>, grid, 256, 0, s, p);
}

template <int D>
fa_status launch_kv8_decode_d(const Kv8DecodeArgs& a, cudaStream_t s) {
    Kv8DecParams p;
    p.pool = a.pool;
    p.q = a.q;
    p.o = a.o;
    p.lse = a.lse;
    p.kv_lens = a.kv_lens;
    p.o_part = a.o_part;
    p.lse_part = a.lse_part;
    p.B = a.B;
    p.Sq = a.Sq;
    p.Hq = a.Hq;
    p.group = a.Hq / a.pool.Hkv;
    p.capacity = a.pool.page_size * a.pool.max_pages;
    p.causal = a.causal ? 1 : 0;
    p.page_recip = (unsigned)((1ull << 32) / (unsigned)a.pool.page_size) + 1u;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    // As many ranges as CTAs are resident at once, where the workspace's slots (a partial result
    // of one pair each) allow it: ranges + min(ranges, pairs) of them.  Cutting costs a second
    // kernel (2 us); it pays where it evens out the work of more pairs than CTAs, or cuts fewer
    // pairs into two pieces each or more (8 pairs of 148..445 keys, D = 64, 10 rows, took 11.5 us in 8
    // ranges and 9.6 whole).
    const int per_sm = p.group * p.Sq <= 4   ? Kv8Cfg<D, 1>::resident(a.B)
                       : p.group * p.Sq <= 8 ? Kv8Cfg<D, 2>::resident(a.B)
                                             : Kv8Cfg<D, 4>::resident(a.B);
    const long long pairs = (long long)a.B * a.pool.Hkv, resident = (long long)per_sm * a.num_sms;
    const long long most = pairs * ((p.capacity + kKv8Unit - 1) / kKv8Unit);
    const long long ranges = std::min({resident, most, std::max(a.slots / 2, a.slots - pairs)});
    p.whole = a.slots == 0 || ranges < std::min(resident, 2 * pairs);
    p.grid = (int)(p.whole ? std::min(resident, pairs) : ranges);
    // A warp alone needs no join, but its tiles come one after another: better while they are few
    // and the pairs many.  Measured, in microseconds with CTAs and with warps, one query row and
    // D = 64 where not said.  At least a pair for each warp: 2048 pairs of 10..500 keys 26.9, 25.4, with
    // 8 rows 40.2, 34.5, of 10..1000 with 8 rows 53.1, 50.1, of 100..1000 with 8 rows, D = 128, 68.9, 73.1.
    // Fewer: 1024 of 10..500 18.4, 20.9; of 64, D = 128 (2048), 18.4, 13.0.  Fewer than two for each CTA:
    // 488 of 4 6.8, 4.9; 512 of 1..128 7.3, 7.3, of 1..250 8.7, 9.8.  D = 256: 1600 of 10..120 25.0, 22.2,
    // of 10..300 34.7, 40.6.
    p.solo_keys = 0;
    if (p.group * p.Sq <= 8 ? Kv8Cfg<D, 2>::QRegs : Kv8Cfg<D, 4>::QRegs) {
        if (pairs > p.grid) p.solo_keys = 128;
        if (D != 256 && pairs >= 2ll * p.grid) p.solo_keys = pairs >= (long long)kKv8Warps * p.grid ? 512 : 320;
    }
    fa_status st;
    if (p.group * p.Sq <= 4)
        st = a.bf16 ? launch_kv8_split<D, 1, true>(p, s) : launch_kv8_split<D, 1, false>(p, s);
    else if (p.group * p.Sq <= 8)
        st = a.bf16 ? launch_kv8_split<D, 2, true>(p, s) : launch_kv8_split<D, 2, false>(p, s);
    else
        st = a.bf16 ? launch_kv8_split<D, 4, true>(p, s) : launch_kv8_split<D, 4, false>(p, s);
    if (st != FA_OK || p.whole) return st;
    // Few rows are cut into many pieces: eight warps each.
    return a.B * a.Sq * a.Hq <= 8 * a.num_sms ? launch_kv8_merge<D, 8>(p, a.bf16, s)
                                              : launch_kv8_merge<D, 1>(p, a.bf16, s);
}

}  // namespace fa

