// fa_kv8_decode.cuh -- split-KV decode over the 8-bit paged cache.
//
// For sequence b, query token i of Sq and query head h (kv head hk = h / (Hq / Hkv)):
//     s_j = scale * 2^(ks_j - 127) * (q . kcode_j),   j visible: j < len_b, and with `causal`
//                                                     j <= len_b - Sq + i
//     o   = sum_j softmax(s)_j 2^(vs_j - 127) vcode_j,    lse = log sum_j exp(s_j)
//
// Plan: the keys of every (sequence, kv head) pair, in 128-key tiles, lie end to end in the
// order (b, hk), and CTA c takes tiles [c W, (c + 1) W): every CTA streams the same number
// of bytes whatever the mix of lengths.  W also keeps a pair within num_splits pieces.  A
// pair that lies in one range is finished by its CTA; one that is cut leaves a partial
// output and its log-sum-exp per piece, which the merge kernel joins.
#pragma once

#include "fa_kv8.cuh"

namespace fa {

struct Kv8DecParams {
    Kv8Pool pool;
    const void* q;
    void* o;
    float* lse;
    const int32_t* kv_lens;
    float* o_part;
    float* lse_part;
    int B, Sq, Hq, group, capacity, ns, causal;
    int grid;  // CTAs of the split kernel
    float scale_log2;
};

constexpr int kKv8Tile = 128;  // keys per tile of the plan
constexpr int kKv8Threads = 128;
constexpr int kKv8Warps = kKv8Threads / 32;
constexpr int kKv8MaxB = 1024;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ int kv8_len(const Kv8DecParams& p, int b) {
    return min(max(p.kv_lens[b], 0), p.capacity);
}

__device__ __forceinline__ int kv8_tiles(int len) { return (len + kKv8Tile - 1) / kKv8Tile; }

// W, from the tiles of one pair of each sequence summed, and the longest pair's.
__device__ __forceinline__ int kv8_width(const Kv8DecParams& p, int sum_tiles, int max_tiles) {
    const int total = p.pool.Hkv * sum_tiles;
    int w = (int)(((long long)total + p.grid - 1) / p.grid);
    w = max(w, p.ns >= 2 ? (max_tiles + p.ns - 2) / (p.ns - 1) : total);
    return max(w, 1);
}

// Pieces of the pair whose tb tiles begin at tile `start`.
__device__ __forceinline__ int kv8_pieces(int start, int tb, int w) {
    return tb > 0 ? (start + tb - 1) / w - start / w + 1 : 0;
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

struct Kv8Plan {
    int lens[kKv8MaxB];
    int prefix[kKv8MaxB + 1];  // tiles of one pair of each sequence before b
    int warp_sum[kKv8Warps], warp_max[kKv8Warps];
};

// Fills the plan from kv_lens (all threads; ends with a barrier) and returns W.
__device__ __forceinline__ int kv8_make_plan(const Kv8DecParams& p, Kv8Plan& t) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.B + kKv8Threads - 1) / kKv8Threads;
    int sum = 0, most = 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            const int len = kv8_len(p, b);
            t.lens[b] = len;
            sum += kv8_tiles(len);
            most = max(most, kv8_tiles(len));
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
        t.warp_sum[warp] = incl;
        t.warp_max[warp] = most;
    }
    __syncthreads();
    int run = incl - sum;
    most = 0;
    for (int w = 0; w < kKv8Warps; ++w) {
        if (w < warp) run += t.warp_sum[w];
        most = max(most, t.warp_max[w]);
    }
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b < p.B) {
            t.prefix[b] = run;
            run += kv8_tiles(t.lens[b]);
        }
    }
    if (threadIdx.x == kKv8Threads - 1) t.prefix[p.B] = run;
    __syncthreads();
    return kv8_width(p, t.prefix[p.B], most);
}

// ------------------------------------------------------------------ shared layout ----
// Each warp streams its own tiles of KT keys through a ring of NST stages in shared memory:
// K codes, V codes, K scales, V scales.  A row is split into a part of WA bytes and, at
// D = 96, one of 32; each part's rows lie in 128-byte lines whose 16-byte units are permuted
// so that the reads below, K by (row g, unit t) and V by (row 2 t, unit g), meet no bank
// twice.
template <int D_>
struct Kv8Cfg {
    static constexpr int D = D_;
    static constexpr int KT = D == 64 ? 64 : (D == 256 ? 16 : 32);
    static constexpr int NSUB = KT / 16;  // runs of 16 keys
    static constexpr int NST = D == 96 ? 4 : 3;
    static constexpr int TileBytes = KT * D;
    static constexpr int StageBytes = 2 * TileBytes + 128;
    static constexpr int RingBytes = NST * StageBytes;
    static constexpr int SmemBytes = kKv8Warps * RingBytes + 128;
    static constexpr int WA = D == 96 ? 64 : D;
    static constexpr int KS = D / 16;        // steps of 16 dims, and 16-dim blocks of O^T
    static constexpr int Copies = D / 32;    // 16-byte copies of a lane per run and tensor
    static_assert(2 * KT <= 128, "scales of a stage");

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

// NT: blocks of 8 query rows (tokens x heads of one kv head; column token * group + head).
template <int D, int NT, bool kBF16>
__global__ void __launch_bounds__(kKv8Threads, 2) kv8_split_kernel(const Kv8DecParams p) {
    using C = Kv8Cfg<D>;
    constexpr int KT = C::KT, NSUB = C::NSUB, NST = C::NST, KS = C::KS;
    constexpr bool kQRegs = KS * NT <= 16;  // query fragments in registers, else in shared memory
    extern __shared__ uint8_t ring_raw[];
    __shared__ Kv8Plan plan;
    __shared__ float s_mo[kKv8Warps][16], s_ms[kKv8Warps][16], s_l[kKv8Warps][16];
    __shared__ uint2 s_q[kQRegs ? 1 : KS * NT][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int W = kv8_make_plan(p, plan);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const float kNegInf = -__int_as_float(0x7f800000);
    uint16_t* o16 = static_cast<uint16_t*>(p.o);
    const uint16_t* q16 = static_cast<const uint16_t*>(p.q);
    const int rows = p.Sq * p.Hq;
    for (int b = blockIdx.x; b < p.B; b += p.grid) {  // sequences without keys
        if (plan.lens[b] > 0) continue;
        for (int i = tid; i < rows * D; i += kKv8Threads) o16[(size_t)b * rows * D + i] = 0;
        if (p.lse)
            for (int i = tid; i < rows; i += kKv8Threads) p.lse[(size_t)b * rows + i] = kNegInf;
    }
    const uint32_t raw = smem_u32(ring_raw), base = (raw + 127u) & ~127u;
    const uint32_t ring = base + warp * C::RingBytes;
    float* exch = reinterpret_cast<float*>(ring_raw + (base - raw));
    constexpr int XD = D + 4;  // row of the exchange
    static_assert(kKv8Warps * 16 * XD * 4 <= kKv8Warps * C::RingBytes, "exchange fits the ring");

    // This lane's units of a run of 16 rows: unit i * 32 + lane of the run's 16 D bytes.
    uint32_t dst[C::Copies], step[C::Copies];
#pragma unroll
    for (int i = 0; i < C::Copies; ++i) {
        const int u = i * 32 + lane, row = u / (D / 16), c = u % (D / 16);
        dst[i] = C::unit(row, c);
        step[i] = C::run_step(c);
    }
    const int Hkv = p.pool.Hkv, cols = p.group * p.Sq;
    const int runs_per_page = p.pool.page_size / 16;
    const int total = Hkv * plan.prefix[p.B];
    int x = (int)min((long long)blockIdx.x * W, (long long)total);
    const int x_end = (int)min((long long)x + W, (long long)total);
    while (x < x_end) {
        int lo = 0, hi = p.B;  // largest b with Hkv * prefix[b] <= x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (Hkv * plan.prefix[mid] <= x) lo = mid; else hi = mid;
        }
        const int b = lo, len = plan.lens[b], tb = kv8_tiles(len);
        const int hk = (x - Hkv * plan.prefix[b]) / tb;
        const int start = Hkv * plan.prefix[b] + hk * tb;
        const int seg_end = min(x_end, start + tb);
        const int slot = (int)blockIdx.x - start / W, pieces = kv8_pieces(start, tb, W);
        const int k0 = (x - start) * kKv8Tile, k1 = min((seg_end - start) * kKv8Tile, len);
        x = seg_end;
        const int tiles = (k1 - k0 + KT - 1) / KT;  // warp w takes tiles w, w + kKv8Warps, ...
        const int32_t* table = p.pool.table + (size_t)b * p.pool.max_pages;

        // The 16-key run of the pool that holds run lane % NSUB of tile j: its index, -1 where
        // there is none (behind k1, or a page outside the pool).
        auto find_run = [&](int j) -> int {
            const int key = k0 + j * KT + (lane % NSUB) * 16;
            if (key >= k1) return -1;
            const unsigned pi = (unsigned)key / (unsigned)p.pool.page_size;
            const int page = table[pi];
            if (page < 0 || page >= p.pool.num_pages) return -1;
            return (page * Hkv + hk) * runs_per_page + (int)((unsigned)key - pi * (unsigned)p.pool.page_size) / 16;
        };
        // Starts the copies of tile j into stage st; rows without a key become zeros.
        auto issue = [&](int j, int st, int run) {
            const uint32_t sk = ring + st * C::StageBytes, sv = sk + C::TileBytes, ss = sv + C::TileBytes;
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                const int r = __shfl_sync(0xffffffffu, run, s);
                const int key = k0 + j * KT + s * 16;
                const int valid = r < 0 ? 0 : min(16, k1 - key) * D;
                const size_t off = (size_t)max(r, 0) * (16 * D) + lane * 16;
#pragma unroll
                for (int i = 0; i < C::Copies; ++i) {
                    const int n = i * 512 + lane * 16 < valid ? 16 : 0;
                    const uint32_t d = dst[i] + s * step[i];
                    cp_async16(sk + d, p.pool.k + off + i * 512, n);
                    cp_async16(sv + d, p.pool.v + off + i * 512, n);
                }
            }
            if (lane < 2 * NSUB) {
                const uint8_t* src = (lane < NSUB ? p.pool.ks : p.pool.vs) + (size_t)max(run, 0) * 16;
                cp_async16(ss + (lane / NSUB) * KT + (lane % NSUB) * 16, src, run < 0 ? 0 : 16);
            }
        };

        int run = find_run(warp);
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) {
            const int j = warp + i * kKv8Warps;
            if (j < tiles) issue(j, i, run);
            cp_async_commit();
            run = find_run(j + kKv8Warps);
        }

        // Query fragments: row n of a block as f16, times a power of two that brings its largest
        // magnitude to [2^13, 2^14).  fp16's subnormals are then 2^-38 of it, so bf16 and fp16
        // queries enter exactly but for values that far below their row's largest.
        uint2 qr[kQRegs ? KS * NT : 1];
        float qf[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = nt * 8 + g;
            const int tok = col / p.group, h = hk * p.group + col % p.group;
            const uint16_t* src = q16 + (((size_t)b * p.Sq + tok) * p.Hq + h) * D;
            uint2 w[KS];
            float amax = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int d = ks * 16 < C::WA ? (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 : 64 + t * 8 + (ks - 4) * 4;
                w[ks] = col < cols ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(float_from16<kBF16>((uint16_t)w[ks].x)),
                                               fabsf(float_from16<kBF16>((uint16_t)(w[ks].x >> 16)))),
                                         fmaxf(fabsf(float_from16<kBF16>((uint16_t)w[ks].y)),
                                               fabsf(float_from16<kBF16>((uint16_t)(w[ks].y >> 16))))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax = f 2^x; the factor is 2^(13 - x), from the exponent field, kept normal
            int ex = (int)(__float_as_uint(amax) >> 23);
            ex = ex == 255 ? 127 + 13 : max(ex, 14);
            const float up = __uint_as_float((uint32_t)(254 + 13 - ex) << 23);
            const float down = p.scale_log2 * __uint_as_float((uint32_t)(ex - 13) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint2 f = {pack_f16x2(float_from16<kBF16>((uint16_t)w[ks].x) * up,
                                            float_from16<kBF16>((uint16_t)(w[ks].x >> 16)) * up),
                                 pack_f16x2(float_from16<kBF16>((uint16_t)w[ks].y) * up,
                                            float_from16<kBF16>((uint16_t)(w[ks].y >> 16)) * up)};
                if constexpr (kQRegs)
                    qr[ks * NT + nt] = f;
                else if (warp == 0)
                    s_q[ks * NT + nt][lane] = f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[nt][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
                const int tk = (nt * 8 + 2 * t + e) / p.group;
                lim[nt][e] = p.causal ? min(k1, len - p.Sq + tk + 1) : k1;
            }
        }
        if constexpr (!kQRegs) __syncthreads();

        float o[KS][NT][4], ms[NT][2], mo[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int m = 0; m < KS; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][nt][i] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ms[nt][e] = mo[nt][e] = kLowest;
                l[nt][e] = 0.f;
            }
        }

        int st = 0;
        for (int j = warp; j < tiles; j += kKv8Warps) {
            cp_async_wait<NST - 2>();
            __syncwarp();
            {
                const int jn = j + (NST - 1) * kKv8Warps;
                if (jn < tiles) issue(jn, st == 0 ? NST - 1 : st - 1, run);
                cp_async_commit();
                run = find_run(jn + kKv8Warps);
            }
            const uint32_t sk = ring + st * C::StageBytes, sv = sk + C::TileBytes, ss = sv + C::TileBytes;
            st = st == NST - 1 ? 0 : st + 1;

            // S^T = K Q^T: 16 keys x 8 query rows at a time, the dims in an order that gives each
            // lane whole 16-byte units of its rows.
            float sc[NSUB][NT][4];
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
                        if constexpr (kQRegs)
                            q = qr[ks * NT + nt];
                        else
                            q = s_q[ks * NT + nt][lane];
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
                    for (int i = 0; i < 4; ++i) sc[s][nt][i] = acc[0][nt][i] + acc[1][nt][i];
            }

            // Softmax in base 2.  ms, l: this lane's own maximum and sum of exp2(s - ms) (joined at
            // the end); mo: the reference of P = exp2(s + log2 V scale - mo), one for all lanes.
            float lv[NSUB][2];
            bool grow = false;
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
                        for (int e = 0; e < 2; ++e) {
                            float& v = sc[s][nt][i * 2 + e];
                            v = key < lim[nt][e] ? v * (kf * qf[nt][e]) : kNegInf;
                            grow |= v + lv[s][i] > mo[nt][e] + kPSlack;
                        }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = ms[nt][e];
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) m = fmaxf(m, fmaxf(sc[s][nt][e], sc[s][nt][2 + e]));
                    float sum = l[nt][e] * ex2_approx(ms[nt][e] - m);
#pragma unroll
                    for (int s = 0; s < NSUB; ++s)
                        sum += ex2_approx(sc[s][nt][e] - m) + ex2_approx(sc[s][nt][2 + e] - m);
                    l[nt][e] = sum;
                    ms[nt][e] = m;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = mo[nt][e];
#pragma unroll
                        for (int s = 0; s < NSUB; ++s)
                            m = fmaxf(m, fmaxf(sc[s][nt][e] + lv[s][0], sc[s][nt][2 + e] + lv[s][1]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                        const float f = ex2_approx(mo[nt][e] - m);
                        mo[nt][e] = m;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[k][nt][e] *= f;
                            o[k][nt][2 + e] *= f;
                        }
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
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            v[e] = ex2_approx((sc[s][nt][i * 2 + e] + lv[s][i]) - (mo[nt][e] - kPShift));
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

        // Join the warps: per query row the maxima and sums over the lanes of one t, then the four
        // warps through shared memory (the ring, which nobody reads any more).
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = ms[nt][e];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                float sum = l[nt][e] * ex2_approx(ms[nt][e] - m);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                const int col = nt * 8 + 2 * t + e;
                if (g == 0) {
                    s_mo[warp][col] = mo[nt][e];
                    s_ms[warp][col] = m;
                    s_l[warp][col] = sum;
                }
                if (col < cols) {
                    float* row = exch + (warp * 16 + col) * XD;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        int d;  // dims d, d + 1: rows g and g + 8 of block k
                        if constexpr (C::WA == 64)
                            d = k < 4 ? g * 8 + k * 2 : 64 + g * 4 + (k - 4) * 2;
                        else
                            d = (k >> 3) * 128 + g * 16 + (k & 7) * 2;
                        *reinterpret_cast<float2*>(row + d) = make_float2(o[k][nt][e], o[k][nt][2 + e]);
                    }
                }
            }
        __syncthreads();
        for (int i = tid; i < cols * (D / 2); i += kKv8Threads) {
            const int col = i / (D / 2), d = i % (D / 2) * 2;
            float Mo = s_mo[0][col], Ms = s_ms[0][col];
#pragma unroll
            for (int w = 1; w < kKv8Warps; ++w) {
                Mo = fmaxf(Mo, s_mo[w][col]);
                Ms = fmaxf(Ms, s_ms[w][col]);
            }
            float L = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int w = 0; w < kKv8Warps; ++w) {
                const float f = ex2_approx(s_mo[w][col] - Mo);
                const float2 v = *reinterpret_cast<const float2*>(exch + (w * 16 + col) * XD + d);
                a0 = fmaf(f, v.x, a0);
                a1 = fmaf(f, v.y, a1);
                L = fmaf(ex2_approx(s_ms[w][col] - Ms), s_l[w][col], L);
            }
            // O = a 2^(Mo - kPShift - Ms) / L, the power in two halves (V scales go down to 2^-127)
            const float f = ex2_approx((Mo - kPShift - Ms) * 0.5f);
            const float inv = 1.f / L;
            a0 = L == 0.f ? 0.f : a0 * inv * f * f;
            a1 = L == 0.f ? 0.f : a1 * inv * f * f;
            const int tok = col / p.group, h = hk * p.group + col % p.group;
            const size_t row = ((size_t)b * p.Sq + tok) * p.Hq + h;
            const float lse = L == 0.f ? kNegInf : (Ms + lg2_approx(L)) * kLn2;
            if (pieces == 1) {
                *reinterpret_cast<uint32_t*>(o16 + row * D + d) = pack2<kBF16>(a0, a1);
                if (d == 0 && p.lse) p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = lse;
            } else {
                *reinterpret_cast<float2*>(p.o_part + (row * p.ns + slot) * D + d) = make_float2(a0, a1);
                if (d == 0) p.lse_part[row * p.ns + slot] = lse;
            }
        }
        __syncthreads();  // before the ring and the plan's next segment
    }
}

template <int D, int NT, bool kBF16>
fa_status launch_kv8_split(const Kv8DecParams& p, cudaStream_t s) {
    static int attr[64] = {0};
    constexpr int bytes = Kv8Cfg<D>::SmemBytes;
    if (!ensure_smem_attr((const void*)kv8_split_kernel<D, NT, kBF16>, bytes, attr)) return FA_ERR_CUDA;
    return launch_overlapped(kv8_split_kernel<D, NT, kBF16>, p.grid, kKv8Threads, bytes, s, p);
}

// Joins the pieces of each row (b, token, head): lse = log sum_c exp(lse_c), and the outputs
// weighted with exp(lse_c - lse).  WPR warps share a row, each taking every WPR-th piece; a
// lane holds D / 32 dims.  It moves few bytes: its time is the launch and two or three
// dependent trips to L2, so the pieces of a warp are loaded several at a time.
template <int D, int WPR, bool kBF16>
__global__ void __launch_bounds__(256) kv8_merge_kernel(const Kv8DecParams p) {
    constexpr int V = D / 32, Rows = 8 / WPR, NB = V <= 4 ? 8 : 4;
    __shared__ float s_acc[WPR > 1 ? 8 : 1][D], s_sum[8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * Rows + warp / WPR, part = warp % WPR;
    if (row >= p.B * p.Sq * p.Hq) return;  // whole CTAs where WPR = 8
    const int b = row / (p.Sq * p.Hq), tok = row / p.Hq % p.Sq, h = row % p.Hq;
    int before = 0, sum = 0, most = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int t = kv8_tiles(kv8_len(p, i));
        before += i < b ? t : 0;
        sum += t;
        most = max(most, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    const int tb = kv8_tiles(kv8_len(p, b));
    const int W = kv8_width(p, sum, most);
    const int n = kv8_pieces(p.pool.Hkv * before + h / p.group * tb, tb, W);
    if (n < 2) return;  // the split kernel has written this row (n is the same in all of a row's warps)
    const float kNegInf = -__int_as_float(0x7f800000);
    const float* lrow = p.lse_part + (size_t)row * p.ns;
    const float* orow = p.o_part + (size_t)row * p.ns * D + lane;
    float m = kNegInf;
    for (int c = lane; c < n; c += 32) m = fmaxf(m, lrow[c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[V], s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (m != kNegInf) {
        for (int c0 = part; c0 < n; c0 += WPR * NB) {
            float w[NB], v[NB][V];
#pragma unroll
            for (int u = 0; u < NB; ++u) {  // pieces past n: the last one, with weight 0
                const int c = min(c0 + u * WPR, n - 1);
                w[u] = c0 + u * WPR < n ? lrow[c] : kNegInf;
#pragma unroll
                for (int i = 0; i < V; ++i) v[u][i] = orow[(size_t)c * D + i * 32];
            }
#pragma unroll
            for (int u = 0; u < NB; ++u) {
                const float f = ex2_approx((w[u] - m) * (1.f / kLn2));
                s += f;
                // a piece without a visible key has weight 0 and an output of 0; a weight of 0
                // that pads the batch must not meet a NaN or an infinity
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(f, w[u] == kNegInf ? 0.f : v[u][i], acc[i]);
            }
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[warp][lane + i * 32] = acc[i];
        if (lane == 0) s_sum[warp] = s;
        __syncthreads();
        if (warp != 0) return;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            s += s_sum[w];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += s_acc[w][lane + i * 32];
        }
    }
    const float inv = 1.f / s;
    uint16_t* out = static_cast<uint16_t*>(p.o) + (size_t)row * D + lane;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i * 32] = float_to16<kBF16>(m == kNegInf ? 0.f : acc[i] * inv);
    if (p.lse && lane == 0)
        p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = m == kNegInf ? kNegInf : m + lg2_approx(s) * kLn2;
}

template <int D, int WPR>
fa_status launch_kv8_merge(const Kv8DecParams& p, bool bf16, cudaStream_t s) {
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
    p.ns = a.num_splits;
    p.causal = a.causal ? 1 : 0;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    // No more CTAs than the cache could ever hold tiles.
    const long long most = (long long)a.B * a.pool.Hkv * ((p.capacity + kKv8Tile - 1) / kKv8Tile);
    p.grid = (int)(most < 2LL * a.num_sms ? most : 2LL * a.num_sms);
    fa_status st;
    if (p.group * p.Sq <= 8)
        st = a.bf16 ? launch_kv8_split<D, 1, true>(p, s) : launch_kv8_split<D, 1, false>(p, s);
    else
        st = a.bf16 ? launch_kv8_split<D, 2, true>(p, s) : launch_kv8_split<D, 2, false>(p, s);
    if (st != FA_OK || p.ns < 2) return st;
    // Few rows are cut into many pieces: eight warps each.
    return a.B * a.Sq * a.Hq <= 8 * a.num_sms ? launch_kv8_merge<D, 8>(p, a.bf16, s)
                                              : launch_kv8_merge<D, 1>(p, a.bf16, s);
}

}  // namespace fa
