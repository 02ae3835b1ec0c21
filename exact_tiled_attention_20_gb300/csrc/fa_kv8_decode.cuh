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
    int w = (total + p.grid - 1) / p.grid;
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

template <int D, bool kBF16>
__global__ void __launch_bounds__(kKv8Threads) kv8_split_kernel(const Kv8DecParams p) {
    constexpr int V = D / 32;
    __shared__ Kv8Plan plan;
    __shared__ float s_o[kKv8Warps][D], s_m[kKv8Warps], s_l[kKv8Warps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int W = kv8_make_plan(p, plan);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float kNegInf = -__int_as_float(0x7f800000);
    uint16_t* o16 = static_cast<uint16_t*>(p.o);
    const uint16_t* q16 = static_cast<const uint16_t*>(p.q);
    for (int b = blockIdx.x; b < p.B; b += p.grid) {  // sequences without keys
        if (plan.lens[b] > 0) continue;
        for (int i = threadIdx.x; i < p.Sq * p.Hq * D; i += kKv8Threads) o16[(size_t)b * p.Sq * p.Hq * D + i] = 0;
        if (p.lse)
            for (int i = threadIdx.x; i < p.Sq * p.Hq; i += kKv8Threads) p.lse[(size_t)b * p.Sq * p.Hq + i] = kNegInf;
    }
    const int Hkv = p.pool.Hkv;
    const int total = Hkv * plan.prefix[p.B];
    int x = (int)min((long long)blockIdx.x * W, (long long)total);
    const int x_end = (int)min((long long)x + W, (long long)total);
    while (x < x_end) {
        int lo = 0, hi = p.B;  // largest b with Hkv * prefix[b] <= x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (Hkv * plan.prefix[mid] <= x) lo = mid; else hi = mid;
        }
        const int b = lo, tb = kv8_tiles(plan.lens[b]);
        const int hk = (x - Hkv * plan.prefix[b]) / tb;
        const int start = Hkv * plan.prefix[b] + hk * tb;
        const int seg_end = min(x_end, start + tb);
        const int slot = (int)blockIdx.x - start / W, pieces = kv8_pieces(start, tb, W);
        const int len = plan.lens[b];
        const int k0 = (x - start) * kKv8Tile, k1 = min((seg_end - start) * kKv8Tile, len);
        x = seg_end;
        for (int col = 0; col < p.group * p.Sq; ++col) {
            const int tok = col / p.group, h = hk * p.group + col % p.group;
            const size_t row = ((size_t)b * p.Sq + tok) * p.Hq + h;
            const int lim = p.causal ? min(k1, len - p.Sq + tok + 1) : k1;
            float q[V], acc[V], m = kNegInf, l = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                q[i] = float_from16<kBF16>(q16[row * D + lane + i * 32]);
                acc[i] = 0.f;
            }
            for (int j = k0 + warp; j < lim; j += kKv8Warps) {
                const int pi = j / p.pool.page_size;
                const int page = p.pool.table[(size_t)b * p.pool.max_pages + pi];
                const bool ok = page >= 0 && page < p.pool.num_pages;
                const size_t r = ok ? ((size_t)page * Hkv + hk) * p.pool.page_size + (j - pi * p.pool.page_size) : 0;
                const float ks = ok ? kv8_scale(p.pool.ks[r]) : 0.f, vs = ok ? kv8_scale(p.pool.vs[r]) : 0.f;
                float dot = 0.f, v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint16_t kc = ok ? p.pool.k[r * D + lane + i * 32] : 0;
                    const uint16_t vc = ok ? p.pool.v[r * D + lane + i * 32] : 0;
                    dot += q[i] * float_from16<false>((uint16_t)(e4m3x2_to_f16x2(kc) & 0xffffu));
                    v[i] = float_from16<false>((uint16_t)(e4m3x2_to_f16x2(vc) & 0xffffu));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                const float s = dot * ks * p.scale_log2;
                const float mn = fmaxf(m, s);
                const float f = ex2_approx(m - mn), e = ex2_approx(s - mn);
                l = l * f + e;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = acc[i] * f + e * vs * v[i];
                m = mn;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) s_o[warp][lane + i * 32] = acc[i];
            if (lane == 0) {
                s_m[warp] = m;
                s_l[warp] = l;
            }
            __syncthreads();
            float M = kNegInf, L = 0.f, w[kKv8Warps];
            for (int i = 0; i < kKv8Warps; ++i) M = fmaxf(M, s_m[i]);
            for (int i = 0; i < kKv8Warps; ++i) {
                w[i] = M == kNegInf ? 0.f : ex2_approx(s_m[i] - M);
                L += w[i] * s_l[i];
            }
            const float lse = M == kNegInf ? kNegInf : (M + lg2_approx(L)) * kLn2;
            for (int d = threadIdx.x; d < D; d += kKv8Threads) {
                float o = 0.f;
                for (int i = 0; i < kKv8Warps; ++i) o += w[i] * s_o[i][d];
                if (M != kNegInf) o /= L;
                if (pieces == 1)
                    o16[row * D + d] = float_to16<kBF16>(o);
                else
                    p.o_part[(row * p.ns + slot) * D + d] = o;
            }
            if (threadIdx.x == 0) {
                if (pieces > 1)
                    p.lse_part[row * p.ns + slot] = lse;
                else if (p.lse)
                    p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = lse;
            }
            __syncthreads();
        }
    }
}

// Joins the pieces of each row (b, token, head): lse = log sum exp(lse_c), and the outputs
// weighted with exp(lse_c - lse), in the order of the pieces.  One warp per row.
template <int D, bool kBF16>
__global__ void __launch_bounds__(128) kv8_merge_kernel(const Kv8DecParams p) {
    constexpr int V = D / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= p.B * p.Sq * p.Hq) return;
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
    if (n < 2) return;  // the split kernel has written this row
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
        for (int c = 0; c < n; ++c) {
            const float w = ex2_approx((lrow[c] - m) / kLn2);
            s += w;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += w * orow[(size_t)c * D + i * 32];
        }
    }
    uint16_t* out = static_cast<uint16_t*>(p.o) + (size_t)row * D + lane;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i * 32] = float_to16<kBF16>(m == kNegInf ? 0.f : acc[i] / s);
    if (p.lse && lane == 0)
        p.lse[((size_t)b * p.Hq + h) * p.Sq + tok] = m == kNegInf ? kNegInf : m + lg2_approx(s) * kLn2;
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
    const fa_status st = a.bf16 ? launch_overlapped(kv8_split_kernel<D, true>, p.grid, kKv8Threads, 0, s, p)
                                : launch_overlapped(kv8_split_kernel<D, false>, p.grid, kKv8Threads, 0, s, p);
    if (st != FA_OK || p.ns < 2) return st;
    const unsigned rows = (unsigned)(a.B * a.Sq * a.Hq);
    return a.bf16 ? launch_overlapped(kv8_merge_kernel<D, true>, (rows + 3) / 4, 128, 0, s, p)
                  : launch_overlapped(kv8_merge_kernel<D, false>, (rows + 3) / 4, 128, 0, s, p);
}

}  // namespace fa
