// fa_kv8_cache.cu -- writing rows into the 8-bit paged KV cache, and reading them back.
//
// Both are copies with a conversion on the way, bound by HBM: a row of D values costs 2 D
// bytes on the 16-bit side and D + 1 on the cache's.
#include "fa_kv8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxB = 1024;

// Where a packed row's token lies in the pool: (page, slot); page -1: nowhere in the pool,
// -2: the row belongs to no sequence.
struct TokenAt {
    int page, slot;
};

// The sequence that owns packed row t: the first b with cu[b + 1] > t.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t) {
    int lo = 0, hi = B;  // cu[lo] <= t where any is; the answer is in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ TokenAt token_at(const Kv8Pool& p, int b, long long key) {
    if (key < 0 || key >= (long long)p.page_size * p.max_pages) return {-1, 0};
    const int i = (int)key / p.page_size;
    const int page = p.table[(size_t)b * p.max_pages + i];
    if (page < 0 || page >= p.num_pages) return {-1, 0};
    return {page, (int)key - i * p.page_size};
}

// ------------------------------------------------------------------------ append ----
template <int D>
struct AppendCfg {
    // Lanes of one row, 8 values (16 bytes) each; at D = 96 the last 4 of 16 idle.
    static constexpr int G = D == 96 ? 16 : D / 8;
    static constexpr int Groups = kThreads / G;
};

template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBF16) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        } else {
            asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
                : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
                : "r"(r[i]));
        }
    }
}

// Quantises one row held by the G lanes of a group, 8 values each.  Returns the scale byte;
// the 8 codes go to `out`.  A value that is not finite takes no part in the scale and
// becomes NaN (e4m3 has no infinity): an overflow upstream stays visible.
template <int G, bool kBF16>
__device__ __forceinline__ uint32_t quantise(const uint4& w, uint2& out) {
    float x[8];
    unpack8<kBF16>(w, x);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        if (a < __int_as_float(0x7f800000)) amax = fmaxf(amax, a);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const uint32_t s = kv8_scale_byte(amax);
    const float inv = kv8_inv_scale(s);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float v = x[2 * i + j];
            y[j] = fabsf(v) < __int_as_float(0x7f800000) ? v * inv : __int_as_float(0x7fc00000);
        }
        c[i] = e4m3x2_from_floats(y[0], y[1]);
    }
    out.x = c[0] | c[1] << 16;
    out.y = c[2] | c[3] << 16;
    return s;
}

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Kv8AppendArgs a) {
    using C = AppendCfg<D>;
    __shared__ int cu[kMaxB + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    if (a.cu)
        for (int i = threadIdx.x; i <= a.B; i += kThreads) cu[i] = a.cu[i];
    __syncthreads();
    const int lane_g = threadIdx.x % C::G;
    const long long row = (long long)blockIdx.x * C::Groups + threadIdx.x / C::G;  // (token, head)
    const int t = (int)(row / a.pool.Hkv), h = (int)(row % a.pool.Hkv);
    const bool in = row < (long long)a.total * a.pool.Hkv && lane_g * 8 < D;
    uint4 wk = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
    TokenAt at = {-2, 0};
    if (in) {
        const uint16_t* k = static_cast<const uint16_t*>(a.k_new) + t * a.k_stride + h * D + lane_g * 8;
        const uint16_t* v = static_cast<const uint16_t*>(a.v_new) + t * a.v_stride + h * D + lane_g * 8;
        wk = *reinterpret_cast<const uint4*>(k);
        wv = *reinterpret_cast<const uint4*>(v);
        int b, n, i;
        if (a.cu) {
            b = sequence_of(cu, a.B, t);
            n = b < a.B ? cu[b + 1] - cu[b] : 0;
            i = b < a.B ? t - cu[b] : -1;
        } else {
            n = a.total / a.B;
            b = t / n;
            i = t - b * n;
        }
        // The n new tokens are the last n of the sequence's kv_lens[b] keys.
        if (i >= 0) at = token_at(a.pool, b, (long long)a.kv_lens[b] - n + i);
    }
    uint2 ck, cv;
    const uint32_t sk = quantise<C::G, kBF16>(wk, ck);
    const uint32_t sv = quantise<C::G, kBF16>(wv, cv);
    if (in && at.page >= 0) {
        const size_t r = ((size_t)at.page * a.pool.Hkv + h) * a.pool.page_size + at.slot;
        *reinterpret_cast<uint2*>(a.pool.k + r * D + lane_g * 8) = ck;
        *reinterpret_cast<uint2*>(a.pool.v + r * D + lane_g * 8) = cv;
        if (lane_g == 0) {
            a.pool.ks[r] = (uint8_t)sk;
            a.pool.vs[r] = (uint8_t)sv;
        }
    }
}

// -------------------------------------------------------------------------- read ----
template <bool kBF16>
__device__ __forceinline__ uint4 dequantise8(const uint2& c, float scale) {
    const uint32_t r[2] = {c.x, c.y};
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t f = e4m3x2_to_f16x2((uint16_t)(r[i / 2] >> (16 * (i % 2))));
        float x, y;
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
            : "=f"(x), "=f"(y)
            : "r"(f));
        d[i] = pack2<kBF16>(x * scale, y * scale);
    }
    return {d[0], d[1], d[2], d[3]};
}

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8ReadArgs a) {
    constexpr int PerRow = D / 8;  // threads of one row, 8 values each
    __shared__ int cu[kMaxB + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    for (int i = threadIdx.x; i <= a.B; i += kThreads) cu[i] = a.cu[i];
    __syncthreads();
    const long long x = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long row = x / PerRow;
    const int c8 = (int)(x % PerRow) * 8;
    if (row >= (long long)a.total * a.pool.Hkv) return;
    const int t = (int)(row / a.pool.Hkv), h = (int)(row % a.pool.Hkv);
    const int b = sequence_of(cu, a.B, t);
    if (b >= a.B || t < cu[b]) return;
    const long long key = (long long)(a.starts ? a.starts[b] : 0) + (t - cu[b]);
    const TokenAt at = token_at(a.pool, b, key);
    uint4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (at.page >= 0) {
        const size_t r = ((size_t)at.page * a.pool.Hkv + h) * a.pool.page_size + at.slot;
        k = dequantise8<kBF16>(*reinterpret_cast<const uint2*>(a.pool.k + r * D + c8), kv8_scale(a.pool.ks[r]));
        v = dequantise8<kBF16>(*reinterpret_cast<const uint2*>(a.pool.v + r * D + c8), kv8_scale(a.pool.vs[r]));
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + row * D + c8) = k;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + row * D + c8) = v;
}

template <int D>
fa_status append_d(const Kv8AppendArgs& a, cudaStream_t s) {
    const long long rows = (long long)a.total * a.pool.Hkv;
    const unsigned grid = (unsigned)((rows + AppendCfg<D>::Groups - 1) / AppendCfg<D>::Groups);
    return a.bf16 ? launch_overlapped(kv8_append_kernel<D, true>, grid, kThreads, 0, s, a)
                  : launch_overlapped(kv8_append_kernel<D, false>, grid, kThreads, 0, s, a);
}

template <int D>
fa_status read_d(const Kv8ReadArgs& a, cudaStream_t s) {
    const long long n = (long long)a.total * a.pool.Hkv * (D / 8);
    const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads);
    return a.bf16 ? launch_overlapped(kv8_read_kernel<D, true>, grid, kThreads, 0, s, a)
                  : launch_overlapped(kv8_read_kernel<D, false>, grid, kThreads, 0, s, a);
}

}  // namespace

fa_status launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s) {
    switch (a.D) {
        case 64: return append_d<64>(a, s);
        case 96: return append_d<96>(a, s);
        case 128: return append_d<128>(a, s);
        case 256: return append_d<256>(a, s);
        default: return FA_ERR_UNSUPPORTED;
    }
}

fa_status launch_kv8_read(const Kv8ReadArgs& a, cudaStream_t s) {
    switch (a.D) {
        case 64: return read_d<64>(a, s);
        case 96: return read_d<96>(a, s);
        case 128: return read_d<128>(a, s);
        case 256: return read_d<256>(a, s);
        default: return FA_ERR_UNSUPPORTED;
    }
}

}  // namespace fa
