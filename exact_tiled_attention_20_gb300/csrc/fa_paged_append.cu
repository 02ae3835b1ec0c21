// fa_paged_append.cu -- writing rows into the 16-bit paged cache, rotated on the way.
//
// A pair (x, y) of a row turns by the angle of its token's position: with the table's cosine c
// and sine s it becomes (x c - y s, y c + x s), in fp32, rounded once.  The pairs are
// (d, d + rot / 2) or, interleaved, (2 d, 2 d + 1), d < rot / 2; dims from rot on are copied, and
// so are the rows of V.
//
// It is a copy, bound by HBM: 2 D bytes in and 2 D out for each row of queries, keys and values.  A lane
// has two 16-byte pieces of a row, the two sides of eight pairs, so a row is D / 16 lanes.  A
// group of lanes takes U rows of one token (rows i, i + S, ... of its Hq + 2 Hkv): U rows in
// flight, and the eight cosines and sines of a lane are loaded once for all of them.
#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxB = 1024;

__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// A word's two values in fp32.
template <bool kBF16>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
    if constexpr (kBF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
            : "=f"(lo), "=f"(hi)
            : "r"(w));
    }
}

// Turns the eight pairs of a lane: pair i is element i of a and of b, or elements 2 i and 2 i + 1 of
// a followed by b.
template <bool kBF16, bool kInterleaved>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
    uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kInterleaved) {
            float x, y;
            unpack2<kBF16>(wa[i], x, y);
            wa[i] = pack2<kBF16>(x * c[i] - y * s[i], y * c[i] + x * s[i]);
            unpack2<kBF16>(wb[i], x, y);
            wb[i] = pack2<kBF16>(x * c[4 + i] - y * s[4 + i], y * c[4 + i] + x * s[4 + i]);
        } else {
            float x0, x1, y0, y1;
            unpack2<kBF16>(wa[i], x0, x1);
            unpack2<kBF16>(wb[i], y0, y1);
            wa[i] = pack2<kBF16>(x0 * c[2 * i] - y0 * s[2 * i], x1 * c[2 * i + 1] - y1 * s[2 * i + 1]);
            wb[i] = pack2<kBF16>(y0 * c[2 * i] + x0 * s[2 * i], y1 * c[2 * i + 1] + x1 * s[2 * i + 1]);
        }
    }
    a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

template <int D, int U, bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedAppendArgs a) {
    constexpr int G = D / 16, Groups = kThreads / G;  // D = 96: 21 groups of 6, two threads idle
    __shared__ int cu[kMaxB + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int rows = a.Hq + 2 * a.Hkv, S = (rows + U - 1) / U;
    const int group = threadIdx.x / G, l = threadIdx.x - group * G;
    const long long item = (long long)blockIdx.x * Groups + group;
    const int t = (int)(item / S), r0 = (int)(item - (long long)t * S);
    const bool live = group < Groups && t < a.total;

    // The lane's two pieces of a row, in elements.
    const bool turned = l * 16 < a.rot;
    const int d0 = turned && !kInterleaved ? l * 8 : l * 16;
    const int d1 = turned && !kInterleaved ? a.rot / 2 + l * 8 : l * 16 + 8;
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = r0 + u * S;
        x[u] = y[u] = make_uint4(0, 0, 0, 0);
        if (!live || r >= rows) continue;
        const uint16_t* src;
        if (r < a.Hq)
            src = static_cast<const uint16_t*>(a.q) + t * a.q_stride + (long long)r * D;
        else if (r < a.Hq + a.Hkv)
            src = static_cast<const uint16_t*>(a.k_new) + t * a.k_stride + (long long)(r - a.Hq) * D;
        else
            src = static_cast<const uint16_t*>(a.v_new) + t * a.v_stride + (long long)(r - a.Hq - a.Hkv) * D;
        x[u] = load_once(src + d0);
        y[u] = load_once(src + d1);
    }
    if (a.cu) {
        for (int i = threadIdx.x; i <= a.B; i += kThreads) cu[i] = a.cu[i];
        __syncthreads();
    }
    if (!live) return;
    // The token's sequence b, and which of its n new tokens it is: the last n of kv_lens[b] keys.
    int b, n, i;
    if (a.cu) {
        int lo = 0, hi = a.B;  // the first b with cu[b + 1] > t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
        }
        b = lo;
        if (b >= a.B || t < cu[b]) return;  // a row of no sequence
        n = cu[b + 1] - cu[b];
        i = t - cu[b];
    } else {
        n = a.total / a.B;
        b = t / n;
        i = t - b * n;
    }
    const long long key = (long long)a.kv_lens[b] - n + i;
    long long place = -1;  // the pool's row of the token's head 0
    if (key >= 0 && key < (long long)a.page_size * a.max_pages) {
        const int pi = (int)key / a.page_size;
        const int page = a.table[(size_t)b * a.max_pages + pi];
        if (page >= 0 && page < a.num_pages)
            place = ((long long)page * a.page_size + ((int)key - pi * a.page_size)) * a.Hkv;
    }
    float c[8], s[8];
    if (turned) {
        const long long want = a.positions ? (long long)a.positions[t] : key;
        const long long pos = min(max(want, 0ll), (long long)a.max_pos - 1);
        const float4* pc = reinterpret_cast<const float4*>(a.cos + pos * (a.rot / 2) + l * 8);
        const float4* ps = reinterpret_cast<const float4*>(a.sin + pos * (a.rot / 2) + l * 8);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 vc = __ldg(pc + k), vs = __ldg(ps + k);
            c[4 * k] = vc.x, c[4 * k + 1] = vc.y, c[4 * k + 2] = vc.z, c[4 * k + 3] = vc.w;
            s[4 * k] = vs.x, s[4 * k + 1] = vs.y, s[4 * k + 2] = vs.z, s[4 * k + 3] = vs.w;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = r0 + u * S;
        if (r >= rows) continue;
        if (turned && r < a.Hq + a.Hkv) turn<kBF16, kInterleaved>(x[u], y[u], c, s);
        uint16_t* dst;
        if (r < a.Hq) {
            dst = static_cast<uint16_t*>(a.q_out) + ((long long)t * a.Hq + r) * D;
        } else {
            if (place < 0) continue;
            const int h = r - a.Hq;
            dst = h < a.Hkv ? static_cast<uint16_t*>(a.k_pages) + (place + h) * D
                            : static_cast<uint16_t*>(a.v_pages) + (place + h - a.Hkv) * D;
        }
        *reinterpret_cast<uint4*>(dst + d0) = x[u];
        *reinterpret_cast<uint4*>(dst + d1) = y[u];
    }
}

template <int D, int U>
fa_status append_u(const PagedAppendArgs& a, cudaStream_t s) {
    constexpr int groups = kThreads / (D / 16);
    const int per = (a.Hq + 2 * a.Hkv + U - 1) / U;
    const unsigned grid = (unsigned)(((long long)a.total * per + groups - 1) / groups);
    if (a.interleaved)
        return a.bf16 ? launch_overlapped(paged_append_kernel<D, U, true, true>, grid, kThreads, 0, s, a)
                      : launch_overlapped(paged_append_kernel<D, U, false, true>, grid, kThreads, 0, s, a);
    return a.bf16 ? launch_overlapped(paged_append_kernel<D, U, true, false>, grid, kThreads, 0, s, a)
                  : launch_overlapped(paged_append_kernel<D, U, false, false>, grid, kThreads, 0, s, a);
}

// Rows of a group: several where the rows fill the SMs many times over, one where they do not.
template <int D>
fa_status append_d(const PagedAppendArgs& a, cudaStream_t s) {
    const long long rows = (long long)a.total * (a.Hq + 2 * a.Hkv);
    return rows / (kThreads / (D / 16)) >= 32ll * a.num_sms ? append_u<D, 4>(a, s) : append_u<D, 1>(a, s);
}

}  // namespace

fa_status launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    switch (a.D) {
        case 64: return append_d<64>(a, s);
        case 96: return append_d<96>(a, s);
        case 128: return append_d<128>(a, s);
        default: return append_d<256>(a, s);
    }
}

}  // namespace fa
