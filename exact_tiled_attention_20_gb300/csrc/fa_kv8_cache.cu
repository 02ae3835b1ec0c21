// fa_kv8_cache.cu -- writing rows into the 8-bit paged KV cache, and reading them back.
//
// Both are copies with a conversion on the way, bound by HBM: a row of D values costs 2 D
// bytes on the 16-bit side and D + 1 on the cache's.  A CTA takes a run of consecutive packed
// rows (token, head), U of them for each group of lanes that shares a row, so that every lane
// has several 16-byte loads in flight; where the run's tokens lie in the pool is then
// worked out once per token, by one thread each, into shared memory.
#include "fa_kv8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxB = 1024;

// Where a packed row's token lies: the pool's row of its head 0 (head h is h * page_size rows on),
// or one of these.
constexpr long long kNoPlace = -1;     // outside the table's capacity or the pool
constexpr long long kNoSequence = -2;  // the row belongs to no sequence

// The sequence that owns packed row t: the first b with cu[b + 1] > t.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t) {
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ long long place_of(const Kv8Pool& p, int b, long long key) {
    if (key < 0 || key >= (long long)p.page_size * p.max_pages) return kNoPlace;
    const int i = (int)key / p.page_size;
    const int page = p.table[(size_t)b * p.max_pages + i];
    if (page < 0 || page >= p.num_pages) return kNoPlace;
    return (long long)page * p.Hkv * p.page_size + ((int)key - i * p.page_size);
}

// A 16-byte load of data that is read once.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// ------------------------------------------------------------------------ append ----
template <int D, int U>
struct AppendCfg {
    // Lanes of one row, 8 values (16 bytes) each; at D = 96 the last 4 of 16 idle.
    static constexpr int G = D == 96 ? 16 : D / 8;
    static constexpr int Groups = kThreads / G;
    static constexpr int Run = Groups * U;  // rows of a CTA
};

// Of each half, the larger magnitude of a and b (NaN where either is), with some sign.
template <bool kBF16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (kBF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A mask of the halves of a word that hold infinities or NaNs.
template <bool kBF16>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    return ((w & 0x7fffu) >= kInf ? 0xffffu : 0u) | ((w >> 16 & 0x7fffu) >= kInf ? 0xffff0000u : 0u);
}

// The largest magnitudes of a K row (low half) and a V row (high half) held by the G lanes of a
// group, 8 values of each a lane; from the words `k` and `v` of a lane's own maxima.
template <int G, bool kBF16>
__device__ __forceinline__ uint32_t group_max(uint32_t k, uint32_t v) {
    uint32_t m = max_abs2<kBF16>(__byte_perm(k, v, 0x5410), __byte_perm(k, v, 0x7632));
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) m = max_abs2<kBF16>(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m & 0x7fff7fffu;
}

template <bool kBF16>
__device__ __forceinline__ uint32_t lane_max(const uint4& w) {
    return max_abs2<kBF16>(max_abs2<kBF16>(w.x, w.y), max_abs2<kBF16>(w.z, w.w));
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

// The codes of two words' four values times `inv`.
template <bool kBF16>
__device__ __forceinline__ uint32_t codes4(uint32_t x, uint32_t y, float inv) {
    float a, b, c, d;
    unpack2<kBF16>(x, a, b);
    unpack2<kBF16>(y, c, d);
    uint32_t r;
    asm("{\n.reg .b16 p, q;\ncvt.rn.satfinite.e4m3x2.f32 p, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 q, %4, %3;\n"
        "mov.b32 %0, {p, q};\n}"
        : "=r"(r)
        : "f"(a * inv), "f"(b * inv), "f"(c * inv), "f"(d * inv));
    return r;
}

template <bool kBF16>
__device__ __forceinline__ uint2 codes8(const uint4& w, float inv) {
    return {codes4<kBF16>(w.x, w.y, inv), codes4<kBF16>(w.z, w.w, inv)};
}

// The same with NaN in the place of what is not finite.
template <bool kBF16>
__device__ __noinline__ uint2 codes8_nan(uint4 w, float inv) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
    uint32_t c[2];
    for (int i = 0; i < 2; ++i) {
        const uint32_t b0 = nonfinite<kBF16>(r[2 * i]), b1 = nonfinite<kBF16>(r[2 * i + 1]);
        c[i] = codes4<kBF16>(r[2 * i] & ~b0, r[2 * i + 1] & ~b1, inv);
        const uint32_t bad = __byte_perm(b0, b1, 0x6420);  // a byte of each mask's halves
        c[i] = (c[i] & ~bad) | (0x7f7f7f7fu & bad);
    }
    return {c[0], c[1]};
}

template <bool kBF16>
__device__ __forceinline__ uint4 finite_only(const uint4& w) {
    return {w.x & ~nonfinite<kBF16>(w.x), w.y & ~nonfinite<kBF16>(w.y), w.z & ~nonfinite<kBF16>(w.z),
            w.w & ~nonfinite<kBF16>(w.w)};
}

// Quantises a K and a V row held by the G lanes of a group, 8 values of each a lane (all lanes of
// the warp take part): the scale bytes and the lane's 8 codes of each.  The instructions of this
// kernel bound it more than HBM does (with 140 for a lane's 8 values the ALU ran at 68 % of its
// rate and the kernel at 57 % of a copy's; now 53 % and 88 %), so the largest magnitudes are
// found on 16-bit pairs and both rows' reduced in one word.
// A value that is not finite takes no part in the scale and becomes NaN (e4m3 has no
// infinity): an overflow upstream stays visible.
template <int G, bool kBF16>
__device__ __forceinline__ void quantise(const uint4& wk, const uint4& wv, uint32_t& sk, uint32_t& sv, uint2& ck,
                                         uint2& cv) {
    constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
    uint32_t m = group_max<G, kBF16>(lane_max<kBF16>(wk), lane_max<kBF16>(wv));
    // a half at or past kInf carries into its top bit
    const bool odd = __any_sync(0xffffffffu, ((m + (0x8000u - kInf) * 0x10001u) & 0x80008000u) != 0);
    if (odd) m = group_max<G, kBF16>(lane_max<kBF16>(finite_only<kBF16>(wk)), lane_max<kBF16>(finite_only<kBF16>(wv)));
    sk = kv8_scale_byte<kBF16>(m & 0xffffu);
    sv = kv8_scale_byte<kBF16>(m >> 16);
    const float ik = kv8_inv_scale(sk), iv = kv8_inv_scale(sv);
    ck = odd ? codes8_nan<kBF16>(wk, ik) : codes8<kBF16>(wk, ik);
    cv = odd ? codes8_nan<kBF16>(wv, iv) : codes8<kBF16>(wv, iv);
}

template <int D, int U, bool kBF16>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Kv8AppendArgs a) {
    using C = AppendCfg<D, U>;
    __shared__ int cu[kMaxB + 1];
    __shared__ long long place[U == 1 ? 1 : C::Run + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int Hkv = a.pool.Hkv;
    const long long rows = (long long)a.total * Hkv, first = (long long)blockIdx.x * C::Run;
    const int t0 = (int)(first / Hkv);  // the run's first token
    const int h0 = (int)(first - (long long)t0 * Hkv);
    const int lane_g = threadIdx.x % C::G, group = threadIdx.x / C::G;
    int tok[U], head[U];  // the row's token, counted from t0
    uint4 wk[U], wv[U];
    const int tok_step = C::Groups / Hkv, head_step = C::Groups - tok_step * Hkv;
    const bool lanes = lane_g * 8 < D;
    const int left = (int)min(rows - first - group, (long long)C::Run);  // rows of this group: u * Groups < left
    const uint16_t* kp = static_cast<const uint16_t*>(a.k_new) + lane_g * 8;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v_new) + lane_g * 8;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u == 0) {
            tok[0] = (h0 + group) / Hkv;
            head[0] = h0 + group - tok[0] * Hkv;
        } else {
            head[u] = head[u - 1] + head_step;
            tok[u] = tok[u - 1] + tok_step;
            if (head[u] >= Hkv) {
                head[u] -= Hkv;
                ++tok[u];
            }
        }
        wk[u] = wv[u] = make_uint4(0, 0, 0, 0);
        if (u * C::Groups < left && lanes) {
            wk[u] = load_once(kp + (t0 + tok[u]) * a.k_stride + (long long)head[u] * D);
            wv[u] = load_once(vp + (t0 + tok[u]) * a.v_stride + (long long)head[u] * D);
        }
    }
    if (a.cu) {
        for (int i = threadIdx.x; i <= a.B; i += kThreads) cu[i] = a.cu[i];
        __syncthreads();
    }
    // The n new tokens are the last n of the sequence's kv_lens[b] keys.
    auto find = [&](int t) -> long long {
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
        return i >= 0 ? place_of(a.pool, b, (long long)a.kv_lens[b] - n + i) : kNoSequence;
    };
    long long mine = kNoSequence;
    if constexpr (U == 1) {
        if (left > 0) mine = find(t0 + tok[0]);
    } else {
        const long long last = first + C::Run - 1 < rows ? first + C::Run - 1 : rows - 1;
        const int tokens = (int)(last / Hkv) - t0 + 1;
        if (threadIdx.x < tokens) place[threadIdx.x] = find(t0 + threadIdx.x);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint2 ck, cv;
        uint32_t sk, sv;
        quantise<C::G, kBF16>(wk[u], wv[u], sk, sv, ck, cv);
        if (u * C::Groups >= left || !lanes) continue;
        const long long at = U == 1 ? mine : place[tok[u]];
        if (at < 0) continue;
        const long long r = at + (long long)head[u] * a.pool.page_size;
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

template <int D, int U>
struct ReadCfg {
    static constexpr int PerRow = D / 8;                       // threads of one row, 8 values each
    static constexpr int Groups = kThreads / PerRow;           // 10 rows at D = 96, 8 threads idle
    static constexpr int Run = Groups * U;
};

template <int D, int U, bool kBF16>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8ReadArgs a) {
    using C = ReadCfg<D, U>;
    __shared__ int cu[kMaxB + 1];
    __shared__ long long place[U == 1 ? 1 : C::Run + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int Hkv = a.pool.Hkv;
    const long long rows = (long long)a.total * Hkv, first = (long long)blockIdx.x * C::Run;
    const int t0 = (int)(first / Hkv);
    for (int i = threadIdx.x; i <= a.B; i += kThreads) cu[i] = a.cu[i];
    __syncthreads();
    auto find = [&](int t) -> long long {
        const int b = sequence_of(cu, a.B, t);
        return b < a.B && t >= cu[b] ? place_of(a.pool, b, (long long)(a.starts ? a.starts[b] : 0) + (t - cu[b]))
                                     : kNoSequence;
    };
    if constexpr (U > 1) {
        const long long last = first + C::Run - 1 < rows ? first + C::Run - 1 : rows - 1;
        const int tokens = (int)(last / Hkv) - t0 + 1;
        if (threadIdx.x < tokens) place[threadIdx.x] = find(t0 + threadIdx.x);
        __syncthreads();
    }
    const int group = threadIdx.x / C::PerRow, c8 = threadIdx.x % C::PerRow * 8;
    if (group >= C::Groups) return;
    bool owned[U];  // rows of no sequence are left as they were
    uint2 ck[U], cv[U];
    uint32_t sk[U], sv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long row = first + u * C::Groups + group;
        owned[u] = false;
        ck[u] = cv[u] = make_uint2(0, 0);
        sk[u] = sv[u] = 0;
        if (row >= rows) continue;
        const int t = (int)(row / Hkv), h = (int)(row - (long long)t * Hkv);
        const long long at = U == 1 ? find(t) : place[t - t0];
        owned[u] = at != kNoSequence;
        if (at < 0) continue;
        const long long r = at + (long long)h * a.pool.page_size;
        ck[u] = *reinterpret_cast<const uint2*>(a.pool.k + r * D + c8);
        cv[u] = *reinterpret_cast<const uint2*>(a.pool.v + r * D + c8);
        sk[u] = a.pool.ks[r];
        sv[u] = a.pool.vs[r];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!owned[u]) continue;
        const size_t to = (size_t)(first + u * C::Groups + group) * D + c8;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + to) = dequantise8<kBF16>(ck[u], kv8_scale(sk[u]));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + to) = dequantise8<kBF16>(cv[u], kv8_scale(sv[u]));
    }
}

// Rows of a group: more of them for the loads in flight where the rows fill the SMs many times
// over, one where they do not, since then a CTA's latency is what a call takes.  Measured, in
// microseconds for 1, 2 and 4 rows: append of 540672 rows of 128 92.5, 69.5, 69.4 (61.3 at the rate
// of a copy), of 42936 rows of 96 8.7, 7.2, 8.1, of 64 rows of 128 2.2, 2.7, 3.3; read of 540672
// rows of 128 81.3, 66.4, 64.6 (61.3).
int rows_of_a_group(long long rows, int groups, int num_sms) {
    const long long waves = rows / ((long long)groups * num_sms);
    return waves >= 64 ? 4 : waves >= 8 ? 2 : 1;
}

template <int D, int U>
fa_status append_u(const Kv8AppendArgs& a, cudaStream_t s) {
    constexpr int run = AppendCfg<D, U>::Run;
    const unsigned grid = (unsigned)(((long long)a.total * a.pool.Hkv + run - 1) / run);
    return a.bf16 ? launch_overlapped(kv8_append_kernel<D, U, true>, grid, kThreads, 0, s, a)
                  : launch_overlapped(kv8_append_kernel<D, U, false>, grid, kThreads, 0, s, a);
}

template <int D>
fa_status append_d(const Kv8AppendArgs& a, cudaStream_t s) {
    switch (rows_of_a_group((long long)a.total * a.pool.Hkv, AppendCfg<D, 1>::Groups, a.num_sms)) {
        case 4: return append_u<D, 4>(a, s);
        case 2: return append_u<D, 2>(a, s);
        default: return append_u<D, 1>(a, s);
    }
}

template <int D, int U>
fa_status read_u(const Kv8ReadArgs& a, cudaStream_t s) {
    constexpr int run = ReadCfg<D, U>::Run;
    const unsigned grid = (unsigned)(((long long)a.total * a.pool.Hkv + run - 1) / run);
    return a.bf16 ? launch_overlapped(kv8_read_kernel<D, U, true>, grid, kThreads, 0, s, a)
                  : launch_overlapped(kv8_read_kernel<D, U, false>, grid, kThreads, 0, s, a);
}

template <int D>
fa_status read_d(const Kv8ReadArgs& a, cudaStream_t s) {
    switch (rows_of_a_group((long long)a.total * a.pool.Hkv, ReadCfg<D, 1>::Groups, a.num_sms)) {
        case 4: return read_u<D, 4>(a, s);
        case 2: return read_u<D, 2>(a, s);
        default: return read_u<D, 1>(a, s);
    }
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
