// fa_kv8_api.cu -- C entry points of the 8-bit paged KV cache: argument checks and dispatch.
#include <cmath>

#include "fa_kv8.cuh"

namespace fa {
namespace {

// SMs of the current device, asked for once per device; 0 where it cannot be queried.
int device_sms() {
    static int known[64] = {0};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    sms = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
    if (sms > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    __atomic_store_n(&known[dev], sms, __ATOMIC_RELAXED);
    return sms;
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Checks of the pool that all three entry points share.
fa_status check_pool(const void* k_pages, const void* v_pages, const void* k_scales, const void* v_scales,
                     const int32_t* table, int B, int Hkv, int D, int num_pages, int page_size, int max_pages,
                     fa_dtype dtype) {
    if (!k_pages || !v_pages || !k_scales || !v_scales || !table) return FA_ERR_INVALID_ARG;
    if (misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(k_scales, 16) || misaligned(v_scales, 16) ||
        misaligned(table, 4))
        return FA_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    if (D != 64 && D != 96 && D != 128 && D != 256) return FA_ERR_UNSUPPORTED;
    if (page_size % 16 != 0 || B > 1024) return FA_ERR_UNSUPPORTED;
    // The kernels count keys (a little past the last one) and the pool's 16-key runs in 32 bits.
    if ((long long)page_size * max_pages > 0x7fffffffLL - 4095) return FA_ERR_UNSUPPORTED;
    if ((long long)num_pages * Hkv > 0x7fffffffLL / (page_size / 16)) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

Kv8Pool make_pool(const void* k_pages, const void* v_pages, const uint8_t* k_scales, const uint8_t* v_scales,
                  const int32_t* table, int Hkv, int num_pages, int page_size, int max_pages) {
    return {static_cast<uint8_t*>(const_cast<void*>(k_pages)),
            static_cast<uint8_t*>(const_cast<void*>(v_pages)),
            const_cast<uint8_t*>(k_scales),
            const_cast<uint8_t*>(v_scales),
            table,
            Hkv,
            num_pages,
            page_size,
            max_pages};
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_kv_append_paged_fp8(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                 const int32_t* cu_seqlens_new, const int32_t* block_table, const int32_t* kv_lens,
                                 void* k_pages, void* v_pages, uint8_t* k_scales, uint8_t* v_scales, int B,
                                 int total_new, int Hkv, int D, int num_pages, int page_size, int max_pages_per_seq,
                                 fa_dtype dtype, fa_stream_t stream) {
    const fa_status chk = check_pool(k_pages, v_pages, k_scales, v_scales, block_table, B, Hkv, D, num_pages,
                                     page_size, max_pages_per_seq, dtype);
    if (chk != FA_OK) return chk;
    if (!kv_lens || misaligned(kv_lens, 4) || misaligned(cu_seqlens_new, 4)) return FA_ERR_INVALID_ARG;
    if (total_new < 0 || (!cu_seqlens_new && total_new % B != 0)) return FA_ERR_INVALID_ARG;
    if (total_new == 0) return FA_OK;
    if (!k_new || !v_new || misaligned(k_new, 16) || misaligned(v_new, 16)) return FA_ERR_INVALID_ARG;
    const long long width = (long long)Hkv * D;
    if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0) return FA_ERR_INVALID_ARG;
    if ((long long)total_new * Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return FA_ERR_CUDA;
    const Kv8AppendArgs a{make_pool(k_pages, v_pages, k_scales, v_scales, block_table, Hkv, num_pages, page_size,
                                    max_pages_per_seq),
                          k_new, v_new, k_stride, v_stride, cu_seqlens_new, kv_lens, B, total_new, D,
                          dtype == FA_BF16, sms};
    return launch_kv8_append(a, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_kv_read_paged_fp8(const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                               const uint8_t* v_scales, const int32_t* block_table, const int32_t* kv_starts,
                               const int32_t* cu_seqlens, void* k, void* v, int B, int total, int Hkv, int D,
                               int num_pages, int page_size, int max_pages_per_seq, fa_dtype dtype,
                               fa_stream_t stream) {
    const fa_status chk = check_pool(k_pages, v_pages, k_scales, v_scales, block_table, B, Hkv, D, num_pages,
                                     page_size, max_pages_per_seq, dtype);
    if (chk != FA_OK) return chk;
    if (!cu_seqlens || misaligned(cu_seqlens, 4) || misaligned(kv_starts, 4) || total < 0) return FA_ERR_INVALID_ARG;
    if (total == 0) return FA_OK;
    if (!k || !v || misaligned(k, 16) || misaligned(v, 16)) return FA_ERR_INVALID_ARG;
    if ((long long)total * Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return FA_ERR_CUDA;
    const Kv8ReadArgs a{make_pool(k_pages, v_pages, k_scales, v_scales, block_table, Hkv, num_pages, page_size,
                                  max_pages_per_seq),
                        k, v, cu_seqlens, kv_starts, B, total, D, dtype == FA_BF16, sms};
    return launch_kv8_read(a, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_splitkv_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                                      const uint8_t* k_scales, const uint8_t* v_scales, const int32_t* block_table,
                                      const int32_t* kv_lens, void* o, float* lse, int B, int Sq, int Hq, int Hkv,
                                      int D, int num_pages, int page_size, int max_pages_per_seq, float scale,
                                      int causal, int num_splits, void* workspace, size_t workspace_bytes,
                                      fa_dtype dtype, fa_stream_t stream) {
    const fa_status pool_chk = check_pool(k_pages, v_pages, k_scales, v_scales, block_table, B, Hkv, D, num_pages,
                                          page_size, max_pages_per_seq, dtype);
    if (pool_chk != FA_OK) return pool_chk;
    if (!q || !kv_lens || !o) return FA_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(o, 16) || misaligned(kv_lens, 4) || misaligned(lse, 4)) return FA_ERR_INVALID_ARG;
    if (Sq <= 0 || Hq <= 0 || Hq % Hkv != 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
    if ((long long)(Hq / Hkv) * Sq > 16) return FA_ERR_UNSUPPORTED;
    const int capacity = page_size * max_pages_per_seq;
    // The plan counts 64-key units, and a few more for each (sequence, kv head) pair, in 32 bits.
    if ((long long)B * Hkv > 0x7fffffffLL / (capacity / 64 + 8)) return FA_ERR_UNSUPPORTED;
    if ((long long)B * Sq * Hq > 0x7fffffffLL - 8) return FA_ERR_UNSUPPORTED;  // the merge counts past the last row
    // The values of a sequence without keys are written by one CTA, which counts a little past them.
    if ((long long)Sq * Hq * D > 0x7fffffffLL - 255) return FA_ERR_UNSUPPORTED;
    // The bytes of the partial results (of each row D values and a log-sum-exp), in 64 bits.
    if (num_splits > 1 &&
        (long long)B * Sq * Hq * num_splits > (0x7fffffffffffffffLL - 512) / ((D + 1) * (int)sizeof(float)))
        return FA_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return FA_ERR_CUDA;
    const bool whole = num_splits == 1;
    if (num_splits <= 0) num_splits = fa_decode_default_splits(B, Hkv, capacity, sms);
    const size_t need = fa_decode_workspace_bytes(B * Sq, Hq, D, num_splits);
    if (!whole && (!workspace || workspace_bytes < need || misaligned(workspace, 16))) return FA_ERR_WORKSPACE;
    // The workspace holds num_splits partial results of every pair: [slots, Hq / Hkv * Sq, D] and
    // their log-sum-exps.
    const size_t rows = (size_t)B * Sq * Hq * num_splits;
    float* o_part = static_cast<float*>(workspace);
    float* lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                               ((rows * D * sizeof(float) + 255) & ~size_t(255)));
    const Kv8DecodeArgs a{make_pool(k_pages, v_pages, k_scales, v_scales, block_table, Hkv, num_pages, page_size,
                                    max_pages_per_seq),
                          q, o, lse, kv_lens, B, Sq, Hq, D, scale, causal,
                          whole ? 0 : (long long)B * Hkv * num_splits, o_part, lse_part, dtype == FA_BF16, sms};
    switch (D) {
        case 64: return launch_kv8_decode_d64(a, reinterpret_cast<cudaStream_t>(stream));
        case 96: return launch_kv8_decode_d96(a, reinterpret_cast<cudaStream_t>(stream));
        case 128: return launch_kv8_decode_d128(a, reinterpret_cast<cudaStream_t>(stream));
        default: return launch_kv8_decode_d256(a, reinterpret_cast<cudaStream_t>(stream));
    }
}

}  // extern "C"
