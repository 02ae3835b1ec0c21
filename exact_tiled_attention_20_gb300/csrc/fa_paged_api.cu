// fa_paged_api.cu -- C entry points of the 16-bit paged cache: the rotated append and the decodes
// under a draft tree or a window with sinks.  Argument checks, tensor maps and dispatch.
#include <cmath>

#include "fa_paged.cuh"

namespace fa {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, asked for until it is found.
EncodeTiledFn encoder() {
    static EncodeTiledFn known = nullptr;
    EncodeTiledFn fn = __atomic_load_n(&known, __ATOMIC_ACQUIRE);
    if (fn) return fn;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
        return nullptr;
    fn = reinterpret_cast<EncodeTiledFn>(p);
    __atomic_store_n(&known, fn, __ATOMIC_RELEASE);
    return fn;
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Rows of a partial result: those of a row block, at most two sub-tiles of 128.
long long part_rows(int Sq, int Hq, int Hkv) {
    const long long rows = (long long)(Hq / Hkv) * Sq;
    return rows < 256 ? rows : 256;
}

// Checks of the pool that the entry points share.
fa_status check_pool(const void* k_pages, const void* v_pages, const int32_t* table, const int32_t* kv_lens, int B,
                     int Hkv, int D, int num_pages, int page_size, int max_pages, fa_dtype dtype) {
    if (!k_pages || !v_pages || !table || !kv_lens) return FA_ERR_INVALID_ARG;
    if (misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(table, 4) || misaligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    if (D != 64 && D != 96 && D != 128 && D != 256) return FA_ERR_UNSUPPORTED;
    if (B > 1024 || Hkv > 65536 || page_size > (1 << 28)) return FA_ERR_UNSUPPORTED;
    // Keys are counted in 32 bits, a little past the last one.
    if ((long long)page_size * max_pages > 0x7fffffffLL - 4095) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

fa_status decode(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                 const int32_t* kv_lens, const int32_t* tree, void* o, float* lse, int B, int Sq, int Hq, int Hkv, int D,
                 int num_pages, int page_size, int max_pages, float scale, int window_left, int sinks, void* workspace,
                 size_t workspace_bytes, fa_dtype dtype, fa_stream_t stream) {
    const fa_status chk = check_pool(k_pages, v_pages, block_table, kv_lens, B, Hkv, D, num_pages, page_size, max_pages,
                                     dtype);
    if (chk != FA_OK) return chk;
    if (!q || !o || misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4)) return FA_ERR_INVALID_ARG;
    if (Sq <= 0 || Hq <= 0 || Hq % Hkv != 0 || !std::isfinite(scale) || scale <= 0.f) return FA_ERR_INVALID_ARG;
    if (window_left < -1 || sinks < 0) return FA_ERR_INVALID_ARG;
    if (page_size % 16 != 0 || Sq > 256 || Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
    if ((long long)Sq * Hq * D > 0x7fffffffLL || (long long)B * Sq * Hq > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    // A tensor map's strides stay below 2^40 bytes, and a page past the last one is a coordinate.
    if ((long long)page_size * Hkv * D * 2 >= (1LL << 40) || num_pages == 0x7fffffff) return FA_ERR_UNSUPPORTED;
    int sms = 0;
    int* status = nullptr;
    if (!current_device(&sms, &status)) return FA_ERR_CUDA;
    if (!workspace || misaligned(workspace, 16) ||
        workspace_bytes < fa_decode_paged_workspace_bytes(B, Sq, Hq, Hkv, D, sms))
        return FA_ERR_WORKSPACE;
    const int capacity = page_size * max_pages;
    if (window_left >= capacity) window_left = -1;
    if (sinks > capacity) sinks = capacity;
    const size_t rows = (size_t)(2LL * sms * part_rows(Sq, Hq, Hkv));
    char* part = static_cast<char*>(workspace) + (misaligned(workspace, 32) ? 16 : 0);
    float* o_part = reinterpret_cast<float*>(part);
    float* lse_part = reinterpret_cast<float*>(part + up256(rows * D * sizeof(float)));
    const PagedDecodeArgs a{q, k_pages, v_pages, block_table, kv_lens, tree, o, lse, B, Sq, Hq, Hkv, D, num_pages,
                            page_size, max_pages, scale, window_left, sinks, o_part, lse_part, dtype == FA_BF16, sms,
                            status};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (D) {
        case 64: return launch_paged_decode_d64(a, s);
        case 96: return launch_paged_decode_d96(a, s);
        case 128: return launch_paged_decode_d128(a, s);
        default: return launch_paged_decode_d256(a, s);
    }
}

}  // namespace

bool encode_paged_tmap(CUtensorMap* map, const void* base, bool bf16, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                       uint64_t dim3, uint32_t box1, uint32_t box2) {
    const EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {dim0, dim1, dim2, dim3};
    const cuuint64_t strides[3] = {dim0 * 2, dim0 * dim1 * 2, dim0 * dim1 * dim2 * 2};
    const cuuint32_t box[4] = {64, box1, box2, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_kv_append_paged_rope(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                                  int64_t k_stride, int64_t v_stride, void* q_out, const int32_t* cu_seqlens_new,
                                  const int32_t* block_table, const int32_t* kv_lens, const int32_t* positions,
                                  const float* cos, const float* sin, void* k_pages, void* v_pages, int B, int total_new,
                                  int Hq, int Hkv, int D, int rot_dim, int interleaved, int max_pos, int num_pages,
                                  int page_size, int max_pages_per_seq, fa_dtype dtype, fa_stream_t stream) {
    const fa_status chk = check_pool(k_pages, v_pages, block_table, kv_lens, B, Hkv, D, num_pages, page_size,
                                     max_pages_per_seq, dtype);
    if (chk != FA_OK) return chk;
    if (misaligned(cu_seqlens_new, 4) || misaligned(positions, 4)) return FA_ERR_INVALID_ARG;
    if (total_new < 0 || Hq < 0 || (!cu_seqlens_new && total_new % B != 0)) return FA_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0) return FA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!cos || !sin || misaligned(cos, 16) || misaligned(sin, 16) || max_pos <= 0))
        return FA_ERR_INVALID_ARG;
    if (total_new == 0) return FA_OK;
    if (!k_new || !v_new || misaligned(k_new, 16) || misaligned(v_new, 16)) return FA_ERR_INVALID_ARG;
    const long long width = (long long)Hkv * D, q_width = (long long)Hq * D;
    if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0) return FA_ERR_INVALID_ARG;
    if (Hq > 0 && (!q || !q_out || misaligned(q, 16) || misaligned(q_out, 16) || q_stride < q_width || q_stride % 8 != 0))
        return FA_ERR_INVALID_ARG;
    if ((long long)total_new * ((long long)Hq + 2LL * Hkv) > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    int sms = 0;
    int* status = nullptr;
    if (!current_device(&sms, &status)) return FA_ERR_CUDA;
    const PagedAppendArgs a{q, k_new, v_new, q_stride, k_stride, v_stride, q_out, cu_seqlens_new, block_table, kv_lens,
                            positions, cos, sin, k_pages, v_pages, B, total_new, Hq, Hkv, D, rot_dim,
                            interleaved ? 1 : 0, max_pos, num_pages, page_size, max_pages_per_seq, dtype == FA_BF16,
                            sms};
    return launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_decode_paged_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int num_sms) {
    if (B <= 0 || Sq <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return 0;
    if (num_sms <= 0) {
        int* status = nullptr;
        if (!current_device(&num_sms, &status)) return 0;
    }
    const size_t rows = (size_t)(2LL * num_sms * part_rows(Sq, Hq, Hkv));
    return up256(rows * D * sizeof(float)) + up256(rows * sizeof(float)) + 16;  // 16: to a 32-byte boundary
}

fa_status fa_decode_splitkv_paged_tree(const void* q, const void* k_pages, const void* v_pages,
                                       const int32_t* block_table, const int32_t* kv_lens, const int32_t* tree_mask,
                                       void* o, float* lse, int B, int Sq, int Hq, int Hkv, int D, int num_pages,
                                       int page_size, int max_pages_per_seq, float scale, void* workspace,
                                       size_t workspace_bytes, fa_dtype dtype, fa_stream_t stream) {
    if (!tree_mask || misaligned(tree_mask, 4)) return FA_ERR_INVALID_ARG;
    return decode(q, k_pages, v_pages, block_table, kv_lens, tree_mask, o, lse, B, Sq, Hq, Hkv, D, num_pages, page_size,
                  max_pages_per_seq, scale, -1, 0, workspace, workspace_bytes, dtype, stream);
}

fa_status fa_decode_splitkv_paged_window(const void* q, const void* k_pages, const void* v_pages,
                                         const int32_t* block_table, const int32_t* kv_lens, void* o, float* lse, int B,
                                         int Sq, int Hq, int Hkv, int D, int num_pages, int page_size,
                                         int max_pages_per_seq, float scale, int window_left, int sinks,
                                         void* workspace, size_t workspace_bytes, fa_dtype dtype, fa_stream_t stream) {
    return decode(q, k_pages, v_pages, block_table, kv_lens, nullptr, o, lse, B, Sq, Hq, Hkv, D, num_pages, page_size,
                  max_pages_per_seq, scale, window_left, sinks, workspace, workspace_bytes, dtype, stream);
}

}  // extern "C"
