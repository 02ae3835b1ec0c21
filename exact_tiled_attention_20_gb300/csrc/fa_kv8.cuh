// fa_kv8.cuh -- the 8-bit paged KV cache: its format, and what its kernels share.
//
// A cache row is one token's D values of one kv head, held as e4m3 codes with one scale
// 2^(s - 127), s a byte:
//     k_pages, v_pages    [num_pages, Hkv, page_size, D]   codes
//     k_scales, v_scales  [num_pages, Hkv, page_size]      exponent bytes s
// page_size is a multiple of 16, so 16 consecutive keys that start at a multiple of 16 are
// one aligned run of 16 D bytes of codes and of 16 bytes of scales.  The head comes before
// the slot (unlike the 16-bit pools, [num_pages, page_size, Hkv, D]): a CTA of the decode
// streams one head, whose codes are then whole runs of memory and not one 64..256-byte row
// in every Hkv of them.
//
// The scale is a power of two because e4m3 keeps its relative precision over its binades:
// a finer scale would gain nothing but range, while with this one the division by the
// scale, and the multiplication when the row is read, are exact.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

struct Kv8Pool {
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;
    uint8_t* vs;
    const int32_t* table;  // [B, max_pages]
    int Hkv, num_pages, page_size, max_pages;
};

struct Kv8AppendArgs {
    Kv8Pool pool;
    const void* k_new;  // token t, head h: k_new + t * k_stride + h * D (elements)
    const void* v_new;
    long long k_stride, v_stride;
    const int32_t* cu;  // [B + 1] or null: total / B tokens each
    const int32_t* kv_lens;
    int B, total, D;
    bool bf16;
    int num_sms;
};

struct Kv8ReadArgs {
    Kv8Pool pool;
    void* k;  // [total, Hkv, D]
    void* v;
    const int32_t* cu;      // [B + 1]
    const int32_t* starts;  // [B] or null: 0
    int B, total, D;
    bool bf16;
    int num_sms;
};

struct Kv8DecodeArgs {
    Kv8Pool pool;
    const void* q;  // [B, Sq, Hq, D]
    void* o;
    float* lse;  // [B, Hq, Sq] or null
    const int32_t* kv_lens;
    int B, Sq, Hq, D;
    float scale;
    int causal;
    long long slots;  // room in the workspace: partial results of one pair; 0: cut no pair
    float* o_part;    // [slots, Hq / Hkv * Sq, D]
    float* lse_part;  // [slots, Hq / Hkv * Sq]
    bool bf16;
    int num_sms;
};

fa_status launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s);
fa_status launch_kv8_read(const Kv8ReadArgs& a, cudaStream_t s);
// One translation unit per head dim, compiled in parallel.
fa_status launch_kv8_decode_d64(const Kv8DecodeArgs& a, cudaStream_t s);
fa_status launch_kv8_decode_d96(const Kv8DecodeArgs& a, cudaStream_t s);
fa_status launch_kv8_decode_d128(const Kv8DecodeArgs& a, cudaStream_t s);
fa_status launch_kv8_decode_d256(const Kv8DecodeArgs& a, cudaStream_t s);

// Launches `kern` so that its start may overlap the end of the kernel before it on the
// stream; the kernel itself waits (grid_dependency_wait), in every thread, before it writes global
// memory or uses what that kernel may write.  What may be read earlier: by the split kernel lengths
// and table entries, for a guess that it checks after the wait and that decides nothing but which
// lines of the pool go to L2 (indices are held inside the table and the pool whatever they are);
// by the merge kernel the lengths, since every CTA of the split kernel before it lets it start
// only after its own wait, when all that came before is done.
template <typename... P, typename... A>
inline fa_status launch_overlapped(void (*kern)(P...), unsigned grid, unsigned block, size_t smem,
                                   cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return FA_OK;
    cudaGetLastError();  // reported here, not by the caller's next call
    return FA_ERR_CUDA;
}

// Everything that earlier kernels of the stream wrote is visible after this.
__device__ __forceinline__ void grid_dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The next kernel of the stream may start to launch.
__device__ __forceinline__ void grid_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 2^(s - 127) of a scale byte: s is a float's exponent field, but for 0 (2^-127, subnormal).
__device__ __forceinline__ float kv8_scale(uint32_t s) {
    return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// The scale byte of a row from the 16 bits of its largest finite magnitude: the least
// e >= -127 with amax <= 448 * 2^e, plus 127.  448 = 1.75 * 2^8 is e4m3's largest value, so with
// amax = f * 2^x, 1 <= f < 2, e = x - 8, and one more where f > 1.75: adding a quarter less one
// step to the fraction carries into the exponent just then.  (bf16's own subnormals have a zero
// exponent field and e = -127; fp16's are normal in fp32.)
template <bool kBF16>
__device__ __forceinline__ uint32_t kv8_scale_byte(uint32_t amax16) {
    int x;
    if constexpr (kBF16) {
        x = (int)((amax16 + 0x1fu) >> 7);
    } else {
        float f;
        asm("{\n.reg .b16 a;\ncvt.u16.u32 a, %1;\ncvt.f32.f16 %0, a;\n}" : "=f"(f) : "r"(amax16));
        x = (int)((__float_as_uint(f) + 0x1fffffu) >> 23);
    }
    return (uint32_t)max(x - 8, 0);
}

// 2^(127 - s), the exact factor that the codes are taken at; s <= 247.
__device__ __forceinline__ float kv8_inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Two e4m3 codes (low byte first) -> f16x2, exactly (NaN codes become NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(codes));
    return d;
}

// Two floats -> e4m3 codes, round to nearest even; `lo` in the low byte.
__device__ __forceinline__ uint16_t e4m3x2_from_floats(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

}  // namespace fa
