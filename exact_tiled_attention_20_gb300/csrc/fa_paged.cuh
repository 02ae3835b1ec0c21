// fa_paged.cuh -- what the kernels over the 16-bit paged cache share: their arguments.
//
//     k_pages, v_pages  [num_pages, page_size, Hkv, D]
//     block_table       [B, max_pages]: key r of sequence b is row r % page_size of page
//                       block_table[b][r / page_size]
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_kv8.cuh"  // launch_overlapped, grid_dependency_wait
#include "fa_ptx.cuh"

namespace fa {

struct PagedAppendArgs {
    const void* q;  // token t, head h: q + t * q_stride + h * D (elements); null where Hq is 0
    const void* k_new;
    const void* v_new;
    long long q_stride, k_stride, v_stride;
    void* q_out;               // [total, Hq, D]
    const int32_t* cu;         // [B + 1] or null: total / B tokens each
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* positions;  // [total] or null: a token's position is its key
    const float* cos;          // [max_pos, rot / 2]
    const float* sin;
    void* k_pages;
    void* v_pages;
    int B, total, Hq, Hkv, D, rot, interleaved, max_pos, num_pages, page_size, max_pages;
    bool bf16;
    int num_sms;
};

struct PagedDecodeArgs {
    const void* q;  // [B, Sq, Hq, D]
    const void* k_pages;
    const void* v_pages;
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* tree;  // [B, Sq, (Sq + 31) / 32] or null: causal with a window
    void* o;
    float* lse;  // [B, Hq, Sq] or null
    int B, Sq, Hq, Hkv, D, num_pages, page_size, max_pages;
    float scale;
    int window_left, sinks;  // -1: unbounded
    float* o_part;
    float* lse_part;
    bool bf16;
    int num_sms;
    int* dev_status;
};

fa_status launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);
// One translation unit per head dim, compiled in parallel.
fa_status launch_paged_decode_d64(const PagedDecodeArgs& a, cudaStream_t s);
fa_status launch_paged_decode_d96(const PagedDecodeArgs& a, cudaStream_t s);
fa_status launch_paged_decode_d128(const PagedDecodeArgs& a, cudaStream_t s);
fa_status launch_paged_decode_d256(const PagedDecodeArgs& a, cudaStream_t s);

}  // namespace fa
