// rrf_cache.cu -- reading a paged FP8 cache back: the keys and values of a
// batch of sequences, one sequence after the other, as bf16,
//   out[seq_starts[s] + t][h][:] = RN_bf16(code * scale)
// with the codes and scale of head h in slot t % page_size of page
// block_table[s][t / page_size].
//
// A gather with one product per value: 1 byte in and 2 out, bound by HBM.  A
// block takes a run of output rows.  It first finds their slots, one thread
// per row: the sequence of the run's first row is the number of sequences
// that end at or before it, counted by the whole block in one sweep of
// seq_starts (a binary search would be a chain of dependent loads), and a
// later row goes on from there.  Then its threads take 16 codes at a time.
#include <cuda_runtime.h>

#include "rrf_device.cuh"
#include "rrf_internal.h"

namespace rrf {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // rows of a block

// 16 codes times a scale as 16 bf16.
__device__ __forceinline__ void widen16(const uint4 q, float scale, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            o[2 * i + j] =
                f32x2_to_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheReadArgs a) {
    __shared__ int ended;
    __shared__ int64_t slot_codes[kReadRows];   // code offset of a row's slot, or -1
    __shared__ int64_t slot_scales[kReadRows];
    wait_for_previous_grid();
    allow_next_grid();
    const int tid = opaque((int)threadIdx.x);
    const int row0 = (int)blockIdx.x * kReadRows;
    if (tid == 0) ended = 0;
    __syncthreads();
    int n = 0;
    for (int s = tid; s < a.sequences; s += kReadThreads) n += a.seq_starts[s + 1] <= row0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if ((tid & 31) == 0 && n != 0) atomicAdd(&ended, n);
    __syncthreads();
    if (tid < kReadRows) {
        const int row = row0 + tid;
        int64_t code_at = -1, scale_at = 0;
        int s = ended;
        if (row < a.rows) {
            while (s < a.sequences && a.seq_starts[s + 1] <= row) ++s;
            if (s < a.sequences) {
                const int t = row - a.seq_starts[s];
                if (t >= 0) {  // (rows before the first sequence are left alone)
                    const int p = t / a.page_size;
                    const int page =
                        p < a.table_width ? a.block_table[s * a.table_stride + p] : -1;
                    if (page < 0 || page >= a.num_pages) {
                        atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
                    } else {
                        const int place = t - p * a.page_size;
                        code_at = page * a.code_page + place * a.code_slot;
                        scale_at = page * a.scale_page + place * a.scale_slot;
                    }
                }
            }
        }
        slot_codes[tid] = code_at;
        slot_scales[tid] = scale_at;
    }
    __syncthreads();

    const int per_head = a.dim / 16;
    const int per_row = a.heads * per_head;  // 16-code vectors of a row's keys
    const int items = kReadRows * per_row;
    for (int i = tid; i < 2 * items; i += kReadThreads) {
        const bool key = i < items;
        const int j = key ? i : i - items;
        const int r = j / per_row, e = j - r * per_row;
        const int64_t code_at = slot_codes[r];
        if (code_at < 0) continue;
        const int head = e / per_head, v = e - head * per_head;
        if (!RRF_IN_BOUNDS(row0 + r < a.rows && head < a.heads &&
                               code_at + head * a.code_head + a.dim <= a.code_end &&
                               slot_scales[r] + head * a.scale_head < a.scale_end,
                           a.err))
            continue;
        const uint4 q = ld_once(reinterpret_cast<const uint4*>(
            (key ? a.k_codes : a.v_codes) + code_at + head * a.code_head) + v);
        const float scale =
            (key ? a.k_scales : a.v_scales)[slot_scales[r] + head * a.scale_head];
        uint4 lo, hi;
        widen16(q, scale, lo, hi);
        uint4* out = reinterpret_cast<uint4*>(
            (key ? a.k_out : a.v_out) + ((int64_t)(row0 + r) * per_row + e) * 16);
        st_once(out, lo);
        st_once(out + 1, hi);
    }
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadArgs& a, int sm_count, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows + kReadRows - 1) / kReadRows), 1, 1);
    cfg.blockDim = dim3(kReadThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_read_kernel, a);
}

}  // namespace rrf
