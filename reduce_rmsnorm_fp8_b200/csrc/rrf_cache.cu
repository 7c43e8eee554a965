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
// later row goes on from there.  Then L lanes take a row (L a power of two, 32
// unless a row's keys are fewer than 32 vectors of 16 codes), its keys and
// values together, so that each lane has several loads in flight.  B200, 131072
// rows x 8 heads x 128: 132 us, 94% of the copy rate (138 with keys and values
// apart and 16-byte stores); a few rows: 3.3 us, a launch and three dependent
// trips to memory.
#include <cuda_runtime.h>

#include "rrf_device.cuh"
#include "rrf_internal.h"

namespace rrf {
namespace {

constexpr int kReadThreads = 256;
constexpr int kRowsPerLaneGroup = 2;  // rows that a group of L lanes takes in turn

// 16 codes times a scale as 16 bf16: one store of 32 bytes where the outputs
// are aligned to it (`whole`), else two.
__device__ __forceinline__ void store_wide(uint16_t* out, const uint4 q, float scale, bool whole) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
            const float2 f = __fmul2_rn(__half22float2(__half2(h)), make_float2(scale, scale));
            o[2 * i + j] = f32x2_to_bf16x2(f.x, f.y);
        }
    }
    if (!whole) {
        st_once(reinterpret_cast<uint4*>(out), make_uint4(o[0], o[1], o[2], o[3]));
        st_once(reinterpret_cast<uint4*>(out) + 1, make_uint4(o[4], o[5], o[6], o[7]));
        return;
    }
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(out), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]),
                    "r"(o[6]), "r"(o[7])
                 : "memory");
}

// The slot of a row: the offsets of its codes (or -1: the row is left alone)
// and scales.  `s` is a sequence that does not begin after the row.
__device__ __forceinline__ longlong2 slot_of(const CacheReadArgs& a, int row, int s) {
    longlong2 at = {-1, 0};
    if (row >= a.rows) return at;
    while (s < a.sequences && a.seq_starts[s + 1] <= row) ++s;
    if (s >= a.sequences) return at;
    const int t = row - a.seq_starts[s];
    if (t < 0) return at;  // before the first sequence
    const int p = t / a.page_size;
    const int page = p < a.table_width ? a.block_table[s * a.table_stride + p] : -1;
    if (page < 0 || page >= a.num_pages) {
        atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
        return at;
    }
    const int place = t - p * a.page_size;
    at.x = page * a.code_page + place * a.code_slot;
    at.y = page * a.scale_page + place * a.scale_slot;
    return at;
}

template <int L>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheReadArgs a) {
    constexpr int kGroups = kReadThreads / L;
    constexpr int kRows = kGroups * kRowsPerLaneGroup;  // of a block
    __shared__ int ended;
    __shared__ longlong2 slots[kRows];
    wait_for_previous_grid();  // see rrf_device.cuh: programmatic dependent launch
    allow_next_grid();
    const int tid = opaque((int)threadIdx.x);
    const int row0 = (int)blockIdx.x * kRows;
    if (tid == 0) ended = 0;
    __syncthreads();
    int n = 0;
    for (int s = tid; s < a.sequences; s += kReadThreads) n += a.seq_starts[s + 1] <= row0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if ((tid & 31) == 0 && n != 0) atomicAdd(&ended, n);
    __syncthreads();
    for (int r = tid; r < kRows; r += kReadThreads) slots[r] = slot_of(a, row0 + r, ended);
    __syncthreads();

    const int per_head = a.dim / 16;
    const int per_row = a.heads * per_head;  // 16-code vectors of a row's keys
    const int group = tid / L, lane = tid % L;
#pragma unroll
    for (int i = 0; i < kRowsPerLaneGroup; ++i) {
        const int r = group + i * kGroups;
        const longlong2 at = slots[r];
        if (at.x < 0) continue;
        const int64_t out = (int64_t)(row0 + r) * per_row * 16;
#pragma unroll 2
        for (int e = lane; e < per_row; e += L) {
            // e / per_head (e < 2^17, per_head <= 32: exact)
            const int head = per_head == 1 ? e : (int)__umulhi((uint32_t)e, a.head_magic);
            const int64_t code = at.x + head * a.code_head + (e - head * per_head) * 16;
            const int64_t scale = at.y + head * a.scale_head;
            if (!RRF_IN_BOUNDS(row0 + r < a.rows && head < a.heads && code >= 0 &&
                                   code + 16 <= a.code_end && scale >= 0 && scale < a.scale_end,
                               a.err))
                continue;
            const uint4 kq = ld_once(reinterpret_cast<const uint4*>(a.k_codes + code));
            const uint4 vq = ld_once(reinterpret_cast<const uint4*>(a.v_codes + code));
            const float ks = a.k_scales[scale], vs = a.v_scales[scale];
            store_wide(a.k_out + out + e * 16, kq, ks, a.whole);
            store_wide(a.v_out + out + e * 16, vq, vs, a.whole);
        }
    }
}

template <int L>
cudaError_t launch_lanes(const CacheReadArgs& a, cudaStream_t stream) {
    constexpr int kRows = kReadThreads / L * kRowsPerLaneGroup;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows + kRows - 1) / kRows), 1, 1);
    cfg.blockDim = dim3(kReadThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_read_kernel<L>, a);
}

}  // namespace

cudaError_t launch_cache_read(CacheReadArgs a, cudaStream_t stream) {
    const int per_head = a.dim / 16, per_row = a.heads * per_head;
    a.whole = (((uintptr_t)a.k_out | (uintptr_t)a.v_out) & 31) == 0;
    a.head_magic = (uint32_t)((((uint64_t)1 << 32) + per_head - 1) / per_head);
    if (per_row >= 32) return launch_lanes<32>(a, stream);
    if (per_row >= 16) return launch_lanes<16>(a, stream);
    if (per_row >= 8) return launch_lanes<8>(a, stream);
    return launch_lanes<4>(a, stream);
}

}  // namespace rrf
