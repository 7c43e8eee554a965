// rrf_heads.cu -- per-head work between a layer's projection and its
// attention, one pass over the projection's output:
//   queries, keys   x -> rotate(x * rsqrt(mean(x^2) + eps) * (gamma + weight_offset)),
//                   written as bf16, or (keys) quantised into the cache
//   values          quantised into the cache
// with one scale per token and head, scale = max(min(max|x|, scale_ub), 1e-12) / 448,
// and the code the e4m3 value nearest to x / scale.
//
// The pass is a stream: 2 bytes in and 2 (bf16) or 1 (cache) bytes out per
// value, and some 10 instructions per value between them, so HBM bounds it
// once enough loads are in flight, and the launch and one round trip to
// memory bound a single token.  Nothing is exchanged between warps.
//
// Layout of the work.  A head is held by G lanes (the power of two that
// covers head_dim / 16), two 16-byte vectors of 8 values each; a warp takes
// 32 / G heads of one kind (a chunk) at a time, and U chunks are loaded
// before the first is worked on.  The two vectors of a lane are the partners
// of the rotation (vector j and j + rot_dim / 16 of the rotated part, and the
// same split of the part that is not rotated), so that a rotation never
// leaves its lane in either pairing, a lane needs 8 cosines and 8 sines for
// all the heads of its token, and neighbouring lanes load neighbouring
// vectors.
#include <cuda_runtime.h>

#include "rrf_device.cuh"
#include "rrf_internal.h"

namespace rrf {
namespace {

constexpr int kWarpsPerBlock = 4;

// Sum and maximum over the G lanes of a head (xor butterflies: every lane
// gets the same bits).
template <int G>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = 1; off < G; off <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

template <int G>
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
    for (int off = 1; off < G; off <<= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// The codes of x[16] under amax (already clamped).  A bf16 x and a bf16 amax
// often make x / scale = 448 x / amax an exact midpoint of the e4m3 grid, and
// a product with a rounded reciprocal would land on either side of it.  So
// the quotient n / amax (n = 448 x, exact for a bf16 x) is corrected once by
// its exact remainder (Markstein's final step: y + (n - y amax) / amax),
// which makes a representable quotient exact; two packed multiply-adds for
// two values.  Rows above 1e30 are scaled by 2^-64 first, so that 448 x stays
// finite, and values beyond a clamped amax are cut to it (they saturate).
__device__ __forceinline__ void quantise(float2 x[8], float amax, bool clamped, uint2& qa,
                                         uint2& qb) {
    if (clamped) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (a NaN stays one)
            x[i].x = x[i].x > amax ? amax : x[i].x < -amax ? -amax : x[i].x;
            x[i].y = x[i].y > amax ? amax : x[i].y < -amax ? -amax : x[i].y;
        }
    }
    const float down = amax > 1e30f ? 5.421010862427522e-20f : 1.0f;  // 2^-64
    const float d = amax * down, f = 448.0f * down, inv = 1.0f / d;
    const float2 inv2 = make_float2(inv, inv), f2 = make_float2(f, f);
    float2 y[8];
    if (d < __int_as_float(0x7F800000)) {
        const float2 minus_d = make_float2(-d, -d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 n = __fmul2_rn(x[i], f2);
            const float2 y0 = __fmul2_rn(n, inv2);
            y[i] = __ffma2_rn(__ffma2_rn(y0, minus_d, n), inv2, y0);
        }
    } else {  // an infinite scale: finite values are 0, infinities NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(x[i], inv2);
    }
    qa = f32x2_to_e4m3x8(y);
    qb = f32x2_to_e4m3x8(y + 4);
}

// The kinds of a chunk's heads, in the order of a token's chunks.
enum Kind { kQuery, kKey, kValue };

template <int G, int U, bool NORM>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) heads_kernel(const HeadsArgs a) {
    constexpr int kHeads = 32 / G;  // heads of a chunk
    wait_for_previous_grid();  // see rrf_device.cuh: programmatic dependent launch
    allow_next_grid();
    const int lane = threadIdx.x & 31;
    const int64_t wid = opaque((int64_t)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5));
    const int64_t token = wid / a.warps_per_token;
    if (token >= a.tokens) return;
    const int first = (int)(wid - token * a.warps_per_token);

    const int g = lane & (G - 1);          // place in the head
    const int sub = lane / G;              // head of the chunk
    const bool active = g < a.dim / 16;    // lanes past the head carry zeros
    // the lane's two vectors of the head
    const int rp = a.rot / 16;
    const bool rotated = NORM && g < rp;
    const int va = rotated ? g : rp + g;
    const int vb = rotated ? g + rp : a.dim / 16 + g;

    // the token's slot: where its keys and values go, if anywhere
    int64_t code_at = 0, scale_at = 0;
    bool cached = false;
    if (a.slots != nullptr) {
        const int64_t slot = a.slots[token];
        if (slot >= a.num_slots) {
            if (lane == 0) atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
        } else if (slot >= 0) {
            cached = true;
            const int64_t page = (slot >> 32) == 0 ? (uint32_t)slot / (uint32_t)a.page_size
                                                   : slot / a.page_size;
            const int64_t place = slot - page * a.page_size;
            code_at = page * a.code_page + place * a.code_slot;
            scale_at = page * a.scale_page + place * a.scale_slot;
        }
    }
    // cosines and sines of the lane's 8 pairs
    float cs[8], sn[8];
    if constexpr (NORM) {
        if (a.rot > 0) {
            const int64_t pos = a.positions[token];
            if (pos < 0 || pos >= a.max_positions) {
                if (lane == 0) atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
                return;
            }
            if (rotated) {
                // pairs (i, i + rot / 2): the 8 of vector g; pairs
                // (2i, 2i + 1): the 4 of vector va, then the 4 of vb
                const float* row = a.cos_sin + pos * a.rot;
                const int i0 = a.interleaved ? 4 * va : 8 * g;
                const int i1 = a.interleaved ? 4 * vb : 8 * g + 4;
                const int half = a.rot / 2;
                *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(row + i0);
                *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(row + i1);
                *reinterpret_cast<float4*>(sn) =
                    *reinterpret_cast<const float4*>(row + half + i0);
                *reinterpret_cast<float4*>(sn + 4) =
                    *reinterpret_cast<const float4*>(row + half + i1);
            }
        }
    }

    for (int c0 = first; c0 < a.chunks; c0 += a.warps_per_token * U) {
        uint4 raw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * a.warps_per_token;
            const int kind = c < a.key_chunk ? kQuery : c < a.value_chunk ? kKey : kValue;
            const HeadView& in = kind == kQuery ? a.q : kind == kKey ? a.k : a.v;
            const int head = (c - (kind == kQuery  ? 0
                                   : kind == kKey ? a.key_chunk
                                                  : a.value_chunk)) * kHeads + sub;
            const bool wanted = kind == kQuery || a.slots == nullptr || cached;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (c < a.chunks && active && wanted && head < in.heads &&
                RRF_IN_BOUNDS(head >= 0 && token >= 0 && va >= 0 && vb < a.dim / 8, a.err)) {
                const uint4* p = reinterpret_cast<const uint4*>(
                    in.p + token * in.token_stride + head * in.head_stride);
                raw[u][0] = ld_once_coherent(p + va);
                raw[u][1] = ld_once_coherent(p + vb);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * a.warps_per_token;
            if (c >= a.chunks) break;
            const int kind = c < a.key_chunk ? kQuery : c < a.value_chunk ? kKey : kValue;
            const int heads = kind == kQuery ? a.q.heads : a.k.heads;
            const int head = (c - (kind == kQuery  ? 0
                                   : kind == kKey ? a.key_chunk
                                                  : a.value_chunk)) * kHeads + sub;
            const bool mine = active && head < heads;
            const bool to_cache = kind == kValue || (kind == kKey && a.slots != nullptr);
            if (to_cache && !cached) continue;  // uniform: the token is padding
            float2 x[8];  // pair k of vector va, then of vb
            bf16x8_to_f32x2(raw[u][0], x);
            bf16x8_to_f32x2(raw[u][1], x + 4);
            if (NORM && kind != kValue) {
                float ss = sumsq_bf16x8_x2(x) + sumsq_bf16x8_x2(x + 4);
                ss = head_sum<G>(ss);
                const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, a.inv_dim), a.eps));
                const uint4* gamma = kind == kQuery ? a.q_gamma : a.k_gamma;
                if (active) {
                    float2 w[8];
                    bf16x8_to_f32x2(ld_shared_by_all(gamma + va), w);
                    bf16x8_to_f32x2(ld_shared_by_all(gamma + vb), w + 4);
                    const float2 r2 = make_float2(r, r);
                    const float2 wo = make_float2(a.weight_offset, a.weight_offset);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = __fmul2_rn(__fmul2_rn(x[i], r2), __fadd2_rn(w[i], wo));
                }
                if (rotated) {
                    if (a.interleaved) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 t = x[i];
                            x[i].x = __fmaf_rn(t.x, cs[i], -(t.y * sn[i]));
                            x[i].y = __fmaf_rn(t.y, cs[i], t.x * sn[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 u0 = x[i], u1 = x[i + 4];
                            const float2 cc = make_float2(cs[2 * i], cs[2 * i + 1]);
                            const float2 ns = make_float2(-sn[2 * i], -sn[2 * i + 1]);
                            const float2 ps = make_float2(sn[2 * i], sn[2 * i + 1]);
                            x[i] = __ffma2_rn(u0, cc, __fmul2_rn(u1, ns));
                            x[i + 4] = __ffma2_rn(u1, cc, __fmul2_rn(u0, ps));
                        }
                    }
                }
            }
            if (!to_cache) {
                const HeadView& out = kind == kQuery ? a.q_out : a.k_out;
                if (mine && RRF_IN_BOUNDS(head >= 0 && head < out.heads && vb < a.dim / 8, a.err)) {
                    uint4* p = reinterpret_cast<uint4*>(
                        out.p + token * out.token_stride + head * out.head_stride);
                    p[va] = f32x2_to_bf16x8(x);
                    p[vb] = f32x2_to_bf16x8(x + 4);
                }
            } else {
                float m = 0.0f;  // fmaxf: a NaN does not count
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
                m = head_max<G>(m);
                const bool clamped = m > a.scale_ub;
                m = fmaxf(fminf(m, a.scale_ub), 1e-12f);
                uint2 qa, qb;
                quantise(x, m, clamped, qa, qb);
                if (mine &&
                    RRF_IN_BOUNDS(code_at >= 0 && scale_at >= 0 && head >= 0 &&
                                      code_at + head * a.code_head + a.dim <= a.code_end &&
                                      scale_at + head * a.scale_head < a.scale_end,
                                  a.err)) {
                    const bool key = kind == kKey;
                    uint8_t* codes = (key ? a.k_codes : a.v_codes) + code_at + head * a.code_head;
                    reinterpret_cast<uint2*>(codes)[va] = qa;
                    reinterpret_cast<uint2*>(codes)[vb] = qb;
                    if (g == 0)
                        (key ? a.k_scales : a.v_scales)[scale_at + head * a.scale_head] =
                            __fdiv_rn(m, 448.0f);
                }
            }
        }
    }
}

template <int G, int U, bool NORM>
cudaError_t launch_units(HeadsArgs a, cudaStream_t stream) {
    constexpr int kHeads = 32 / G;
    a.key_chunk = NORM ? (a.q.heads + kHeads - 1) / kHeads : 0;
    a.value_chunk = a.key_chunk + (a.k.heads + kHeads - 1) / kHeads;
    a.chunks = a.value_chunk + (a.slots != nullptr ? (a.k.heads + kHeads - 1) / kHeads : 0);
    a.warps_per_token = (a.chunks + U - 1) / U;
    const int64_t blocks =
        ((int64_t)a.tokens * a.warps_per_token + kWarpsPerBlock - 1) / kWarpsPerBlock;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(32 * kWarpsPerBlock, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, heads_kernel<G, U, NORM>, a);
}

template <int G>
cudaError_t launch_lanes(const HeadsArgs& a, bool norm, cudaStream_t stream) {
    return norm ? launch_units<G, 4, true>(a, stream) : launch_units<G, 4, false>(a, stream);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, bool norm, int sm_count, cudaStream_t stream) {
    const int lanes = (a.dim + 15) / 16;
    if (lanes <= 1) return launch_lanes<1>(a, norm, stream);
    if (lanes <= 2) return launch_lanes<2>(a, norm, stream);
    if (lanes <= 4) return launch_lanes<4>(a, norm, stream);
    if (lanes <= 8) return launch_lanes<8>(a, norm, stream);
    if (lanes <= 16) return launch_lanes<16>(a, norm, stream);
    return launch_lanes<32>(a, norm, stream);
}

}  // namespace rrf
