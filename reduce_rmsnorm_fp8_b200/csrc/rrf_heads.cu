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
// covers head_dim / 16), two 16-byte vectors of 8 values each, and a warp
// takes 32 / G heads of one kind (a chunk) at a time.  The two vectors of a lane are the partners
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

// Measured on B200 (8192 tokens x 72 heads x 128, norm and rotation; 306 MB in
// 51.2 us, 91% of the copy rate).  The first form loaded a warp's chunks into
// registers: 112 of them a thread, 16 warps an SM, 87 us.  Copies into a ring
// of shared memory, which hold no registers, keep 3 chunks of each warp in
// flight: 52 us.
constexpr int kStages = 4;        // (6 stages: 51.2 us, and slower at small heads)
constexpr int kStageVecs = 2 * 32 * kWarpsPerBlock;  // 16-byte vectors of a block's stage
// 5 blocks an SM, 96 registers: 51.4 us; 4 (no spills): 51.8; 6: 56.0.
constexpr int kBlocksPerSm = 5;
// The work of a warp, in chunks of a token (or, writing alone, in tokens of a
// chunk).  Blocks run in rounds of as many as are resident, and a warp's time
// is near its chunks plus a set-up of kSetUp chunks, so the launch takes the
// split of the least rounds * (chunks + kSetUp).  B200, 72 heads of 128:
// 4096 tokens 27.7 us with 9 chunks a warp (3 rounds) against 30.1 with all 18
// (2 rounds), 1536 tokens 12.7 with 6 against 14.1, 8192 tokens 51.4 with 18
// against 51.7 with 9.
constexpr double kSetUp = 2.5;
// Writing alone: 7 blocks an SM.  Compiled for 5 it takes 68 registers, of which
// 7 blocks still fit; compiled for 7 (62 registers) the loads are further from
// their use and 8192 tokens of 8 + 8 heads of 128 take 11.2 us against 10.3.
constexpr int kWriteBlocksPerSm = 7;
constexpr int kWriteBlocksCompiled = 5;

__device__ __forceinline__ void load4(const float* p, float2 v[2]) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = make_float2(f.x, f.y);
    v[1] = make_float2(f.z, f.w);
}

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

__device__ __forceinline__ float fast_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The codes of x[16], a row of largest magnitude `most`, and the row's scale.
// For values that are bf16, x / scale = 448 x / m is often exactly a midpoint
// of the e4m3 grid, and a product with a rounded reciprocal would land on
// either side of it.  So the quotient of n = 448 x (exact then) is corrected
// once by its exact remainder (Markstein's final step, y + (n - y m) / m),
// which makes a representable quotient exact and any other one correct to
// about half an ulp.  Rows above 1e30 are scaled by 2^-64 first, so that n
// stays finite.  Values beyond a bound (scale_ub) saturate; only where they are
// 1e30 times the bound or infinite, and y might not be finite, is the row left
// uncorrected (an infinite y would make its remainder a NaN).
// (Cutting x to the bound instead costs every row some 20 instructions.)
__device__ __forceinline__ float quantise(const float2 x[8], float most, float scale_ub, uint2& qa,
                                          uint2& qb) {
    const float m = fmaxf(fminf(most, scale_ub), 1e-12f);
    const float down = most > 1e30f ? 5.421010862427522e-20f : 1.0f;  // 2^-64
    const float d = m * down, f = 448.0f * down, inv = fast_reciprocal(d);
    const float2 k2 = make_float2(f * inv, f * inv);
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(x[i], k2);
    // (an infinite scale: finite values are 0, infinities NaN.  For m above
    // 3.4e8 m * 1e30 is infinite, and y at most 448 * 3.4e38 / m.)
    if (most <= m * 1e30f && most < __int_as_float(0x7F800000)) {
        const float2 minus_d = make_float2(-d, -d), f2 = make_float2(f, f);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = __ffma2_rn(__ffma2_rn(y[i], minus_d, __fmul2_rn(x[i], f2)), inv2, y[i]);
    }
    qa = f32x2_to_e4m3x8(y);
    qb = f32x2_to_e4m3x8(y + 4);
    // m / 448, with the same correction
    const float s = m * (1.0f / 448.0f);
    return s < __int_as_float(0x7F800000)
               ? __fmaf_rn(__fmaf_rn(s, -448.0f, m), 1.0f / 448.0f, s)
               : s;
}

// The largest magnitude of 16 bf16 (like fmaxf, it passes over a NaN).
__device__ __forceinline__ float max_bf16x16(const uint4 u, const uint4 v) {
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i)  // (magnitudes; the sign is of no use)
        asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    // (0 where all are NaN)
    return fmaxf(0.0f, fmaxf(fabsf(__uint_as_float(m << 16)),
                             fabsf(__uint_as_float(m & 0xFFFF0000u))));
}

// n / d for n >= 0, d > 0, in 32 bits where they do.
__device__ __forceinline__ int64_t divide(int64_t n, int d) {
    return (n >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}

// What a lane keeps of its token, and its place in a head.
struct Lane {
    int64_t token;
    int g, sub;          // lane of the head, head of the chunk
    int va, vb;          // its two vectors
    bool active;         // it holds a part of the head (else zeros)
    bool rotated;
    bool cached;         // the token has a slot
    int64_t code_at, scale_at;  // where that begins
    const float* turn;          // the token's row of cos_sin
};

enum Kind { kQuery, kKey, kValue };

// The lane's weights of the norm, w = gamma + weight_offset, and of the
// rotation, multiplied into it once for all the heads of a kind:
//   out_a = a (w_a cos) + b (-w_b sin),  out_b = b (w_b cos) + a (w_a sin)
// for the partners a, b.  Pairs (i, i + rot / 2): a in vector va, b in vb, 8
// angles (those of vector g).  Pairs (2i, 2i + 1): both in one vector, 4
// angles for va, then 4 for vb.  Lanes that are not rotated have w in aa, bb.
struct Turn {
    float2 aa[4], ab[4], bb[4], ba[4];
};

__device__ __forceinline__ void load_turn(const HeadsArgs& a, const Lane& l, const uint4* gamma,
                                          Turn& t) {
    float2 wa[4], wb[4];
    const uint4 z = make_uint4(0, 0, 0, 0);
    bf16x8_to_f32x2(l.active ? ld_shared_by_all(gamma + l.va) : z, wa);
    bf16x8_to_f32x2(l.active ? ld_shared_by_all(gamma + l.vb) : z, wb);
    const float2 wo = make_float2(a.weight_offset, a.weight_offset);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t.aa[i] = wa[i] = __fadd2_rn(wa[i], wo);
        t.bb[i] = wb[i] = __fadd2_rn(wb[i], wo);
        t.ab[i] = t.ba[i] = make_float2(0.0f, 0.0f);
    }
    if (!l.rotated) return;
    float2 c[4], s[4];
    const float* i0 = l.turn + (a.interleaved ? 4 * l.va : 8 * l.g);
    const float* i1 = l.turn + (a.interleaved ? 4 * l.vb : 8 * l.g + 4);
    const int half = a.rot / 2;
    load4(i0, c);
    load4(i1, c + 2);
    load4(i0 + half, s);
    load4(i1 + half, s + 2);
    if (a.interleaved) {
        // pair k of vector va: (wa[k].x, wa[k].y) with angle k; of vb: 4 + k
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float ca = i % 2 ? c[i / 2].y : c[i / 2].x;
            const float sa = i % 2 ? s[i / 2].y : s[i / 2].x;
            const float cb = i % 2 ? c[2 + i / 2].y : c[2 + i / 2].x;
            const float sb = i % 2 ? s[2 + i / 2].y : s[2 + i / 2].x;
            t.aa[i] = make_float2(wa[i].x * ca, wa[i].y * ca);
            t.ab[i] = make_float2(-(wa[i].y * sa), wa[i].x * sa);
            t.bb[i] = make_float2(wb[i].x * cb, wb[i].y * cb);
            t.ba[i] = make_float2(-(wb[i].y * sb), wb[i].x * sb);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.aa[i] = __fmul2_rn(wa[i], c[i]);
            t.ab[i] = __fmul2_rn(wb[i], make_float2(-s[i].x, -s[i].y));
            t.bb[i] = __fmul2_rn(wb[i], c[i]);
            t.ba[i] = __fmul2_rn(wa[i], s[i]);
        }
    }
}

// Norm and rotation of the lane's values (pair k of vector va, then of vb).
template <int G>
__device__ __forceinline__ void norm_turn(const HeadsArgs& a, const Lane& l, const Turn& t,
                                          float2 x[8]) {
    float2 s0 = __fmul2_rn(x[0], x[0]), s1 = __fmul2_rn(x[1], x[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s0 = __ffma2_rn(x[i], x[i], s0);
        s1 = __ffma2_rn(x[i + 1], x[i + 1], s1);
    }
    s0 = __fadd2_rn(s0, s1);
    const float ss = head_sum<G>(s0.x + s0.y);
    const float r = rsqrtf(__fmaf_rn(ss, a.inv_dim, a.eps));
    const float2 r2 = make_float2(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], r2);
    if (!l.rotated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __fmul2_rn(x[i], t.aa[i]);
            x[i + 4] = __fmul2_rn(x[i + 4], t.bb[i]);
        }
    } else if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = x[i], v = x[i + 4];
            x[i].x = __fmaf_rn(u.x, t.aa[i].x, u.y * t.ab[i].x);
            x[i].y = __fmaf_rn(u.y, t.aa[i].y, u.x * t.ab[i].y);
            x[i + 4].x = __fmaf_rn(v.x, t.bb[i].x, v.y * t.ba[i].x);
            x[i + 4].y = __fmaf_rn(v.y, t.bb[i].y, v.x * t.ba[i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = x[i], v = x[i + 4];
            x[i] = __ffma2_rn(u, t.aa[i], __fmul2_rn(v, t.ab[i]));
            x[i + 4] = __ffma2_rn(v, t.bb[i], __fmul2_rn(u, t.ba[i]));
        }
    }
}

// 16 bytes from global to shared memory, asynchronously; zeros unless `wanted`.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool wanted) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(wanted ? 16 : 0)
                 : "memory");
}

// The copies of a warp's chunks, kStages - 1 ahead of its work.  A lane reads
// only what it has copied itself, so its own wait is all the ring needs.
template <int G>
struct Feed {
    uint32_t ring;          // the lane's 32 bytes of stage 0
    const uint16_t* src;    // its vector va of the next chunk
    int64_t step;
    int head, heads;        // the next chunk's head, and where they end
    int left;               // chunks left of this kind
    int stage;

    __device__ __forceinline__ void begin(const HeadsArgs& a, const Lane& l, const HeadView& in,
                                          int chunk, int n) {
        constexpr int kHeads = 32 / G;
        head = l.active ? chunk * kHeads + l.sub : INT32_MAX / 2;
        heads = in.heads;
        src = in.p + l.token * in.token_stride + (chunk * kHeads + l.sub) * in.head_stride +
              8 * l.va;
        step = kHeads * in.head_stride;
        left = n;
    }
};

// Issue the copies of the next chunk of [.., hi), or of nothing behind it.
template <int G>
__device__ __forceinline__ void feed_next(const HeadsArgs& a, const Lane& l, Feed<G>& f, int& next,
                                          int hi) {
    if (next < hi) {
        if (f.left == 0) {
            if (next < a.value_chunk)
                f.begin(a, l, a.k, next - a.key_chunk, a.value_chunk - next);
            else
                f.begin(a, l, a.v, next - a.value_chunk, a.chunks - next);
        }
        const bool wanted = f.head < f.heads &&
                            RRF_IN_BOUNDS(8 * l.vb + 8 <= a.dim && l.token < a.tokens, a.err);
        const uint16_t* p = wanted ? f.src : a.k.p;  // (nothing is read)
        copy16(f.ring + f.stage * (kStageVecs * 16), p, wanted);
        copy16(f.ring + f.stage * (kStageVecs * 16) + kStageVecs * 8,
               p + (wanted ? 8 * (l.vb - l.va) : 0), wanted);
        f.src += f.step;
        f.head += 32 / G;
        --f.left;
        ++next;
        f.stage = (f.stage + 1) % kStages;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// (the bounds-checking build) Eight codes at `codes` and `second` further on,
// and a scale, lie in the keys' or the values' arrays.
[[maybe_unused]] __device__ __forceinline__ bool in_cache(const HeadsArgs& a,
                                                          const uint8_t* codes, int second,
                                                          const float* scale) {
    const auto inside = [&](const uint8_t* c, const float* s) {
        return codes >= c && codes + second + 8 <= c + a.code_end && scale >= s &&
               scale < s + a.scale_end;
    };
    return inside(a.k_codes, a.k_scales) || inside(a.v_codes, a.v_scales);
}

// A head's codes and scale into the cache: x and the largest magnitude of the
// lane; the lane's codes go to `codes` and `second` further on.
template <int G>
__device__ __forceinline__ void store_codes(const HeadsArgs& a, const float2 x[8], float m,
                                            bool store, bool first_lane, uint8_t* codes,
                                            int second, float* scale_out) {
    uint2 qa, qb;
    const float scale = quantise(x, head_max<G>(m), a.scale_ub, qa, qb);
    if (store && RRF_IN_BOUNDS(in_cache(a, codes, second, scale_out), a.err)) {
        *reinterpret_cast<uint2*>(codes) = qa;
        *reinterpret_cast<uint2*>(codes + second) = qb;
        if (first_lane) *scale_out = scale;
    }
}

// The warp's chunks of one kind, from the token's chunk `c` to `end`.
template <int G, Kind KIND>
__device__ __forceinline__ void work_chunks(const HeadsArgs& a, const Lane& l, const uint4* ring,
                                            Feed<G>& f, int& next, int& stage, int c, int end,
                                            int from, int hi) {
    constexpr int kHeads = 32 / G;  // heads of a chunk
    if (c >= end) return;
    const bool to_cache = KIND == kValue || (KIND == kKey && a.slots != nullptr);
    const int first = (c - from) * kHeads + l.sub;
    const int heads = KIND == kQuery ? a.q.heads : a.k.heads;
    int left = l.active ? heads - first : 0;  // heads from the lane's first on
    const int da = 8 * l.va, db = 8 * l.vb;
    Turn turn;
    if constexpr (KIND != kValue) load_turn(a, l, KIND == kQuery ? a.q_gamma : a.k_gamma, turn);
    // the output, as bf16 or as codes and scales
    const HeadView& out = KIND == kQuery ? a.q_out : a.k_out;
    uint16_t* dst = out.p + l.token * out.token_stride + first * out.head_stride;
    uint8_t* codes = (KIND == kKey ? a.k_codes : a.v_codes) + l.code_at + first * a.code_head + da;
    float* scales = (KIND == kKey ? a.k_scales : a.v_scales) + l.scale_at + first * a.scale_head;

#pragma unroll 1
    for (; c < end; ++c, left -= kHeads) {
        asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
        const uint4 ra = ring[stage * kStageVecs];
        const uint4 rb = ring[stage * kStageVecs + kStageVecs / 2];
        float2 x[8];
        bf16x8_to_f32x2(ra, x);
        bf16x8_to_f32x2(rb, x + 4);
        stage = (stage + 1) % kStages;
        feed_next<G>(a, l, f, next, hi);
        if constexpr (KIND != kValue) norm_turn<G>(a, l, turn, x);
        if (!to_cache) {
            if (left > 0 && RRF_IN_BOUNDS(heads - left < out.heads && left <= heads, a.err)) {
                *reinterpret_cast<uint4*>(dst + da) = f32x2_to_bf16x8(x);
                *reinterpret_cast<uint4*>(dst + db) = f32x2_to_bf16x8(x + 4);
            }
            dst += kHeads * out.head_stride;
        } else if (l.cached) {  // uniform in the warp
            float m = 0.0f;  // fmaxf: a NaN does not count
            if constexpr (KIND == kValue) {
                m = max_bf16x16(ra, rb);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
            }
            store_codes<G>(a, x, m, left > 0, l.g == 0, codes, db - da, scales);
            codes += kHeads * a.code_head;
            scales += kHeads * a.scale_head;
        }
    }
}

// The place of a token in the cache; false for padding (and, with the error
// bit, for a slot behind the cache).
__device__ __forceinline__ bool place_of(const HeadsArgs& a, int64_t slot, int64_t& code_at,
                                         int64_t& scale_at) {
    code_at = scale_at = 0;
    if (slot < 0) return false;
    if (slot >= a.num_slots) {
        atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
        return false;
    }
    const int64_t page = divide(slot, a.page_size);
    const int64_t place = slot - page * a.page_size;
    code_at = page * a.code_page + place * a.code_slot;
    scale_at = page * a.scale_page + place * a.scale_slot;
    return true;
}

template <int G>
__device__ __forceinline__ void place_lane(const HeadsArgs& a, Lane& l) {
    const int lane = threadIdx.x & 31;
    l.g = lane & (G - 1);
    l.sub = lane / G;
    l.active = l.g < a.dim / 16;
    const int rp = a.rot / 16;
    l.rotated = l.g < rp;
    l.va = l.rotated ? l.g : rp + l.g;
    l.vb = l.rotated ? l.g + rp : a.dim / 16 + l.g;
}

// Queries and keys normalised and rotated; with slots, keys and values into
// the cache.  A warp takes `per` chunks of one token: the fewer warps share a
// token, the fewer repeat its set-up (its position, angles and weights), the
// more there are, the more bytes are in flight.
template <int G>
__global__ void __launch_bounds__(32 * kWarpsPerBlock, kBlocksPerSm) heads_kernel(const HeadsArgs a) {
    __shared__ uint4 rings[kStages * kStageVecs];  // [stage][half][thread]
    wait_for_previous_grid();  // see rrf_device.cuh: programmatic dependent launch
    allow_next_grid();
    Lane l;
    l.token = opaque((int)blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5);
    if (l.token >= a.tokens) return;
    // the token's slot and position, on their way while the lane sets itself up
    const int64_t slot = a.slots != nullptr ? a.slots[l.token] : -1;
    const int64_t pos = a.rot > 0 ? a.positions[l.token] : 0;
    place_lane<G>(a, l);
    const int lo = blockIdx.y * a.per;
    const int hi = lo + a.per < a.chunks ? lo + a.per : a.chunks;

    // the first copies, before anything waits for the token's place
    const uint4* ring = rings + threadIdx.x;
    Feed<G> feed;
    feed.ring = smem_u32(ring);
    feed.stage = 0;
    feed.left = 0;
    if (lo < a.key_chunk) feed.begin(a, l, a.q, lo, a.key_chunk - lo);
    int next = lo, stage = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) feed_next<G>(a, l, feed, next, hi);

    const bool valid = a.rot == 0 || (pos >= 0 && pos < a.max_positions);
    if (!valid) atomicOr(a.err, RRF_DEVICE_ERROR_INDEX);
    l.turn = a.cos_sin + (valid ? pos : 0) * a.rot;
    l.cached = place_of(a, slot, l.code_at, l.scale_at);
    if (valid) {
        const int k0 = lo > a.key_chunk ? lo : a.key_chunk;
        const int v0 = lo > a.value_chunk ? lo : a.value_chunk;
        work_chunks<G, kQuery>(a, l, ring, feed, next, stage, lo,
                               hi < a.key_chunk ? hi : a.key_chunk, 0, hi);
        work_chunks<G, kKey>(a, l, ring, feed, next, stage, k0,
                             hi < a.value_chunk ? hi : a.value_chunk, a.key_chunk, hi);
        work_chunks<G, kValue>(a, l, ring, feed, next, stage, v0, hi, a.value_chunk, hi);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Keys and values as they are into the cache.  Nothing but its place belongs
// to a token, so a warp keeps to one chunk (4 heads of 128, of the keys or of
// the values) and takes `per` tokens: lane t works out the place of the
// warp's token t, once for all.  (B200, 32768 tokens x 8 heads x 128: 36 us,
// 89% of the copy rate; a warp for all the chunks of one token, which spends
// a third of its instructions on the token's set-up, took 49 us.)
template <int G>
__global__ void __launch_bounds__(32 * kWarpsPerBlock, kWriteBlocksCompiled)
    write_kernel(const HeadsArgs a) {
    constexpr int kHeads = 32 / G;
    __shared__ uint4 rings[kStages * kStageVecs];  // [stage][half][thread]
    __shared__ longlong2 places[kWarpsPerBlock][32];
    wait_for_previous_grid();
    allow_next_grid();
    Lane l;
    place_lane<G>(a, l);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)(opaque((int)blockIdx.x) * kWarpsPerBlock + warp) * a.per;
    if (t0 >= a.tokens) return;
    const int n = a.tokens - t0 < a.per ? (int)(a.tokens - t0) : a.per;
    const bool key = (int)blockIdx.y < a.value_chunk;
    const int head = ((int)blockIdx.y - (key ? 0 : a.value_chunk)) * kHeads + l.sub;
    const HeadView& in = key ? a.k : a.v;
    const bool mine = l.active && head < in.heads;
    const int da = 8 * l.va, db = 8 * l.vb;
    const uint16_t* src = in.p + t0 * in.token_stride + head * in.head_stride + da;
    if (!mine) src = in.p;

    const uint4* ring = rings + threadIdx.x;
    const uint32_t ring_at = smem_u32(ring);
    int fed = 0;
    auto feed = [&]() {
        if (fed < n) {
            const bool wanted = mine && RRF_IN_BOUNDS(db + 8 <= a.dim && t0 + fed < a.tokens, a.err);
            const uint32_t at = ring_at + (fed % kStages) * (kStageVecs * 16);
            copy16(at, src, wanted);
            copy16(at + kStageVecs * 8, src + (wanted ? db - da : 0), wanted);
            if (mine) src += in.token_stride;
            ++fed;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) feed();
    if (lane < n) {
        longlong2 p;
        int64_t code_at, scale_at;
        const bool cached = place_of(a, a.slots[t0 + lane], code_at, scale_at);
        p.x = cached ? code_at : -1;
        p.y = scale_at;
        places[warp][lane] = p;
    }
    __syncwarp();
    // (of a chunk's last heads, some may not be there: their lanes store nothing)
    uint8_t* codes = (key ? a.k_codes : a.v_codes) + head * a.code_head + da;
    float* scales = (key ? a.k_scales : a.v_scales) + head * a.scale_head;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
        const uint4 ra = ring[(t % kStages) * kStageVecs];
        const uint4 rb = ring[(t % kStages) * kStageVecs + kStageVecs / 2];
        const longlong2 place = places[warp][t];
        float2 x[8];
        bf16x8_to_f32x2(ra, x);
        bf16x8_to_f32x2(rb, x + 4);
        feed();
        if (place.x < 0) continue;  // uniform in the warp
        store_codes<G>(a, x, max_bf16x16(ra, rb), mine, l.g == 0, codes + place.x, db - da,
                       scales + place.y);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class Kernel>
cudaError_t launch(Kernel kernel, const HeadsArgs& a, int64_t x, int64_t y, cudaStream_t stream) {
    if (x > INT32_MAX || y > 65535) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)y, 1);
    cfg.blockDim = dim3(32 * kWarpsPerBlock, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int G>
cudaError_t launch_lanes(HeadsArgs a, bool norm, int sm_count, cudaStream_t stream) {
    constexpr int kHeads = 32 / G;
    const int kv_chunks = (a.k.heads + kHeads - 1) / kHeads;
    a.key_chunk = norm ? (a.q.heads + kHeads - 1) / kHeads : 0;
    a.value_chunk = a.key_chunk + kv_chunks;
    a.chunks = a.value_chunk + (a.slots != nullptr ? kv_chunks : 0);
    // blocks for `per` units of work to a warp, and the best `per` up to `most`
    const auto blocks_of = [&](int per) {
        const int64_t warps = norm ? a.tokens : ((int64_t)a.tokens + per - 1) / per;
        const int64_t y = norm ? (a.chunks + per - 1) / per : a.chunks;
        return (warps + kWarpsPerBlock - 1) / kWarpsPerBlock * y;
    };
    const int64_t resident = (int64_t)sm_count * (norm ? kBlocksPerSm : kWriteBlocksPerSm);
    const int most = norm ? a.chunks : 32;  // (a write warp's lanes hold its places)
    double least = 0.0;
    // (one round even with one unit to a warp: no split is cheaper)
    for (int units = blocks_of(1) <= resident ? 1 : most, parts = 1; units >= 1; ++parts) {
        const int64_t rounds = (blocks_of(units) + resident - 1) / resident;
        const double cost = (double)rounds * (units + kSetUp);
        if (least == 0.0 || cost < least) {
            least = cost;
            a.per = units;
        }
        if (units == 1) break;
        while ((most + parts - 1) / parts >= units) ++parts;  // the next smaller split
        units = (most + parts - 1) / parts;
    }
    const int64_t y = norm ? (a.chunks + a.per - 1) / a.per : a.chunks;
    const int64_t x = blocks_of(a.per) / y;
    return norm ? launch(heads_kernel<G>, a, x, y, stream) : launch(write_kernel<G>, a, x, y, stream);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, bool norm, int sm_count, cudaStream_t stream) {
    const int lanes = (a.dim + 15) / 16;
    if (lanes <= 1) return launch_lanes<1>(a, norm, sm_count, stream);
    if (lanes <= 2) return launch_lanes<2>(a, norm, sm_count, stream);
    if (lanes <= 4) return launch_lanes<4>(a, norm, sm_count, stream);
    if (lanes <= 8) return launch_lanes<8>(a, norm, sm_count, stream);
    if (lanes <= 16) return launch_lanes<16>(a, norm, sm_count, stream);
    return launch_lanes<32>(a, norm, sm_count, stream);
}

}  // namespace rrf
