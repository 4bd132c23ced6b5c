// rope.cu -- rotary positions around decode attention: the query rows' 64 rotary dims, and new tokens on
// their way into the paged latent cache (with the latent's norm).
//
// Pair i of the 64 dims (i = 0..31; interleaved: dims 2i, 2i + 1, half: dims i, i + 32) at position p is
// turned by the angle p f_i and scaled by the magnitude a:
//   y0 = a (x0 cos(p f_i) - x1 sin(p f_i)),  y1 = a (x0 sin(p f_i) + x1 cos(p f_i)).
// The angle is reduced exactly: turn_i = round(2^64 f_i / 2 pi) comes from the host, and p * turn_i modulo
// 2^64 is the fraction of a full turn in 64-bit fixed point, off by at most |p| 2^-65 turns, whatever the
// position (an fp32 product would be off by radians at position 10^5). Its top 32 bits go to fp32 (an
// error of at most 2^-26 turns), sine and cosine are taken there, and each result is rounded to bf16 once.
#include <cuda_fp8.h>

#include "rope.cuh"

namespace mla {
namespace rp {

constexpr int kRopeDims = kDqk - kDv;      // 64
constexpr int kPairs = kRopeDims / 2;      // one per lane
constexpr int kWarps = 8;
constexpr int kF8Record = MLA_FP8_RECORD_BYTES;

// cos and sin (times the magnitude) of pair `lane` at position `pos`
__device__ __forceinline__ float2 turn(const mla_rope &rope, long long pos, int lane) {
    const unsigned long long t = (unsigned long long)pos * rope.turns[lane];
    const float half_turns = (float)(int)(t >> 32) * 0x1p-31f;  // angle / pi, in [-1, 1)
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * rope.magnitude, s * rope.magnitude);
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 two = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&two);
}

// Query rows: bounded by bytes (128 in, 128 out per token and head) for prompts, by latency for a decode
// step. A warp takes up to 16 heads of one token: its lanes compute the token's 32 rotations once and pass
// them through shared memory; four lanes then serve a row (8 pairs and 2 x 16 bytes each), so a warp moves
// 8 rows at a time, both batches' loads issued before the angles are needed.
constexpr int kRowsPerWarp = 16;
template <bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) query_kernel(const QueryParams p, const __grid_constant__ mla_rope rope) {
    __shared__ float2 cs[kWarps][kPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t tok = w / p.chunks;
    if (tok >= p.tokens) return;
    const int h0 = (int)(w % p.chunks) * kRowsPerWarp + (lane >> 2), c = lane & 3;
    // interleaved: dims [16c, 16c + 16); half: dims [8c, 8c + 8) and 32 more
    const int d0 = INTERLEAVED ? 16 * c : 8 * c, d1 = INTERLEAVED ? 16 * c + 8 : 8 * c + 32;
    const __nv_bfloat16 *src = p.x + tok * p.ldx;
    uint4 a[2], b[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int h = h0 + 8 * k;
        if (h < p.heads) {
            a[k] = *reinterpret_cast<const uint4 *>(src + h * p.x_head + d0);
            b[k] = *reinterpret_cast<const uint4 *>(src + h * p.x_head + d1);
        }
    }
    const int64_t pos = p.positions ? p.positions[tok] : (int64_t)max(p.seqlens[tok / p.s_q], 0) + tok % p.s_q;
    cs[warp][lane] = turn(rope, pos, lane);
    __syncwarp();
    float2 r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = cs[warp][8 * c + i];
    __nv_bfloat16 *dst = p.y + tok * p.ldy;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int h = h0 + 8 * k;
        if (h >= p.heads) break;
        uint32_t u[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, v[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (INTERLEAVED) {  // word i of u: pair i; of v: pair 4 + i
                const float u0 = lo_f(u[i]), u1 = hi_f(u[i]), v0 = lo_f(v[i]), v1 = hi_f(v[i]);
                u[i] = pack_bf16(u0 * r[i].x - u1 * r[i].y, u0 * r[i].y + u1 * r[i].x);
                v[i] = pack_bf16(v0 * r[4 + i].x - v1 * r[4 + i].y, v0 * r[4 + i].y + v1 * r[4 + i].x);
            } else {  // word i of u: the first values of pairs 2i, 2i + 1; of v: their second ones
                const float2 r0 = r[2 * i], r1 = r[2 * i + 1];
                const float u0 = lo_f(u[i]), u1 = hi_f(u[i]), v0 = lo_f(v[i]), v1 = hi_f(v[i]);
                u[i] = pack_bf16(u0 * r0.x - v0 * r0.y, u1 * r1.x - v1 * r1.y);
                v[i] = pack_bf16(u0 * r0.y + v0 * r0.x, u1 * r1.y + v1 * r1.x);
            }
        }
        *reinterpret_cast<uint4 *>(dst + h * p.y_head + d0) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4 *>(dst + h * p.y_head + d1) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// The sequence that packed token i belongs to (the last b with cu_new[b] <= i; empty ones are stepped
// over), by a 32-way search of the whole warp.
__device__ __forceinline__ int find_sequence(const int32_t *__restrict__ cu, int batch, int64_t i, int lane) {
    int lo = 0, n = batch;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < n && (int64_t)__ldg(&cu[at]) <= i;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// New tokens into the cache: bounded by bytes (1152 in, 1152 or 640 out per token) for prompts, by
// latency for a decode step. One warp per token: a lane holds 16 latent values (32 bytes) and one rotary
// pair; the sum of squares is a warp reduction in fp32, and the row is read and written once.
template <bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p, const __grid_constant__ mla_rope rope) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= p.tokens) return;
    const __nv_bfloat16 *src = p.x + w * p.ld;
    const uint4 xa = reinterpret_cast<const uint4 *>(src)[2 * lane], xb = reinterpret_cast<const uint4 *>(src)[2 * lane + 1];
    float r0, r1;
    if constexpr (INTERLEAVED) {
        const uint32_t two = reinterpret_cast<const uint32_t *>(src + kDv)[lane];
        r0 = lo_f(two);
        r1 = hi_f(two);
    } else {
        r0 = __bfloat162float(src[kDv + lane]);
        r1 = __bfloat162float(src[kDv + kPairs + lane]);
    }
    int b;
    int64_t t;  // place among the sequence's new tokens
    if (p.cu_new) {
        if (w < __ldg(&p.cu_new[0]) || w >= __ldg(&p.cu_new[p.batch])) return;  // rows of no sequence
        b = find_sequence(p.cu_new, p.batch, w, lane);
        t = w - __ldg(&p.cu_new[b]);
    } else {
        b = (int)(w / p.n_new);
        t = w % p.n_new;
    }
    const int64_t at = (int64_t)max(__ldg(&p.seqlens[b]), 0) + t;
    const int64_t bi = at / kBlk;
    const int32_t phys = at >= 0 && bi < p.bt_stride ? __ldg(&p.block_table[(size_t)b * p.bt_stride + bi]) : -1;
    if (phys < 0 || (int64_t)phys >= p.num_blocks) {
        if (lane == 0) raise_error(kErrBounds);
        return;
    }
    const int64_t row = (int64_t)phys * kBlk + at % kBlk;
    const float2 cs = turn(rope, p.positions ? (int64_t)__ldg(&p.positions[w]) : at, lane);
    const float y0 = r0 * cs.x - r1 * cs.y, y1 = r0 * cs.y + r1 * cs.x;

    const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = lo_f(xw[i]);
        v[2 * i + 1] = hi_f(xw[i]);
    }
    if (p.weight) {
        const uint4 wa = __ldg(reinterpret_cast<const uint4 *>(p.weight) + 2 * lane),
                    wb = __ldg(reinterpret_cast<const uint4 *>(p.weight) + 2 * lane + 1);
        const uint32_t ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rn = rsqrtf(ss * (1.f / kDv) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = v[2 * i] * rn * lo_f(ww[i]);
            v[2 * i + 1] = v[2 * i + 1] * rn * hi_f(ww[i]);
        }
    }
    uint8_t *dst = p.kv + row * (int64_t)(F8 ? kF8Record : kDqk * 2);
    if constexpr (F8) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * p.inv_scale, v[4 * i + 1] * p.inv_scale),
                                                        __NV_SATFINITE, __NV_E4M3);
            const uint32_t c = __nv_cvt_float2_to_fp8x2(
                make_float2(v[4 * i + 2] * p.inv_scale, v[4 * i + 3] * p.inv_scale), __NV_SATFINITE, __NV_E4M3);
            o[i] = a | (c << 16);
        }
        reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        reinterpret_cast<uint4 *>(dst)[2 * lane] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    __nv_bfloat16 *rot = reinterpret_cast<__nv_bfloat16 *>(dst + (F8 ? kDv : kDv * 2));
    if constexpr (INTERLEAVED) {
        reinterpret_cast<uint32_t *>(rot)[lane] = pack_bf16(y0, y1);
    } else {
        rot[lane] = __float2bfloat16(y0);
        rot[kPairs + lane] = __float2bfloat16(y1);
    }
}

}  // namespace rp

cudaError_t launch_rope_query(const rp::QueryParams &q, const mla_rope &rope, cudaStream_t stream) {
    rp::QueryParams p = q;
    p.chunks = (p.heads + rp::kRowsPerWarp - 1) / rp::kRowsPerWarp;
    const int64_t grid = ((int64_t)p.tokens * p.chunks + rp::kWarps - 1) / rp::kWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (rope.interleaved)
        rp::query_kernel<true><<<(unsigned)grid, 32 * rp::kWarps, 0, stream>>>(p, rope);
    else
        rp::query_kernel<false><<<(unsigned)grid, 32 * rp::kWarps, 0, stream>>>(p, rope);
    return cudaGetLastError();
}

cudaError_t launch_append_rope(const rp::AppendParams &p, const mla_rope &rope, bool fp8, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.tokens + rp::kWarps - 1) / rp::kWarps);
    auto kernel = fp8 ? (rope.interleaved ? rp::append_kernel<true, true> : rp::append_kernel<true, false>)
                      : (rope.interleaved ? rp::append_kernel<false, true> : rp::append_kernel<false, false>);
    kernel<<<grid, 32 * rp::kWarps, 0, stream>>>(p, rope);
    return cudaGetLastError();
}

}  // namespace mla
