// rope.cu -- rotary positions around decode attention: the query rows' 64 rotary dims, and new tokens on
// their way into the paged latent cache (with the latent's norm).
//
// Pair i of the 64 dims (i = 0..31; interleaved: dims 2i, 2i + 1, half: dims i, i + 32) at position p is
// turned by the angle p f_i and scaled by the magnitude a:
//   y0 = a (x0 cos(p f_i) - x1 sin(p f_i)),  y1 = a (x0 sin(p f_i) + x1 cos(p f_i)).
// The angle is reduced in integers: turn_i = 2^64 f_i / 2 pi comes from the host, within 1.5 units, and p * turn_i
// modulo 2^64 is the fraction of a full turn in 64-bit fixed point, off by less than |p| 2^-63 turns, whatever the
// position (an fp32 product would be off by radians at position 10^5). Its top 32 bits go to fp32 (an
// error of at most 2^-26 turns), sine and cosine are taken there, and each result is rounded to bf16 once.
#include <cuda_fp8.h>

#include "pair_ptx.cuh"
#include "rope.cuh"

namespace mla {
namespace rp {

constexpr int kRopeDims = kDqk - kDv;      // 64
constexpr int kPairs = kRopeDims / 2;      // one per lane
constexpr int kWarps = 4;                   // per block
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
// 8 rows at a time, both batches' loads issued before the angles are needed. 16,384 tokens of 16 heads (67 MB),
// cold: 14.0 us, 4.8 TB/s; with a plain launch 16.4.
constexpr int kRowsPerWarp = 16;
template <bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) query_kernel(const QueryParams p, const __grid_constant__ mla_rope rope) {
    __shared__ float2 cs[kWarps][kPairs];
    sm100::wait_for_previous_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok = blockIdx.x * kWarps + warp;
    if (tok >= p.tokens) return;
    const int h0 = blockIdx.y * kRowsPerWarp + (lane >> 2), c = lane & 3;
    // interleaved: dims [16c, 16c + 16); half: dims [8c, 8c + 8) and 32 more
    const int d0 = INTERLEAVED ? 16 * c : 8 * c, d1 = INTERLEAVED ? 16 * c + 8 : 8 * c + 32;
    const __nv_bfloat16 *src = p.x + (int64_t)tok * p.ldx;
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
    __nv_bfloat16 *dst = p.y + (int64_t)tok * p.ldy;
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

// The sequence b that packed row i belongs to and cu[b] (the last b with cu[b] <= i; empty sequences are stepped
// over), by a 32-way search of the whole warp; (-1, 0) for a row of no sequence. In a broken `cu` b is
// still a sequence.
__device__ __forceinline__ int2 find_sequence(const int32_t *cu, int batch, int i, int lane) {
    const int end = cu[batch];
    int lo = 0, n = batch, start = 0;  // the answer is in [lo, lo + n); start = cu[lo]
    bool first = true;
    while (n > 1 || first) {
        const int step = (n + 31) >> 5;
        const int at = min(lane * step, n - 1);
        const int c = cu[lo + at];
        const uint32_t below = __ballot_sync(0xffffffffu, c <= i && lane * step < n);
        if (first && !(below & 1u)) return make_int2(-1, 0);  // before the first sequence
        const int k = 31 - __clz(below | 1u);
        start = __shfl_sync(0xffffffffu, c, k);
        lo += k * step;
        n = min(step, n - k * step);
        first = false;
    }
    return i < end && start <= i ? make_int2(lo, start) : make_int2(-1, 0);
}

// The normed latent of a row whose squares leave fp32 (a mean past 2^127, or below 2^-100, where squares lose places
// to fp32's smallest step 2^-149): sum and root in 64 bits, where every bf16 value's square fits. A whole path of its
// own, so that the usual one keeps no registers for it.
template <bool F8>
__device__ __noinline__ void far_latent(const __nv_bfloat16 *x, int64_t ld, const __nv_bfloat16 *weight, float eps,
                                        float inv_scale, uint8_t *dst) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *src = x + (int64_t)(blockIdx.x * kWarps + (threadIdx.x >> 5)) * ld;
    double ss = 0.0;
#pragma unroll 1
    for (int i = lane; i < kDv; i += 32) {
        const double x = __bfloat162float(src[i]);
        ss = fma(x, x, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double rn = 1.0 / sqrt(ss / kDv + eps);
#pragma unroll 1
    for (int i = lane; i < kDv; i += 32) {
        const float y = (float)(__bfloat162float(src[i]) * rn) * __bfloat162float(weight[i]);
        if constexpr (F8)
            dst[i] = (uint8_t)__nv_cvt_float_to_fp8(y * inv_scale, __NV_SATFINITE, __NV_E4M3);
        else
            reinterpret_cast<__nv_bfloat16 *>(dst)[i] = __float2bfloat16_rn(y);
    }
}

// New tokens into the cache: bounded by bytes (1152 in, 1152 or 640 out per token) for prompts, by
// latency for a decode step. One warp per token: a lane holds two 16-byte chunks of the latent and one rotary
// pair; the sum of squares is a warp reduction in fp32, and the row is read and written once.
// The input is dead once read, and a prompt's rows are not read back before much else has been: loads, and the latent
// stores into a bf16 cache, are hinted evict-first (an fp8 cache's are plain). A decode step's rows, which the attention
// reads right behind, take the same path: the hint orders evictions and forces none, and at worst those few rows (147 KB
// for 128 tokens) come from HBM again. 36,800 packed tokens into a bf16 cache, cold: 18.6 us (4.5 TB/s); blocks of 8 and 16
// warps 18.9 and 20.0, without the hints 19.5, with a plain launch 20.5; the registers of 48 instead of 64 warps
// an SM cost 0.6 us (at its 32 registers the kernel spills 16 to 28 bytes a thread: 24 MB of stores and as much of
// loads in L1 over that call), two or four tokens a warp with all loads ahead 4 and 9 (no writes beside the reads).
template <bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, 16) append_kernel(const AppendParams p, const __grid_constant__ mla_rope rope) {
    sm100::wait_for_previous_kernel();
    const int lane = threadIdx.x & 31;
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= p.tokens) return;
    const __nv_bfloat16 *src = p.x + (int64_t)w * p.ld;
    const uint4 *chunks = reinterpret_cast<const uint4 *>(src);
    const uint4 xa = __ldcs(chunks + lane), xb = __ldcs(chunks + 32 + lane);
    // the rotary pair: one word (interleaved); half layout: the values of dims 2 (lane % 16), + 1 of this lane's half,
    // so that the row is read in whole words; the pair's other value comes from lane ^ 16
    const uint32_t two = reinterpret_cast<const uint32_t *>(src + kDv)[lane];
    int b, start;  // sequence, row of its first new token
    if (p.cu_new) {
        const int2 f = find_sequence(p.cu_new, p.batch, w, lane);
        b = f.x;
        start = f.y;
        if (b < 0) return;  // a row of no sequence
    } else {
        b = w / p.n_new;
        start = b * p.n_new;
    }
    const int64_t at = (int64_t)max(p.seqlens[b], 0) + ((int64_t)w - start);  // counts may start far below 0
    const int64_t bi = at / kBlk;
    const int32_t phys = bi < p.bt_stride ? p.block_table[(size_t)b * p.bt_stride + bi] : -1;
    if (phys < 0 || (int64_t)phys >= p.num_blocks) {
        if (lane == 0) raise_error(kErrBounds);
        return;
    }
    const int64_t row = (int64_t)phys * kBlk + at % kBlk;
    const int64_t pos = p.positions ? (int64_t)p.positions[w] : at;
    uint32_t rotated;
    if constexpr (INTERLEAVED) {
        const float2 cs = turn(rope, pos, lane);
        const float r0 = lo_f(two), r1 = hi_f(two);
        rotated = pack_bf16(r0 * cs.x - r1 * cs.y, r0 * cs.y + r1 * cs.x);
    } else {  // lane < 16: dims 2 lane, 2 lane + 1 (first values of these pairs); else their second values
        const uint32_t other = __shfl_xor_sync(0xffffffffu, two, 16);
        const float2 mine = turn(rope, pos, lane);  // pair `lane`; this word's pairs are 2 (lane % 16) and the next
        const int pr = 2 * (lane & 15);
        const float2 c0 = make_float2(__shfl_sync(0xffffffffu, mine.x, pr), __shfl_sync(0xffffffffu, mine.y, pr));
        const float2 c1 = make_float2(__shfl_sync(0xffffffffu, mine.x, pr + 1), __shfl_sync(0xffffffffu, mine.y, pr + 1));
        const float sg = lane < 16 ? -1.f : 1.f;  // y0 = x0 c - x1 s, y1 = x1 c + x0 s
        rotated = pack_bf16(lo_f(two) * c0.x + sg * (lo_f(other) * c0.y), hi_f(two) * c1.x + sg * (hi_f(other) * c1.y));
    }

    uint8_t *dst = p.kv + row * (int64_t)(F8 ? kF8Record : kDqk * 2);
    const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = lo_f(xw[i]);
        v[2 * i + 1] = hi_f(xw[i]);
    }
    if (p.weight) {
        const uint4 wa = reinterpret_cast<const uint4 *>(p.weight)[lane],
                    wb = reinterpret_cast<const uint4 *>(p.weight)[32 + lane];
        const uint32_t ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float ms = ss * (1.f / kDv) + p.eps;
        if (!(ms >= 0x1p-100f && ms <= 0x1p127f)) {  // the same way for all lanes
            reinterpret_cast<uint32_t *>(dst + (F8 ? kDv : kDv * 2))[lane] = rotated;
            far_latent<F8>(p.x, p.ld, p.weight, p.eps, p.inv_scale, dst);
            return;
        }
        const float rn = rsqrtf(ms);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = v[2 * i] * rn * lo_f(ww[i]);
            v[2 * i + 1] = v[2 * i + 1] * rn * hi_f(ww[i]);
        }
    }
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
        reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(o[0], o[1]);
        reinterpret_cast<uint2 *>(dst)[32 + lane] = make_uint2(o[2], o[3]);
    } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        __stcs(reinterpret_cast<uint4 *>(dst) + lane, make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4 *>(dst) + 32 + lane, make_uint4(o[4], o[5], o[6], o[7]));
    }
    reinterpret_cast<uint32_t *>(dst + (F8 ? kDv : kDv * 2))[lane] = rotated;
}

// A programmatic launch: it overlaps the end of the kernel before it, whose results every thread awaits first.
template <class P>
cudaError_t launch(void (*kernel)(P, mla_rope), dim3 grid, const P &p, const mla_rope &rope, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, rope);
}

}  // namespace rp

cudaError_t launch_rope_query(const rp::QueryParams &p, const mla_rope &rope, cudaStream_t stream) {
    const dim3 grid((p.tokens + rp::kWarps - 1) / rp::kWarps, (p.heads + rp::kRowsPerWarp - 1) / rp::kRowsPerWarp);
    return rp::launch(rope.interleaved ? rp::query_kernel<true> : rp::query_kernel<false>, grid, p, rope, stream);
}

cudaError_t launch_append_rope(const rp::AppendParams &p, const mla_rope &rope, bool fp8, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.tokens + rp::kWarps - 1) / rp::kWarps);
    auto kernel = fp8 ? (rope.interleaved ? rp::append_kernel<true, true> : rp::append_kernel<true, false>)
                      : (rope.interleaved ? rp::append_kernel<false, true> : rp::append_kernel<false, false>);
    return rp::launch(kernel, dim3(grid), p, rope, stream);
}

}  // namespace mla
