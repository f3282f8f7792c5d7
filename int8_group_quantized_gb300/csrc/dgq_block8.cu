// dgq_block8.cu -- a paged cache in 8 bits with one scale per block and KV head: rows stored by slot, and
// rows read back in bf16 (sm_103a).  Its decode attention: dgq_attn_kernel.cuh.
//
// Block of one head: s = the smallest bf16 number not below amax / top (top = 127 for INT8, 448 for E4M3;
// amax the largest |x| of the block's tokens; s = 0 where amax < 2^-80), and every x is stored as x / s
// rounded to the nearest whole number (the byte 128 + it) or E4M3 number, ties to even.  A token that
// joins a block takes part in amax; where s grows, the codes that are there are made anew from the
// values that they stand for.
//
// Why s has 8 significant bits.  x has 8 as well, so x / s = (a / b) 2^j with whole a, b < 256, and its
// distance from the middle m of two codes is a whole multiple of 1 / (2 b) (INT8) unless it is 0: a
// quotient is a tie, exactly, or at least 2^-9 away from one (E4M3: a relative 2^-13).  So the codes do
// not depend on how x / s is computed.  Here it is x times the rounded 1 / s (off by 2^-17 at most below
// 128), rounded to a grid that has every middle on it and is finer than that distance: for INT8 one fused
// product-sum onto multiples of 2^-10, for E4M3 to 16 significant bits; the second rounding, to the code,
// is then that of the exact quotient.  s rounded up costs at most 2^-7 of the step, and keeps |x / s| <= top.
//
// Bound by HBM: a token's row of a head is 256 bytes read and 128 written by the store, the other way
// round by the load.  Work of the store: a run of tokens that lie one behind the other in a block, for one
// head of K or V: a warp for 16 of the block's rows, 16 bytes a lane, its rows in registers (8 loads in
// flight), so that values are read once for amax and codes.  The four warps of a block of threads take
// four blocks of 16 tokens, or share one of 64.  Runs are found on the fly: a block of threads looks at a
// window of slots, from one token (decode steps: more blocks of threads than SMs) to 128.
// Load: a warp for 16 tokens of one head of K or V, 2 KB of codes.
// Measured, us in a graph: four chunks of 2048 tokens into blocks of 64, 8 heads (50 MB): E4M3 15.0, INT8
// 14.4 (floor 7.4; blocks of 16: 13.0), 16.3 with K and V in one item at four blocks of threads per SM; it is two waves of
// three dependent loads (slots, scale and rows, codes).  Seven blocks of threads per SM spill 12 (INT8) and 20
// bytes a thread, six spill none: 16.1 and 15.3.  The look at the 64 slots in front of a run is 0.3 to 0.5 of it.
// 44240 tokens loaded (272 MB, two thirds of it written): 45.1, 6.0 TB/s; 49.4 from a grid of eight blocks of
// threads per SM that walk the list.
#include "dgq_device.cuh"
#include "dgq.h"
#include "dgq_launch.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace dgq {

constexpr int kB8Threads = 128, kB8Warps = kB8Threads / 32;
constexpr int kB8Window = 128;         // slots that a block of threads looks at, at most
constexpr int kB8Back = 64;            // slots in front of a run among which its block is looked for
constexpr int kB8Rows = 16;            // rows of a warp
constexpr int kB8Vecs = kB8Rows / 2;   // a lane's 16-byte vectors of one tensor: two rows per instruction
constexpr float kB8Least = 0x1p-80f;   // a block below this is stored as zeros
constexpr uint32_t kB8Most = 227u << 23;  // values of 2^100 and more (these bits of an fp32 number) are flagged

struct Block8Args {
    const uint4 *k, *v;          // rows [T][Hkv][16 vectors], tokens k_stride / v_stride vectors apart
    int64_t k_stride, v_stride;
    const int32_t *slots;
    uint8_t *kpool, *vpool;
    float *kscale, *vscale;
    WsHeader *hdr;
    int32_t T, Hkv, bs, num_blocks, window;
};

template <bool E4>
__device__ __forceinline__ float b8_top() { return E4 ? 448.0f : 127.0f; }

// The smallest bf16 number not below amax / top; NaN of what is infinite or NaN.
template <bool E4>
__device__ __forceinline__ float b8_scale(float amax)
{
    if (amax < kB8Least) return 0.0f;
    if (!(amax < INFINITY)) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((__float_as_uint(__fdiv_rn(amax, b8_top<E4>())) + 0xFFFFu) & 0xFFFF0000u);
}

// Four E4M3 codes, and the values of four.  (The halves are named in PTX: the header's functions pack and unpack
// them around each conversion.)
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3)
{
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return w;
}

__device__ __forceinline__ float4 e4m3x4_values(uint32_t w)
{
    uint32_t a, b;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_float4(x.x, x.y, y.x, y.y);
}

// Four codes of the values x (inv = the rounded 1 / s, or 0 where s is 0).
template <bool E4>
__device__ __forceinline__ uint32_t b8_encode4(float x0, float x1, float x2, float x3, float inv)
{
    if constexpr (E4) {
        // to 16 significant bits (a carry into the exponent is right), then to E4M3
        auto snap = [&](float x) { return __uint_as_float((__float_as_uint(x * inv) + 0x80u) & ~0xFFu); };
        return e4m3x4(snap(x0), snap(x1), snap(x2), snap(x3));
    } else {
        // 12288 + y in fp32 is y to multiples of 2^-10; 1.5 2^23 + 128 + that is the whole number, ties to
        // even, in the low bits
        auto code = [&](float x) {
            const float y = __fmaf_rn(x, inv, 12288.0f);
            return __float_as_uint(__fadd_rn(y, 12582912.0f + 128.0f - 12288.0f));
        };
        return __byte_perm(__byte_perm(code(x0), code(x1), 0x0040), __byte_perm(code(x2), code(x3), 0x0040), 0x5410);
    }
}

// The values of four codes in units of the scale.
template <bool E4>
__device__ __forceinline__ float4 b8_decode4(uint32_t w)
{
    if constexpr (E4) {
        return e4m3x4_values(w);
    } else {
        // 2^23 + code as fp32
        auto value = [&](uint32_t sel) { return __uint_as_float(__byte_perm(w, 0x4B000000u, sel)) - 8388736.0f; };
        return make_float4(value(0x7440), value(0x7441), value(0x7442), value(0x7443));
    }
}

__device__ __forceinline__ __nv_bfloat162 b8_absmax(__nv_bfloat162 m, uint32_t w)
{
    return __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
}

// Largest |x| over the warp of a lane's vectors (rows that are not the run's hold zeros), as the bits of
// an fp32 number.
__device__ __forceinline__ uint32_t b8_amax(const uint4 *x)
{
    __nv_bfloat162 m = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kB8Vecs; ++i) {
        m = b8_absmax(m, x[i].x);
        m = b8_absmax(m, x[i].y);
        m = b8_absmax(m, x[i].z);
        m = b8_absmax(m, x[i].w);
    }
    // (as bits: in the order of the numbers they stand for, a NaN above all)
    return __reduce_max_sync(0xffffffffu, max(__float_as_uint(__low2float(m)), __float_as_uint(__high2float(m))));
}

template <bool E4>
__global__ void __launch_bounds__(kB8Threads, 7) store_block8_kernel(const Block8Args a)
{
    __shared__ int32_t s_start[kB8Window];            // tokens of the window that start a run
    __shared__ int32_t s_count[kB8Warps];
    __shared__ uint32_t s_max[2][kB8Warps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t bs = a.bs, shift = __ffs(bs) - 1;
    const int32_t w0 = blockIdx.x * a.window;
    // ---- runs that start in the window: a token with a place, not behind its predecessor in one block
    {
        const int32_t t = w0 + tid;
        bool start = false;
        if (tid < a.window && t < a.T) {
            const int32_t slot = __ldg(a.slots + t);
            if (slot != -1) {
                if ((uint32_t)slot >= (uint32_t)(a.num_blocks * bs)) record_error(a.hdr, kErrBadBlock);  // skipped
                else start = t == 0 || (slot & (bs - 1)) == 0 || __ldg(a.slots + t - 1) != slot - 1;
            }
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, start);
        if (lane == 0) s_count[warp] = __popc(hit);
        __syncthreads();
        int32_t at = 0;
        for (int w = 0; w < warp; ++w) at += s_count[w];
        if (start) s_start[at + __popc(hit & ((1u << lane) - 1u))] = t;
        __syncthreads();
    }
    int32_t runs = 0;
#pragma unroll
    for (int w = 0; w < kB8Warps; ++w) runs += s_count[w];

    const int per = bs / kB8Rows;                     // warps of an item: 1, 2 or 4
    const int group = warp / per, part = warp % per, groups = kB8Warps / per;
    const int32_t items = runs * 2 * a.Hkv;           // (run, K or V, head)
    const int32_t y0 = blockIdx.y * groups, step = gridDim.y * groups;
    int flip = 0;
    for (int32_t base = y0; base < items; base += step, flip ^= 1) {  // (the same turns for all warps: barriers inside)
        const int32_t item = base + group;
        const bool live = item < items;
        int32_t f0 = -1, f1 = -1;
        int32_t t0 = 0, h = 0, blk = 0, r0 = 0, n = 0;
        bool is_v = false;
        if (live) {
            const int32_t q = item / a.Hkv;
            h = item - q * a.Hkv;
            is_v = q & 1;
            t0 = s_start[q >> 1];
            const int32_t slot = __ldg(a.slots + t0);
            blk = slot >> shift;
            r0 = slot & (bs - 1);
            // the run: up to the block's end, as long as the slots go up by one
            const int32_t most = min(bs - r0, a.T - t0);
            const bool a0 = lane < most && __ldg(a.slots + t0 + lane) == slot + lane;
            const bool a1 = lane + 32 < most && __ldg(a.slots + t0 + lane + 32) == slot + lane + 32;
            const uint32_t m0 = __ballot_sync(0xffffffffu, a0), m1 = __ballot_sync(0xffffffffu, a1);
            n = m0 == 0xffffffffu ? 32 + (m1 == 0xffffffffu ? 32 : __ffs(~m1) - 1) : __ffs(~m0) - 1;
            // slots in front of it (looked at when the rows are on their way)
            static_assert(kB8Back == 2 * 32, "two slots a lane");
            if (lane < t0) f0 = __ldg(a.slots + t0 - 1 - lane);
            if (lane + 32 < t0) f1 = __ldg(a.slots + t0 - 33 - lane);
        }
        // this lane: rows 2i + lane / 16 of the warp's 16, 16-byte vector lane % 16
        const int32_t row0 = part * kB8Rows + (lane >> 4), vec = lane & 15;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        const uint4 *from = (is_v ? a.v : a.k) + (int64_t)(t0 - r0 + row0) * stride + h * 16 + vec;
        float *scale = (is_v ? a.vscale : a.kscale) + (int64_t)blk * a.Hkv + h;
        uint4 x[kB8Vecs];
#pragma unroll
        for (int i = 0; i < kB8Vecs; ++i) {
            const int32_t r = row0 + 2 * i - r0;
            x[i] = r >= 0 && r < n ? __ldcs(from + 2 * i * stride) : make_uint4(0u, 0u, 0u, 0u);
        }
        const float had = live && r0 > 0 ? __ldcg(scale) : 0.0f;  // tokens are there already
        uint32_t amax = b8_amax(x);
        if (per > 1) {  // the warps of the item
            if (lane == 0) s_max[flip][warp] = amax;
            __syncthreads();  // (also: every warp has read the scale)
            for (int w = group * per; w < (group + 1) * per; ++w) amax = max(amax, s_max[flip][w]);
        }
        if (!live) continue;
        // a token in front that names the block, too: the block has another owner, the run is left out
        if (__any_sync(0xffffffffu, f0 >> shift == blk || f1 >> shift == blk)) {
            if (lane == 0) record_error(a.hdr, kErrSplitBlock);
            continue;
        }
        if (amax >= kB8Most && lane == 0) record_error(a.hdr, kErrBadValue);
        // (the larger one by their bits, as above: a NaN stays until the block is started anew)
        const float s = __uint_as_float(max(__float_as_uint(had), __float_as_uint(b8_scale<E4>(__uint_as_float(amax)))));
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
        uint2 *pool = reinterpret_cast<uint2 *>(is_v ? a.vpool : a.kpool) + (((int64_t)blk * a.Hkv + h) * bs + row0) * 16 + vec;
        if (part == 0 && lane == 0 && (r0 == 0 || s != had)) *scale = s;
        if (r0 > 0 && s > had) {  // the codes of the tokens in front, anew
            for (int i = 0; i < kB8Vecs; ++i) {
                if (row0 + 2 * i >= r0) break;
                uint2 c = pool[2 * i * 16];
                const float4 p = b8_decode4<E4>(c.x), q = b8_decode4<E4>(c.y);
                // code times scale is exact (15 bits); the quotient is rounded once, and is a tie exactly
                // or 2^-16 away from one at least, which fp32 tells apart
                auto again = [&](float u) { return __fdiv_rn(u * had, s); };
                if constexpr (E4) {
                    c.x = e4m3x4(again(p.x), again(p.y), again(p.z), again(p.w));
                    c.y = e4m3x4(again(q.x), again(q.y), again(q.z), again(q.w));
                } else {
                    c.x = b8_encode4<E4>(rintf(again(p.x)), rintf(again(p.y)), rintf(again(p.z)), rintf(again(p.w)), 1.0f);
                    c.y = b8_encode4<E4>(rintf(again(q.x)), rintf(again(q.y)), rintf(again(q.z)), rintf(again(q.w)), 1.0f);
                }
                pool[2 * i * 16] = c;
            }
        }
#pragma unroll
        for (int i = 0; i < kB8Vecs; ++i) {
            const int32_t r = row0 + 2 * i - r0;
            const uint4 w = x[i];
            uint2 c;
            c.x = b8_encode4<E4>(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x), bf16lo_to_f32(w.y), bf16hi_to_f32(w.y), inv);
            c.y = b8_encode4<E4>(bf16lo_to_f32(w.z), bf16hi_to_f32(w.z), bf16lo_to_f32(w.w), bf16hi_to_f32(w.w), inv);
            if (r >= 0 && r < n) pool[2 * i * 16] = c;
        }
    }
}

cudaError_t launch_store_block8(bool e4m3, const void *k, const void *v, int64_t k_stride, int64_t v_stride, int32_t T,
                                int32_t Hkv, int32_t bs, const int32_t *slots, uint8_t *kpool, uint8_t *vpool,
                                float *kscale, float *vscale, int32_t num_blocks, void *ws, int nsm, cudaStream_t stream)
{
    Block8Args a;
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.slots = slots;
    a.kpool = kpool;
    a.vpool = vpool;
    a.kscale = kscale;
    a.vscale = vscale;
    a.hdr = static_cast<WsHeader *>(ws);
    a.T = T;
    a.Hkv = Hkv;
    a.bs = bs;
    a.num_blocks = num_blocks;
    // the largest window with which there are still eight blocks of threads per SM (decode steps, where
    // every token is a run), each of them with the heads of its runs
    a.window = kB8Window;
    const int64_t want = 8 * (int64_t)nsm;
    const int groups = kB8Warps / (bs / kB8Rows);
    const int32_t heads = (2 * Hkv + groups - 1) / groups;  // turns that one run's heads of K and V take
    while (a.window > 1 && ((int64_t)T + a.window - 1) / a.window * heads < want) a.window /= 2;
    const dim3 grid((unsigned)((T + (int64_t)a.window - 1) / a.window), (unsigned)(heads < 65535 ? heads : 65535));
    if (e4m3) store_block8_kernel<true><<<grid, kB8Threads, 0, stream>>>(a);
    else store_block8_kernel<false><<<grid, kB8Threads, 0, stream>>>(a);
    return cudaGetLastError();
}

// ---- rows back in bf16 ------------------------------------------------------------------------------

struct Load8Args {
    const uint8_t *kpool, *vpool;
    const float *kscale, *vscale;
    const int32_t *bt, *cu;
    uint4 *k, *v;
    WsHeader *hdr;
    int32_t B, Hkv, bs, max_blocks, num_blocks, total;
};

// First row and rows of request b, held inside the buffers and the table's row (flagged when they were not).
__device__ __forceinline__ int2 load8_rows(const Load8Args &a, int32_t b, bool flag)
{
    const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    const int32_t r0 = min(max(c0, 0), a.total), r1 = min(max(c1, r0), a.total);
    const int32_t n = (int32_t)min((int64_t)(r1 - r0), (int64_t)a.max_blocks * a.bs);
    if (flag && (r0 != c0 || r1 != c1 || n != r1 - r0)) record_error(a.hdr, kErrBadLength);
    return make_int2(r0, n);
}

template <bool E4>
__global__ void __launch_bounds__(kB8Threads, 12) load_block8_kernel(const Load8Args a)
{
    extern __shared__ int32_t s_pre[];  // [B + 1] tiles of 16 tokens before each request
    __shared__ int32_t s_sum[kB8Warps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t carry = 0;
    for (int32_t base = 0; base < a.B; base += kB8Threads) {
        const int32_t b = base + tid;
        const int32_t c = b < a.B ? (load8_rows(a, b, blockIdx.x == 0).y + kB8Rows - 1) / kB8Rows : 0;
        int32_t x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        int32_t before = carry;
#pragma unroll
        for (int w = 0; w < kB8Warps; ++w) {
            if (w < warp) before += s_sum[w];
            carry += s_sum[w];
        }
        if (b < a.B) s_pre[b] = before + x - c;
        __syncthreads();
    }
    if (tid == 0) s_pre[a.B] = carry;
    __syncthreads();

    const int64_t items = (int64_t)carry * a.Hkv * 2;
    const int32_t shift = __ffs(a.bs) - 1;
    for (int64_t item = (int64_t)blockIdx.x * kB8Warps + warp; item < items; item += (int64_t)gridDim.x * kB8Warps) {
        // neighbouring warps: heads of the same tokens, whose rows lie side by side in the output
        const int32_t q = (int32_t)(item / a.Hkv), h = (int32_t)(item - (int64_t)q * a.Hkv), tile = q >> 1, kv = q & 1;
        int32_t lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int32_t mid = (lo + hi + 1) >> 1;
            if (s_pre[mid] <= tile) lo = mid;
            else hi = mid - 1;
        }
        const int2 rows = load8_rows(a, lo, false);
        const int32_t t0 = (tile - s_pre[lo]) * kB8Rows, n = min(kB8Rows, rows.y - t0);
        if ((uint32_t)t0 >= (uint32_t)rows.y) continue;  // (lengths so far off that their tiles pass 32 bits)
        int32_t blk = __ldg(a.bt + (int64_t)lo * a.max_blocks + (t0 >> shift));
        if ((uint32_t)blk >= (uint32_t)a.num_blocks) {  // not a block: flagged, and block 0 read instead
            record_error(a.hdr, kErrBadBlock);
            blk = 0;
        }
        const int64_t sc = (int64_t)blk * a.Hkv + h;
        // this lane: rows 2i + lane / 16, eight codes
        const int32_t row0 = lane >> 4, vec = lane & 15;
        const int64_t src = (sc * a.bs + (t0 & (a.bs - 1)) + row0) * 16 + vec;
        const int64_t dst = ((int64_t)(rows.x + t0 + row0) * a.Hkv + h) * 16 + vec;
        uint2 c[kB8Vecs];
#pragma unroll
        for (int i = 0; i < kB8Vecs; ++i)
            if (row0 + 2 * i < n) c[i] = __ldg(reinterpret_cast<const uint2 *>(kv ? a.vpool : a.kpool) + src + 32 * i);
        const float s = __ldg((kv ? a.vscale : a.kscale) + sc);
#pragma unroll
        for (int i = 0; i < kB8Vecs; ++i) {
            if (row0 + 2 * i >= n) continue;
            const float4 p = b8_decode4<E4>(c[i].x), q = b8_decode4<E4>(c[i].y);
            auto two = [&](float x, float y) {
                const __nv_bfloat162 w = __floats2bfloat162_rn(x * s, y * s);
                return *reinterpret_cast<const uint32_t *>(&w);
            };
            __stcs((kv ? a.v : a.k) + dst + (int64_t)2 * i * a.Hkv * 16,
                   make_uint4(two(p.x, p.y), two(p.z, p.w), two(q.x, q.y), two(q.z, q.w)));
        }
    }
}

cudaError_t launch_load_block8(bool e4m3, const uint8_t *kpool, const uint8_t *vpool, const float *kscale,
                               const float *vscale, int32_t num_blocks, const int32_t *bt, int32_t max_blocks,
                               const int32_t *cu, int32_t B, int32_t Hkv, int32_t bs, void *k, void *v, int32_t total,
                               void *ws, int nsm, cudaStream_t stream)
{
    Load8Args a;
    a.kpool = kpool;
    a.vpool = vpool;
    a.kscale = kscale;
    a.vscale = vscale;
    a.bt = bt;
    a.cu = cu;
    a.k = static_cast<uint4 *>(k);
    a.v = static_cast<uint4 *>(v);
    a.hdr = static_cast<WsHeader *>(ws);
    a.B = B;
    a.Hkv = Hkv;
    a.bs = bs;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.total = total;
    const int64_t most = ((int64_t)(total / kB8Rows) + B) * Hkv * 2;  // tiles there can be
    const int64_t need = (most + kB8Warps - 1) / kB8Warps, cap = B <= kB8Threads ? 0x7fffffff : (int64_t)nsm * 32;
    const unsigned grid = (unsigned)(need < cap ? (need < 1 ? 1 : need) : cap);
    const size_t smem = (size_t)(B + 1) * sizeof(int32_t);  // (33 KB at the largest batch)
    if (e4m3) load_block8_kernel<true><<<grid, kB8Threads, smem, stream>>>(a);
    else load_block8_kernel<false><<<grid, kB8Threads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dgq
