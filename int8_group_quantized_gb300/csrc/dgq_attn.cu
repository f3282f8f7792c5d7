// dgq_attn.cu -- decode-step attention: launcher, workspace layout, and the merges of pairs that several
// CTAs share (sm_103a).  The main kernel: dgq_attn_kernel.cuh.
#include "dgq_attn_kernel.cuh"

namespace dgq {

// Merge of the pieces of every pair that several CTAs share, after the main kernel
// (programmatic dependent launch).  One item per (pair, query head); a grid of at most 4 CTAs
// per SM walks the items (at 128 registers a thread the slot arrays below stay in registers),
// and these small CTAs can already be resident while the main kernel runs.  The pieces are
// folded in a fixed order and the current token is added last, as in the single-piece path:
// the warp merge folds an item's pieces in CTA order, kCombineSlots loads in flight per round;
// the block merge gives warp w the pieces of CTAs cfirst + w, + 4, ... (in that order,
// kCombineSlots per round) and then folds the four warps' states in warp order.
constexpr int kCombineWarps = 4;
constexpr int kCombineSlots = 8;    // pieces one warp keeps in flight per round
constexpr int kCombineCtasPerSm = 4;  // 128 registers a thread: the slot arrays stay in registers
// combine_kernel reads the current value and writes the output with one thread per dimension
static_assert(kCombineWarps * 32 == kD, "the block merge has exactly one thread per head dimension");

__global__ void __launch_bounds__(kCombineWarps * 32, kCombineCtasPerSm) combine_kernel(AttnArgs a)
{
    const int32_t G = a.G, Hkv = a.Hkv;
    const int32_t items = a.B * Hkv * G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ float s_m[kCombineWarps], s_l[kCombineWarps];
    __shared__ float4 s_o[kCombineWarps][32];
    __shared__ float s_sn;
    if (blockIdx.x == 0 && tid == 0) a.hdr->path = kPathBlockMerge;  // which merge ran (tests read it)

    bool waited = false;
    for (int32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int32_t p = item / G, g = item - p * G;
        const int32_t b = p / Hkv, h = p - b * Hkv;
        // inputs of this call (not written by the main kernel): loaded before the wait
        const uint2 qv = __ldg(reinterpret_cast<const uint2 *>(a.q + ((int64_t)b * a.Hq + h * G + g) * kD) + lane);
        const uint2 kv = __ldg(reinterpret_cast<const uint2 *>(a.knew + ((int64_t)b * Hkv + h) * kD) + lane);
        const float vn = bf16lo_to_f32((uint32_t)__ldg(a.vnew + ((int64_t)b * Hkv + h) * kD + tid));
        if (!waited) {
            pdl_wait_primary();
            waited = true;
        }
        const int2 info = __ldcg(a.pair_info + p);
        const int32_t cfirst = info.x, clast = info.y;
        if (cfirst == clast) continue;  // finished inside the main kernel
        const bool all_held = __ldcg(&a.hdr->pad[kHdrAllHeld]) != 0;  // no slot is empty

        // warp w folds slots cfirst + w, + 4, ...: per slot its (m, l) and this lane's 4 columns of O
        float m_w = -INFINITY, l_w = 0.0f;
        float4 o_w = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t base = cfirst + warp; base <= clast; base += kCombineWarps * kCombineSlots) {
            float mm[kCombineSlots], ll[kCombineSlots];
            float4 oo[kCombineSlots];
#pragma unroll
            for (int i = 0; i < kCombineSlots; ++i) {
                const int32_t cc = base + i * kCombineWarps;
                mm[i] = -INFINITY;
                ll[i] = 0.0f;
                oo[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cc <= clast) {
                    const float *src = a.part + ((int64_t)(p + cc) * G + g) * kPartStride;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src));
                    mm[i] = ml.x;
                    ll[i] = ml.y;
                    oo[i] = __ldcg(reinterpret_cast<const float4 *>(src + 4) + lane);
                }
            }
            // the slot of a CTA whose slice is empty holds stale data (no piece of this call
            // writes it): dropped
            if (!all_held) {
#pragma unroll
                for (int i = 0; i < kCombineSlots; ++i) {
                    const int32_t cc = base + i * kCombineWarps;
                    if (cc <= clast && __ldcg(a.held + cc) == 0) {
                        mm[i] = -INFINITY;
                        ll[i] = 0.0f;
                        oo[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kCombineSlots; ++i) {  // in slot order: online fold
                const float M = fmaxf(m_w, mm[i]);
                if (M == -INFINITY) continue;
                const float fo = m_w == -INFINITY ? 0.0f : ex2(m_w - M);
                const float fn = mm[i] == -INFINITY ? 0.0f : ex2(mm[i] - M);
                l_w = l_w * fo + ll[i] * fn;
                o_w.x = o_w.x * fo + oo[i].x * fn;
                o_w.y = o_w.y * fo + oo[i].y * fn;
                o_w.z = o_w.z * fo + oo[i].z * fn;
                o_w.w = o_w.w * fo + oo[i].w * fn;
                m_w = M;
            }
        }
        if (lane == 0) {
            s_m[warp] = m_w;
            s_l[warp] = l_w;
        }
        s_o[warp][lane] = o_w;
        if (warp == 0) {  // the current token's score
            float acc = bf16lo_to_f32(qv.x) * bf16lo_to_f32(kv.x);
            acc = fmaf(bf16hi_to_f32(qv.x), bf16hi_to_f32(kv.x), acc);
            acc = fmaf(bf16lo_to_f32(qv.y), bf16lo_to_f32(kv.y), acc);
            acc = fmaf(bf16hi_to_f32(qv.y), bf16hi_to_f32(kv.y), acc);
#pragma unroll
            for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
            if (lane == 0) s_sn = acc * kLog2eOverSqrtD;
        }
        __syncthreads();
        {  // thread d: fold the warps in order, then the current token
            const int d = tid;
            float M = -INFINITY, L = 0.0f, O = 0.0f;
            for (int w = 0; w < kCombineWarps; ++w) {
                const float mw = s_m[w];
                const float Mn = fmaxf(M, mw);
                if (Mn == -INFINITY) continue;
                const float fo = M == -INFINITY ? 0.0f : ex2(M - Mn);
                const float fn = mw == -INFINITY ? 0.0f : ex2(mw - Mn);
                const float ow = reinterpret_cast<const float *>(&s_o[w][d >> 2])[d & 3];
                L = L * fo + s_l[w] * fn;
                O = O * fo + ow * fn;
                M = Mn;
            }
            __nv_bfloat16 ob = __float2bfloat16_rn(finish(M, L, O, s_sn, vn));
            a.out[((int64_t)b * a.Hq + h * G + g) * kD + d] = *reinterpret_cast<uint16_t *>(&ob);
        }
        __syncthreads();  // shared memory is reused by the next item
    }
    if (!waited) pdl_wait_primary();
}

// The same merge with one warp per (pair, query head) item, for calls whose pairs are split over
// few CTAs: the warp folds the pieces in CTA order (kCombineSlots in flight), adds the current
// token and writes its four columns per lane; no shared memory and no block barrier.
__global__ void __launch_bounds__(kCombineWarps * 32, kCombineCtasPerSm) combine_warp_kernel(AttnArgs a)
{
    const int32_t G = a.G, Hkv = a.Hkv;
    const int32_t items = a.B * Hkv * G;
    const int lane = threadIdx.x & 31;
    const int32_t nw = gridDim.x * kCombineWarps;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->path = kPathWarpMerge;  // which merge ran (tests read it)
    bool waited = false;
    for (int32_t item = blockIdx.x * kCombineWarps + (threadIdx.x >> 5); item < items; item += nw) {
        const int32_t p = item / G, g = item - p * G;
        const int32_t b = p / Hkv, h = p - b * Hkv;
        // inputs of this call (not written by the main kernel): loaded before the wait
        const uint2 qv = __ldg(reinterpret_cast<const uint2 *>(a.q + ((int64_t)b * a.Hq + h * G + g) * kD) + lane);
        const uint2 kv = __ldg(reinterpret_cast<const uint2 *>(a.knew + ((int64_t)b * Hkv + h) * kD) + lane);
        const uint2 vv = __ldg(reinterpret_cast<const uint2 *>(a.vnew + ((int64_t)b * Hkv + h) * kD) + lane);
        if (!waited) {
            pdl_wait_primary();
            waited = true;
        }
        const int2 info = __ldcg(a.pair_info + p);
        const int32_t cfirst = info.x, clast = info.y;
        if (cfirst == clast) continue;  // finished inside the main kernel
        const bool all_held = __ldcg(&a.hdr->pad[kHdrAllHeld]) != 0;  // no slot is empty
        float M = -INFINITY, L = 0.0f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t base = cfirst; base <= clast; base += kCombineSlots) {
            float mm[kCombineSlots], ll[kCombineSlots];
            float4 oo[kCombineSlots];
#pragma unroll
            for (int i = 0; i < kCombineSlots; ++i) {
                const int32_t cc = base + i;
                mm[i] = -INFINITY;
                ll[i] = 0.0f;
                oo[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cc <= clast) {
                    const float *src = a.part + ((int64_t)(p + cc) * G + g) * kPartStride;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src));
                    mm[i] = ml.x;
                    ll[i] = ml.y;
                    oo[i] = __ldcg(reinterpret_cast<const float4 *>(src + 4) + lane);
                }
            }
            // the slot of a CTA whose slice is empty holds stale data (no piece of this call
            // writes it): dropped
            if (!all_held) {
#pragma unroll
                for (int i = 0; i < kCombineSlots; ++i) {
                    const int32_t cc = base + i;
                    if (cc <= clast && __ldcg(a.held + cc) == 0) {
                        mm[i] = -INFINITY;
                        ll[i] = 0.0f;
                        oo[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kCombineSlots; ++i) {  // in CTA order: online fold
                const float Mn = fmaxf(M, mm[i]);
                if (Mn == -INFINITY) continue;
                const float fo = M == -INFINITY ? 0.0f : ex2(M - Mn);
                const float fn = mm[i] == -INFINITY ? 0.0f : ex2(mm[i] - Mn);
                L = L * fo + ll[i] * fn;
                O.x = O.x * fo + oo[i].x * fn;
                O.y = O.y * fo + oo[i].y * fn;
                O.z = O.z * fo + oo[i].z * fn;
                O.w = O.w * fo + oo[i].w * fn;
                M = Mn;
            }
        }
        // the current token's score, then this lane's columns 4 lane .. 4 lane + 3
        float acc = bf16lo_to_f32(qv.x) * bf16lo_to_f32(kv.x);
        acc = fmaf(bf16hi_to_f32(qv.x), bf16hi_to_f32(kv.x), acc);
        acc = fmaf(bf16lo_to_f32(qv.y), bf16lo_to_f32(kv.y), acc);
        acc = fmaf(bf16hi_to_f32(qv.y), bf16hi_to_f32(kv.y), acc);
#pragma unroll
        for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        const float sn = acc * kLog2eOverSqrtD;
        uint2 res;
        res.x = pack_bf16x2(finish(M, L, O.x, sn, bf16lo_to_f32(vv.x)), finish(M, L, O.y, sn, bf16hi_to_f32(vv.x)));
        res.y = pack_bf16x2(finish(M, L, O.z, sn, bf16lo_to_f32(vv.y)), finish(M, L, O.w, sn, bf16hi_to_f32(vv.y)));
        reinterpret_cast<uint2 *>(a.out + ((int64_t)b * a.Hq + h * G + g) * kD)[lane] = res;
    }
    if (!waited) pdl_wait_primary();
}

}  // namespace dgq

// ---- host launcher ---------------------------------------------------------------------------

namespace dgq {

size_t attn_smem_bytes(int dec, int32_t B, int32_t G)
{
    const int ring = dec == kDecBf16    ? ring_bytes<kDecBf16>()
                     : dec == kDecFixed ? ring_bytes<kDecFixed>()
                     : dec == kDecBlockI8 || dec == kDecBlockE4 ? ring_bytes<kDecBlockI8>()
                                        : ring_bytes<kDecAffine>();
    const int piece = dec == kDecSplitV ? piece_bytes<kDecSplitV>() : piece_bytes<kDecAffine>();
    return 1024 + (size_t)kWarpsPerCta * ring + 2 * (size_t)piece + 16 + (size_t)kWarpsPerCta * G * kPartStride * 4 +
           8 * 4 + (size_t)(2 * B + 1) * 4;
}

// Short pairs (of the instances that can): every CTA takes whole pairs, and there is no merge, its launch and
// its reads.  Four warps then go through a pair's tiles alone, so it pays up to so many tiles of the longest
// pair, more where there are pairs for most SMs.  us, whole against split: 4 pairs of 256 tokens 7.2 / 8.7, of 512
// 9.8 / 8.8; 64 pairs of 512 10.8 / 11.3, of 1024 14.9 / 12.3; 256 pairs of 512 13.7 / 17.3; 1024 pairs of 512
// 34.1 / 36.1, of 1024 56.4 / 54.9; window 128 of 64 requests up to 32768 15.8 / 19.2, window 512 28.8 / 30.2.
constexpr int64_t kWholeTiles = 24, kWholeTilesMany = 40, kWholeMany = 64;

int attn_max_ctas(int nsm) { return nsm * kMaxCtasPerSm; }

AttnLayout attn_layout(int32_t batch, int32_t Hq, int32_t Hkv, int nsm)
{
    AttnLayout l;
    const size_t P = (size_t)batch * Hkv;
    const size_t G = (size_t)(Hq / Hkv);
    size_t off = sizeof(WsHeader);
    l.off_count = off;  // per-pair piece range (int2)
    off = (off + P * 8 + 255) & ~size_t(255);
    l.off_held = off;  // per CTA of the main kernel (int32)
    off = (off + (size_t)attn_max_ctas(nsm) * 4 + 255) & ~size_t(255);
    l.off_part = off;
    off += (P + (size_t)attn_max_ctas(nsm)) * G * kPartStride * 4;
    l.total = (off + 255) & ~size_t(255);
    return l;
}

cudaError_t launch_attn(int32_t format, const void *q, const void *knew, const void *vnew, const uint8_t *kpool,
                        const uint8_t *vpool, const dgq_seg_record *table, const dgq_seg_record *vtable,
                        const float *kpar, const float *vpar,
                        const int32_t *bt, const int32_t *seq_lens, int32_t max_seqlen, int32_t B, int32_t Hq,
                        int32_t Hkv, int32_t bs, int32_t max_blocks, int32_t num_blocks, int32_t window, int32_t sinks,
                        void *out, void *ws, int nsm, bool *map_failed, cudaStream_t stream)
{
    *map_failed = false;
    const int32_t G = Hq / Hkv;
    AttnLayout l = attn_layout(B, Hq, Hkv, nsm);
    char *base = static_cast<char *>(ws);
    AttnArgs a;
    a.q = static_cast<const uint16_t *>(q);
    a.knew = static_cast<const uint16_t *>(knew);
    a.vnew = static_cast<const uint16_t *>(vnew);
    a.kpool = kpool;
    a.vpool = vpool;
    a.table = table;
    a.vtable = vtable;
    a.kpar = reinterpret_cast<const float4 *>(kpar);
    a.vpar = reinterpret_cast<const float4 *>(vpar);
    a.kscale = kpar;  // (a block cache's scales; 4 bytes each)
    a.vscale = vpar;
    a.window = window;
    a.sinks = sinks;
    a.bt = bt;
    a.seq_lens = seq_lens;
    a.out = static_cast<uint16_t *>(out);
    a.hdr = reinterpret_cast<WsHeader *>(base);
    a.pair_info = reinterpret_cast<int2 *>(base + l.off_count);
    a.held = reinterpret_cast<int32_t *>(base + l.off_held);
    a.part = reinterpret_cast<float *>(base + l.off_part);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.bs = bs;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;

    // the kernel instance for the code format (the symmetric INT8 cache is an affine one)
    const bool win = window > 0;
    const int dec = format == kFormatBf16Cache      ? kDecBf16
                    : format == kFormatBlockInt8    ? kDecBlockI8
                    : format == kFormatBlockE4m3    ? kDecBlockE4
                    : vtable != nullptr             ? kDecSplitV
                    : format == DGQ_FORMAT_FP8_E4M3 ? kDecFp8
                    : format == DGQ_FORMAT_FIXED64  ? kDecFixed
                                                    : kDecAffine;
    AttnKernel kern = win || dec == kDecBlockI8 || dec == kDecBlockE4 ? attn_window_kernel(dec, win)
                      : dec == kDecBf16   ? attn_kernel<kDecBf16, false>
                      : dec == kDecFp8    ? attn_kernel<kDecFp8, false>
                      : dec == kDecFixed  ? attn_kernel<kDecFixed, false>
                      : dec == kDecSplitV ? attn_kernel<kDecSplitV, false>
                                          : attn_kernel<kDecAffine, false>;
    if (!kern) return cudaErrorInvalidValue;
    const int inst = dec + (win ? kNumDec : 0);

    // per-device launch shape, computed once per (instance, device, shared-memory size) and host
    // thread; the kernel's shared-memory limit is raised once per device and host thread to what
    // the largest call needs (every thread sets the same value, so none lowers it under another)
    struct Shape {
        int limit_dev, dev, occ;
        size_t smem;
    };
    static thread_local Shape shapes[2 * kNumDec];
    static thread_local bool fresh = true;
    if (fresh) {
        for (Shape &x : shapes) x = Shape{-1, -1, 0, 0};
        fresh = false;
    }
    Shape &shape = shapes[inst];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const size_t smem = attn_smem_bytes(dec, B, G);
    if (dev != shape.limit_dev) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)attn_smem_bytes(dec, kMaxCallBatch, kMaxGroup));
        if (e != cudaSuccess) return e;
        shape.limit_dev = dev;
    }
    if (dev != shape.dev || smem != shape.smem) {
        int occ = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kAttnThreads, smem);
        if (e != cudaSuccess) return e;
        if (occ < 1) return cudaErrorInvalidConfiguration;
        shape.dev = dev;
        shape.smem = smem;
        shape.occ = occ > kMaxCtasPerSm ? kMaxCtasPerSm : occ;
    }
    // upper bound on tiles (every request at max_seqlen): no more CTAs than tiles
    int64_t per_pair = max_seqlen > 0 ? (max_seqlen + kTile - 1) / kTile : 1;
    if (win) {  // sinks, and a window that begins and ends inside a tile
        const int64_t seen = ((int64_t)sinks + kTile - 1) / kTile + ((int64_t)window + kTile - 1) / kTile + 1;
        if (per_pair > seen) per_pair = seen;
    }
    const int64_t tiles = (int64_t)B * Hkv * per_pair;
    int64_t grid = (int64_t)nsm * shape.occ;
    a.whole = (win || dec == kDecBlockI8 || dec == kDecBlockE4) &&
              per_pair <= ((int64_t)B * Hkv >= kWholeMany ? kWholeTilesMany : kWholeTiles);
    if (a.whole && grid > (int64_t)B * Hkv) grid = (int64_t)B * Hkv;
    if (grid > tiles) grid = tiles;
    if (grid < 1) grid = 1;
    kern<<<(unsigned)grid, kAttnThreads, smem, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.whole) return e;

    // merge of shared pairs, chained with programmatic dependent launch
    cudaLaunchConfig_t cfg = {};
    const int64_t items = (int64_t)B * Hkv * G;
    // pairs split over few CTAs (at least one pair per two CTAs): one warp per item; otherwise
    // the four warps of a CTA share an item's pieces
    const bool warp_merge = (int64_t)B * Hkv * 2 >= grid;
    const int64_t per_cta = warp_merge ? kCombineWarps : 1;
    const int64_t cneed = (items + per_cta - 1) / per_cta;
    const int64_t cgrid = cneed < (int64_t)nsm * kCombineCtasPerSm ? cneed : (int64_t)nsm * kCombineCtasPerSm;
    cfg.gridDim = dim3((unsigned)cgrid);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return warp_merge ? cudaLaunchKernelEx(&cfg, combine_warp_kernel, a) : cudaLaunchKernelEx(&cfg, combine_kernel, a);
}

}  // namespace dgq
