// dgq_tables.cu -- block tables extended and slot maps made from the requests' lengths, and rows written
// to a bf16 paged cache by slot (sm_103a).
//
// Request b has L_b cached tokens in ceil(L_b / bs) blocks and gets n_b new ones: need_b = ceil((L_b + n_b)
// / bs) - ceil(L_b / bs) blocks, the next ids of a free list in request order, so its blocks start at
// used + sum_{a < b} need_a.  New token i sits at position p = L_b + i, in slot table[b][p / bs] * bs + p % bs.
//
// Tables: whole numbers, a few bytes per token, so one launch's latency is the cost.  Every block scans all
// requests by itself (8 bytes each, in L2) rather than wait for another block's scan, and then makes the
// slots of its own tokens: the block of a token is in the table where the request had it before, and else
// follows from the scan, so nothing is read that another block writes.  A column is written by the thread
// of the block's first token.  The outputs that may lie over the inputs (lengths, ids used) are written
// by the last block to have read them (a count in the workspace header, back at 0 afterwards).  Two
// requests of one token: 3.5 us in a graph; 64 requests with 36600 new tokens: 6.2.
//
// Rows: each byte read and written once, so HBM bounds the large calls.  A warp moves 2 KB of K and 2 KB
// of V, eight 16-byte loads per lane in flight before the first store.  36600 tokens of 8 heads (300 MB moved):
// 48.6 us, 92% of the measured copy rate.
#include "dgq_device.cuh"
#include "dgq.h"
#include "dgq_launch.h"

namespace dgq {

constexpr int kExtendThreads = 256;
constexpr int kExtendTokens = 4;  // consecutive tokens of a thread: one 16-byte store

__global__ void __launch_bounds__(kExtendThreads) extend_tables_kernel(const ExtendArgs a, WsHeader *hdr)
{
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm;                // [B + 1] first token of a request, held to total_slots
    int32_t *s_len = s_cu + a.B + 1;   // [B] cached tokens, or -1: the request gets nothing
    int32_t *s_first = s_len + a.B;    // [B] place of its first new block in the free list
    __shared__ int64_t s_tok[kExtendThreads / 32], s_need[kExtendThreads / 32];
    __shared__ int32_t s_used, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first_block = blockIdx.x == 0;
    const int32_t bs = a.bs, shift = __ffs(bs) - 1;
    const int64_t room = (int64_t)a.max_blocks * bs;

    const int32_t used = __ldcg(a.free_used);
    const bool used_ok = used >= 0 && used <= a.num_free;
    if (tid == 0) {
        s_used = used;
        if (!used_ok && first_block) record_error(hdr, kErrBadLength);
    }
    int64_t tok_carry = 0, need_carry = 0;
    for (int32_t base = 0; base < a.B; base += kExtendThreads) {
        const int32_t b = base + tid;
        int64_t n = 0, need = 0;
        int32_t L = -1;
        bool bad = false;
        if (b < a.B) {
            L = __ldcg(a.seq_lens + b);
            n = __ldcg(a.new_lens + b);
            bad = L < 0 || n < 0 || (int64_t)L + n > room;
            if (n < 0) n = 0;
            if (!bad) need = (((int64_t)L + n + bs - 1) >> shift) - (((int64_t)L + bs - 1) >> shift);
        }
        int64_t tx = n, nx = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, tx, o), y = __shfl_up_sync(0xffffffffu, nx, o);
            if (lane >= o) {
                tx += t;
                nx += y;
            }
        }
        if (lane == 31) {
            s_tok[warp] = tx;
            s_need[warp] = nx;
        }
        __syncthreads();
        int64_t tok0 = tok_carry, need0 = need_carry;
#pragma unroll
        for (int w = 0; w < kExtendThreads / 32; ++w) {
            if (w < warp) {
                tok0 += s_tok[w];
                need0 += s_need[w];
            }
            tok_carry += s_tok[w];
            need_carry += s_need[w];
        }
        tok0 += tx - n;
        need0 += nx - need;
        if (b < a.B) {
            bool out = bad || tok0 + n > a.total_slots;  // rows that the buffers do not have
            if (out && first_block) record_error(hdr, kErrBadLength);
            if (!out && need > 0 && (!used_ok || used + need0 + need > a.num_free)) {
                out = true;
                if (first_block) record_error(hdr, kErrNoBlock);
            }
            s_cu[b] = (int32_t)min(tok0, (int64_t)a.total_slots);
            s_len[b] = out ? -1 : L;
            s_first[b] = (int32_t)min(used + need0, (int64_t)INT32_MAX);
            // the blocks that are handed out end with the last request that got some
            if (!out && need > 0) atomicMax(&s_used, (int32_t)(used + need0 + need));
        }
        __syncthreads();
    }
    uint32_t before = 0u;
    if (tid == 0) {
        s_cu[a.B] = (int32_t)min(tok_carry, (int64_t)a.total_slots);
        if (gridDim.x > 1) {
            __threadfence();  // everything above was read; the last block may overwrite it
            before = atomicAdd(&hdr->ended_ctas, 1u);  // (its answer is looked at behind the slots)
        }
    }
    __syncthreads();
    const int32_t total = s_cu[a.B];

    const int64_t stride = (int64_t)gridDim.x * kExtendThreads * kExtendTokens;
    for (int64_t t0 = ((int64_t)blockIdx.x * kExtendThreads + tid) * kExtendTokens; t0 < a.total_slots; t0 += stride) {
        int32_t slot[kExtendTokens];
        int32_t b = 0;
        if (t0 < total) {  // the last request that starts at or before t0 (empty ones share their start with the next)
            int32_t lo = 0, hi = a.B - 1;
            while (lo < hi) {
                const int32_t mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t0) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
        }
#pragma unroll
        for (int k = 0; k < kExtendTokens; ++k) {
            const int32_t t = (int32_t)t0 + k;
            slot[k] = -1;
            if (t >= total) continue;
            while (s_cu[b + 1] <= t) ++b;
            const int32_t L = s_len[b];
            if (L < 0) continue;
            const int32_t p = L + (t - s_cu[b]), col = p >> shift, had = (int32_t)(((int64_t)L + bs - 1) >> shift);
            int32_t *entry = a.tables + (int64_t)b * a.max_blocks + col;
            const int32_t id = col >= had ? __ldg(a.free_ids + s_first[b] + (col - had)) : *entry;
            if ((uint32_t)id >= (uint32_t)a.num_blocks) {  // not a block: flagged, the token has no slot
                record_error(hdr, kErrBadBlock);
                continue;
            }
            slot[k] = (id << shift) + (p & (bs - 1));
            if ((p & (bs - 1)) == 0) *entry = id;
        }
        if (t0 + kExtendTokens <= a.total_slots) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kExtendTokens; ++k)
                if (t0 + k < a.total_slots) a.slots[t0 + k] = slot[k];
        }
    }

    if (tid == 0) {
        s_last = before + 1u == gridDim.x;
        if (s_last && gridDim.x > 1) hdr->ended_ctas = 0u;  // for the next call
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int32_t b = tid; b < a.B; b += kExtendThreads) {
        const int32_t L = s_len[b];
        // (a request that gets nothing keeps its length; the inputs are as they were until here)
        a.seq_lens_out[b] = L < 0 ? __ldcg(a.seq_lens + b) : L + (s_cu[b + 1] - s_cu[b]);
    }
    for (int32_t b = tid; b <= a.B; b += kExtendThreads) a.cu_new[b] = s_cu[b];
    if (tid == 0) *a.free_used_out = s_used;
}

size_t extend_smem_bytes(int32_t B) { return (size_t)(3 * B + 1) * sizeof(int32_t); }

cudaError_t launch_extend_tables(const ExtendArgs &a, void *ws, int nsm, cudaStream_t stream)
{
    static thread_local int limit_dev = -1;  // raised once per device and host thread, to the largest call's
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != limit_dev) {
        e = cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)extend_smem_bytes(kMaxCallBatch));
        if (e != cudaSuccess) return e;
        limit_dev = dev;
    }
    // two blocks per SM: every block repeats the scan
    const int64_t per = kExtendThreads * kExtendTokens, need = (a.total_slots + per - 1) / per, most = 2 * (int64_t)nsm;
    const int64_t grid = need < 1 ? 1 : (need < most ? need : most);
    extend_tables_kernel<<<(unsigned)grid, kExtendThreads, extend_smem_bytes(a.B), stream>>>(a, static_cast<WsHeader *>(ws));
    return cudaGetLastError();
}

// ---- rows by slot ---------------------------------------------------------------------------------

constexpr int kWriteThreads = 128;
constexpr int kWriteVecs = 4;                            // 16-byte vectors of K, and of V, per lane
constexpr int32_t kWriteUnit = 32 * kWriteVecs;          // vectors of a warp: 2 KB

struct WriteArgs {
    const uint4 *k, *v;
    uint4 *kp, *vp;
    const int32_t *slots;
    WsHeader *hdr;
    int64_t k_stride, v_stride;  // vectors from a token to the next
    uint32_t vecs, row_vecs;     // vectors of all tokens and of one token, per tensor (< 2^31)
    int32_t Hkv, shift, num_slots;
};

__global__ void __launch_bounds__(kWriteThreads) write_slots_kernel(const WriteArgs a)
{
    const int lane = threadIdx.x & 31;
    const uint32_t unit = blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
    const uint64_t first = (uint64_t)unit * kWriteUnit + lane;
    uint4 k[kWriteVecs], v[kWriteVecs];
    int64_t to[kWriteVecs];
#pragma unroll
    for (int i = 0; i < kWriteVecs; ++i) {
        to[i] = -1;
        if (first + 32 * i >= a.vecs) continue;
        const uint32_t x = (uint32_t)first + 32 * i, token = x / a.row_vecs, r = x - token * a.row_vecs;
        const int32_t slot = __ldg(a.slots + token);
        if (slot == -1) continue;                             // a token without a place
        if ((uint32_t)slot >= (uint32_t)a.num_slots) {        // not a slot: flagged, nothing written
            record_error(a.hdr, kErrBadBlock);
            continue;
        }
        const int32_t h = r >> 4, in = slot & ((1 << a.shift) - 1);  // 16 vectors to a head's row
        to[i] = (((((int64_t)(slot >> a.shift) * a.Hkv + h) << a.shift) + in) << 4) + (r & 15);
        k[i] = __ldcs(a.k + token * a.k_stride + r);
        v[i] = __ldcs(a.v + token * a.v_stride + r);
    }
#pragma unroll
    for (int i = 0; i < kWriteVecs; ++i)
        if (to[i] >= 0) {
            a.kp[to[i]] = k[i];
            a.vp[to[i]] = v[i];
        }
}

cudaError_t launch_write_slots(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int32_t T, int32_t Hkv,
                               int32_t bs, const int32_t *slots, void *k_pages, void *v_pages, int32_t num_blocks,
                               void *ws, cudaStream_t stream)
{
    WriteArgs a;
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.kp = static_cast<uint4 *>(k_pages);
    a.vp = static_cast<uint4 *>(v_pages);
    a.slots = slots;
    a.hdr = static_cast<WsHeader *>(ws);
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.row_vecs = (uint32_t)Hkv * 16;
    a.vecs = (uint32_t)T * a.row_vecs;
    a.Hkv = Hkv;
    a.shift = __builtin_ctz((unsigned)bs);
    a.num_slots = num_blocks * bs;
    const uint32_t units = (a.vecs + kWriteUnit - 1) / kWriteUnit;
    write_slots_kernel<<<(units + kWriteThreads / 32 - 1) / (kWriteThreads / 32), kWriteThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dgq
