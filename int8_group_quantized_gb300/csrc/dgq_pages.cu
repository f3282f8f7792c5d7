// dgq_pages.cu -- pages of a paged cache copied between slots of its pools, and block tables
// rewritten after a compaction (sm_103a).
//
// One call copies the pages named by a list of (source, destination) ids in every array it is given:
// the K and V pools of all layers, the records of forked requests (a row of records is a page of
// Hkv * 128 bytes).  No arithmetic: each byte is read and written once, so HBM bounds the large
// calls and one launch's latency the small ones.  The plain way, one indexed copy per array, takes a
// gather and a scatter launch per array and moves every byte twice.
//
// Work: a page is cut into units of 4 KB, and a warp copies one unit with eight 16-byte loads per lane
// in flight before the first store; all units of all (pair, array) form one flat list with a warp for
// each.  400 pages of 64 KB in eight pools (420 MB moved): 65.5 us, 6.4 TB/s, 94% of the measured
// copy rate.  A grid of eight CTAs per SM whose warps walk the list took 72 us, bulk copies through
// shared memory (three to six buffers of 8 or 16 KB, three to six CTAs per SM) 72 to 75.
#include "dgq_device.cuh"
#include "dgq.h"
#include "dgq_launch.h"

namespace dgq {

constexpr int kCopyThreads = 128;
constexpr int kCopyCtasPerSm = 8;                         // 64 registers a thread: the loads stay in flight
constexpr int kCopyVecs = 8;                              // 16-byte vectors a lane keeps in flight
constexpr int32_t kUnitVecs = 32 * kCopyVecs;             // 4 KB
constexpr int kArraysPerLaunch = 256;                     // pointers that travel as kernel arguments

struct CopyArgs {
    uint4 *arrays[kArraysPerLaunch];
    const int2 *pairs;
    WsHeader *hdr;
    int64_t units;      // pairs * arrays * units of a page
    int64_t page_vecs;
    int32_t num_arrays, num_pages, num_pairs, page_units;
};

__global__ void __launch_bounds__(kCopyThreads, kCopyCtasPerSm) copy_pages_kernel(const __grid_constant__ CopyArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < a.units; u += warps) {
        // unit u: part of a page, then the pair, then the array (consecutive warps stay in one array)
        const int64_t item = u / a.page_units;
        const int32_t part = (int32_t)(u - item * a.page_units);
        const int32_t arr = (int32_t)(item / a.num_pairs);
        const int32_t pair = (int32_t)(item - (int64_t)arr * a.num_pairs);
        const int2 p = __ldg(a.pairs + pair);
        if ((uint32_t)p.x >= (uint32_t)a.num_pages || (uint32_t)p.y >= (uint32_t)a.num_pages) {
            if (lane == 0) record_error(a.hdr, kErrBadBlock);  // not a page: flagged, nothing copied
            continue;
        }
        const int64_t v0 = (int64_t)part * kUnitVecs + lane;
        const uint4 *src = a.arrays[arr] + p.x * a.page_vecs;
        uint4 *dst = a.arrays[arr] + p.y * a.page_vecs;
        uint4 x[kCopyVecs];
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i)
            if (v0 + 32 * i < a.page_vecs) x[i] = __ldcs(src + v0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i)
            if (v0 + 32 * i < a.page_vecs) __stcs(dst + v0 + 32 * i, x[i]);
    }
}

cudaError_t launch_copy_pages(void *const *arrays, int32_t num_arrays, int64_t page_bytes, int32_t num_pages,
                              const int32_t *pairs, int32_t num_pairs, void *ws, cudaStream_t stream)
{
    CopyArgs a;
    a.pairs = reinterpret_cast<const int2 *>(pairs);
    a.hdr = static_cast<WsHeader *>(ws);
    a.page_vecs = page_bytes / 16;
    a.num_pages = num_pages;
    a.num_pairs = num_pairs;
    a.page_units = (int32_t)((a.page_vecs + kUnitVecs - 1) / kUnitVecs);
    for (int32_t first = 0; first < num_arrays; first += kArraysPerLaunch) {
        a.num_arrays = num_arrays - first < kArraysPerLaunch ? num_arrays - first : kArraysPerLaunch;
        for (int32_t i = 0; i < a.num_arrays; ++i) a.arrays[i] = static_cast<uint4 *>(arrays[first + i]);
        a.units = (int64_t)a.num_arrays * num_pairs * a.page_units;
        const int64_t need = (a.units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
        copy_pages_kernel<<<(unsigned)(need < INT32_MAX ? need : INT32_MAX), kCopyThreads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// out[i] = remap[in[i]]; an entry that names no page is flagged and kept (in == out is allowed: each
// thread reads its entry before it writes it).
__global__ void __launch_bounds__(256) remap_tables_kernel(const int32_t *in, int64_t n, const int32_t *remap,
                                                           int32_t num_pages, int32_t *out, WsHeader *hdr)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
        const int32_t id = in[i];
        int32_t to = id;
        if ((uint32_t)id < (uint32_t)num_pages) to = __ldg(remap + id);
        else record_error(hdr, kErrBadBlock);
        out[i] = to;
    }
}

cudaError_t launch_remap_tables(const int32_t *in, int64_t n, const int32_t *remap, int32_t num_pages, int32_t *out,
                                void *ws, int nsm, cudaStream_t stream)
{
    const int64_t need = (n + 255) / 256, most = (int64_t)nsm * 8;
    remap_tables_kernel<<<(unsigned)(need < most ? need : most), 256, 0, stream>>>(
        in, n, remap, num_pages, out, static_cast<WsHeader *>(ws));
    return cudaGetLastError();
}

}  // namespace dgq
