// dgq_host.cu -- the C ABI of libdgq.so: argument checks, workspace sizing, launch,
// device error read-back, and the host block pool.  Every check runs before any launch.
#include "dgq.h"

#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <new>
#include <vector>

#include "dgq_launch.h"

static_assert(sizeof(dgq_seg_record) == 128, "dgq_seg_record must be 128 bytes");

namespace dgq {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static thread_local PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}
}  // namespace dgq

namespace {

constexpr int32_t kMaxBatch = dgq::kMaxCallBatch;  // per-call limit (the kernels keep per-request prefixes on chip)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A window and its sinks as the kernels take them (no request has more keys than this).
int32_t held(int32_t x) { return x < (1 << 30) ? x : 1 << 30; }

bool window_ok(int32_t window, int32_t sinks) { return window >= 1 && sinks >= 0; }

bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64; }

int device_sm_count(int *nsm)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    return 0;
}

}  // namespace

extern "C" {

const char *dgq_status_str(dgq_status s)
{
    switch (s) {
    case DGQ_OK: return "ok";
    case DGQ_ERR_INVALID_ARG: return "invalid argument";
    case DGQ_ERR_UNSUPPORTED: return "unsupported shape";
    case DGQ_ERR_WORKSPACE: return "workspace too small or missing";
    case DGQ_ERR_CUDA: return "CUDA error";
    case DGQ_ERR_POOL_EXHAUSTED: return "block pool exhausted";
    case DGQ_ERR_DEVICE: return "device-side wait timed out";
    case DGQ_ERR_SCRATCH_LIMIT: return "problem too large for the fixed no-allocation scratch array";
    }
    return "unknown status";
}

size_t dgq_compress_workspace_size(int32_t batch, int32_t max_seqlen, int32_t num_kv_heads)
{
    if (batch <= 0 || max_seqlen < 0 || num_kv_heads <= 0) return 0;
    return dgq::compress_layout(batch, max_seqlen, num_kv_heads).total;
}

dgq_status dgq_compress(const void *k_bf16, const void *v_bf16, int32_t total_tokens, const int32_t *cu_seqlens_dev,
                        int32_t batch, int32_t max_seqlen, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        const int32_t *block_tables_dev, int32_t max_blocks_per_seq, uint8_t *k_pool,
                        uint8_t *v_pool, int32_t num_blocks, dgq_seg_record *seg_table, void *workspace,
                        size_t workspace_bytes, void *cuda_stream)
{
    return dgq_compress_ex(k_bf16, v_bf16, total_tokens, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, head_dim,
                           block_size, block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table,
                           workspace, workspace_bytes, nullptr, cuda_stream);
}

namespace {

// Checks and launch shared by the packed and the paged-source entry points.
dgq_status compress_impl(const dgq::SourceDesc &src, const int32_t *cu_seqlens_dev, int32_t batch,
                         int32_t max_seqlen, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         const int32_t *block_tables_dev, int32_t max_blocks_per_seq, uint8_t *k_pool,
                         uint8_t *v_pool, int32_t num_blocks, dgq_seg_record *seg_table, void *workspace,
                         size_t workspace_bytes, const dgq_compress_options *options, void *cuda_stream)
{
    dgq::GroupSettings gs = {DGQ_MAX_SEG, 0.0f};
    if (options) {
        if (options->max_groups < 1 || options->max_groups > DGQ_MAX_SEG || !(options->min_var >= 0.0f) ||
            !(options->min_var <= 3.4e38f))
            return DGQ_ERR_INVALID_ARG;
        gs.max_groups = options->max_groups;
        gs.min_var = options->min_var;
    }
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || max_seqlen < 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0)
        return DGQ_ERR_INVALID_ARG;
    if ((int64_t)max_seqlen > (int64_t)max_blocks_per_seq * block_size) return DGQ_ERR_INVALID_ARG;
    if (src.bt == nullptr && src.T < 0) return DGQ_ERR_INVALID_ARG;
    if (src.bt != nullptr &&
        (src.num_blocks <= 0 || src.max_blocks <= 0 || (int64_t)max_seqlen > (int64_t)src.max_blocks * block_size ||
         !aligned16(src.bt)))
        return DGQ_ERR_INVALID_ARG;
    // flat window index and pool row index are 32-bit on the device
    const int64_t windows = (int64_t)batch * num_kv_heads * ((max_seqlen + DGQ_WINDOW - 1) / DGQ_WINDOW);
    if (windows >= INT32_MAX || (int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (!src.k || !src.v || !cu_seqlens_dev || !block_tables_dev || !k_pool || !v_pool || !seg_table)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(src.k) || !aligned16(src.v) || !aligned16(k_pool) || !aligned16(v_pool) ||
        !aligned16(seg_table) || !aligned16(cu_seqlens_dev) || !aligned16(block_tables_dev))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < dgq_compress_workspace_size(batch, max_seqlen, num_kv_heads))
        return DGQ_ERR_WORKSPACE;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e =
        max_seqlen <= dgq::cluster_compress_max_seqlen()
            ? dgq::launch_compress_cluster(src, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, block_size,
                                           block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks,
                                           seg_table, workspace, gs, stream)
            : dgq::launch_compress(src, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, block_size,
                                   block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table,
                                   workspace, gs, nsm, stream);
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

}  // namespace

dgq_status dgq_compress_ex(const void *k_bf16, const void *v_bf16, int32_t total_tokens,
                           const int32_t *cu_seqlens_dev, int32_t batch, int32_t max_seqlen, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                           int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                           dgq_seg_record *seg_table, void *workspace, size_t workspace_bytes,
                           const dgq_compress_options *options, void *cuda_stream)
{
    const dgq::SourceDesc src = {k_bf16, v_bf16, total_tokens, nullptr, 0, 0};
    return compress_impl(src, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, head_dim, block_size,
                         block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table, workspace,
                         workspace_bytes, options, cuda_stream);
}

dgq_status dgq_compress_paged(const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                              const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                              const int32_t *cu_seqlens_dev, int32_t batch, int32_t max_seqlen,
                              int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                              const int32_t *block_tables_dev, int32_t max_blocks_per_seq, uint8_t *k_pool,
                              uint8_t *v_pool, int32_t num_blocks, dgq_seg_record *seg_table, void *workspace,
                              size_t workspace_bytes, const dgq_compress_options *options, void *cuda_stream)
{
    if (!src_block_tables_dev) return DGQ_ERR_INVALID_ARG;
    const dgq::SourceDesc src = {k_src_bf16, v_src_bf16, 0, src_block_tables_dev, max_src_blocks_per_seq,
                                 num_src_blocks};
    return compress_impl(src, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, head_dim, block_size,
                         block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table, workspace,
                         workspace_bytes, options, cuda_stream);
}

size_t dgq_append_workspace_size(void) { return 256; }  // the workspace header alone

namespace {
dgq_status append_impl(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                       int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                       dgq_seg_record *seg_table, dgq_seg_record *v_seg_table, int32_t *flags, void *workspace,
                       size_t workspace_bytes, void *cuda_stream);
}  // namespace

dgq_status dgq_append_ex(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                         int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                         dgq_seg_record *seg_table, int32_t *resegment_flags, void *workspace,
                         size_t workspace_bytes, void *cuda_stream)
{
    if (resegment_flags && !aligned16(resegment_flags)) return DGQ_ERR_INVALID_ARG;
    return append_impl(k_new_bf16, v_new_bf16, batch, num_kv_heads, head_dim, block_size, block_tables_dev,
                       max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table, nullptr, resegment_flags,
                       workspace, workspace_bytes, cuda_stream);
}

dgq_status dgq_append(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, int32_t num_kv_heads,
                      int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                      int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                      dgq_seg_record *seg_table, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    return append_impl(k_new_bf16, v_new_bf16, batch, num_kv_heads, head_dim, block_size, block_tables_dev,
                       max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table, nullptr, nullptr, workspace,
                       workspace_bytes, cuda_stream);
}

dgq_status dgq_append_split(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                            int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                            dgq_seg_record *k_seg_table, dgq_seg_record *v_seg_table, void *workspace,
                            size_t workspace_bytes, void *cuda_stream)
{
    if (!v_seg_table || !aligned16(v_seg_table)) return DGQ_ERR_INVALID_ARG;
    return append_impl(k_new_bf16, v_new_bf16, batch, num_kv_heads, head_dim, block_size, block_tables_dev,
                       max_blocks_per_seq, k_pool, v_pool, num_blocks, k_seg_table, v_seg_table, nullptr,
                       workspace, workspace_bytes, cuda_stream);
}

namespace {
dgq_status append_impl(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                       int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                       dgq_seg_record *seg_table, dgq_seg_record *v_seg_table, int32_t *flags, void *workspace,
                       size_t workspace_bytes, void *cuda_stream)
{
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return DGQ_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX) return DGQ_ERR_UNSUPPORTED;
    if (!k_new_bf16 || !v_new_bf16 || !block_tables_dev || !k_pool || !v_pool || !seg_table)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(k_new_bf16) || !aligned16(v_new_bf16) || !aligned16(block_tables_dev) || !aligned16(k_pool) ||
        !aligned16(v_pool) || !aligned16(seg_table))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_append_workspace_size())
        return DGQ_ERR_WORKSPACE;
    const cudaError_t e = dgq::launch_append(k_new_bf16, v_new_bf16, batch, num_kv_heads, block_size,
                                             block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks,
                                             seg_table, v_seg_table, flags, workspace,
                                             static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}
}  // namespace

dgq_status dgq_fork_records(dgq_seg_record *seg_table, int32_t num_rows, int32_t num_kv_heads,
                            const int32_t *forks_dev, int32_t num_forks, void *workspace, size_t workspace_bytes,
                            void *cuda_stream)
{
    if (num_rows <= 0 || num_kv_heads <= 0 || num_forks < 0) return DGQ_ERR_INVALID_ARG;
    if ((int64_t)num_forks * num_kv_heads >= INT32_MAX) return DGQ_ERR_UNSUPPORTED;
    if (!seg_table || !aligned16(seg_table) || (num_forks > 0 && !forks_dev) || !aligned16(forks_dev))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_append_workspace_size())
        return DGQ_ERR_WORKSPACE;
    if (num_forks == 0) return DGQ_OK;
    const cudaError_t e = dgq::launch_fork_records(seg_table, num_rows, num_kv_heads, forks_dev, num_forks, workspace,
                                                   static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

size_t dgq_attn_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t max_seqlen)
{
    (void)max_seqlen;
    if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return 0;
    return dgq::attn_layout(batch, num_q_heads, num_kv_heads, nsm).total;
}

dgq_status dgq_paged_decode_attn(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                                 const uint8_t *k_pool, const uint8_t *v_pool, const dgq_seg_record *seg_table,
                                 const int32_t *block_tables_dev, const int32_t *seq_lens_dev, int32_t max_seqlen,
                                 int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int32_t max_blocks_per_seq, int32_t num_blocks, void *out_bf16,
                                 void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    return dgq_paged_decode_attn_format(DGQ_FORMAT_DGQ, q_bf16, k_new_bf16, v_new_bf16, k_pool, v_pool, seg_table,
                                        nullptr, nullptr, block_tables_dev, seq_lens_dev, max_seqlen, batch,
                                        num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                        num_blocks, out_bf16, workspace, workspace_bytes, cuda_stream);
}

namespace {
dgq_status attn_impl(int32_t format, const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                     const uint8_t *k_pool, const uint8_t *v_pool, const dgq_seg_record *seg_table,
                     const dgq_seg_record *v_seg_table, const float *k_group_params, const float *v_group_params,
                     const int32_t *block_tables_dev, const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t max_blocks_per_seq, int32_t num_blocks, void *out_bf16, void *workspace,
                     size_t workspace_bytes, void *cuda_stream, int32_t window = 0, int32_t sinks = 0);
}  // namespace

dgq_status dgq_paged_decode_attn_split(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                                       const uint8_t *k_pool, const uint8_t *v_pool, const dgq_seg_record *k_seg_table,
                                       const dgq_seg_record *v_seg_table, const int32_t *block_tables_dev,
                                       const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int32_t max_blocks_per_seq, int32_t num_blocks, void *out_bf16,
                                       void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!v_seg_table || !aligned16(v_seg_table)) return DGQ_ERR_INVALID_ARG;
    return attn_impl(DGQ_FORMAT_DGQ, q_bf16, k_new_bf16, v_new_bf16, k_pool, v_pool, k_seg_table, v_seg_table,
                     nullptr, nullptr, block_tables_dev, seq_lens_dev, max_seqlen, batch, num_q_heads, num_kv_heads,
                     head_dim, block_size, max_blocks_per_seq, num_blocks, out_bf16, workspace, workspace_bytes,
                     cuda_stream);
}

dgq_status dgq_paged_decode_attn_format(int32_t format, const void *q_bf16, const void *k_new_bf16,
                                        const void *v_new_bf16, const uint8_t *k_pool, const uint8_t *v_pool,
                                        const dgq_seg_record *seg_table, const float *k_group_params,
                                        const float *v_group_params, const int32_t *block_tables_dev,
                                        const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t block_size, int32_t max_blocks_per_seq, int32_t num_blocks,
                                        void *out_bf16, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (format != DGQ_FORMAT_DGQ && format != DGQ_FORMAT_FIXED64 && format != DGQ_FORMAT_SYM_INT8 &&
        format != DGQ_FORMAT_FP8_E4M3)
        return DGQ_ERR_INVALID_ARG;
    return attn_impl(format, q_bf16, k_new_bf16, v_new_bf16, k_pool, v_pool, seg_table, nullptr, k_group_params,
                     v_group_params, block_tables_dev, seq_lens_dev, max_seqlen, batch, num_q_heads, num_kv_heads,
                     head_dim, block_size, max_blocks_per_seq, num_blocks, out_bf16, workspace, workspace_bytes,
                     cuda_stream);
}

dgq_status dgq_paged_decode_attn_bf16(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                                      const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                                      const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                                      const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                                      int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                      int32_t block_size, void *out_bf16, void *workspace, size_t workspace_bytes,
                                      void *cuda_stream)
{
    return attn_impl(dgq::kFormatBf16Cache, q_bf16, k_new_bf16, v_new_bf16, static_cast<const uint8_t *>(k_src_bf16),
                     static_cast<const uint8_t *>(v_src_bf16), nullptr, nullptr, nullptr, nullptr,
                     src_block_tables_dev, seq_lens_dev, max_seqlen, batch, num_q_heads, num_kv_heads, head_dim,
                     block_size, max_src_blocks_per_seq, num_src_blocks, out_bf16, workspace, workspace_bytes,
                     cuda_stream);
}

dgq_status dgq_paged_decode_attn_window(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                                        const uint8_t *k_pool, const uint8_t *v_pool, const dgq_seg_record *seg_table,
                                        const int32_t *block_tables_dev, const int32_t *seq_lens_dev,
                                        int32_t max_seqlen, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t block_size, int32_t max_blocks_per_seq,
                                        int32_t num_blocks, int32_t window, int32_t sinks, void *out_bf16,
                                        void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!window_ok(window, sinks)) return DGQ_ERR_INVALID_ARG;
    return attn_impl(DGQ_FORMAT_DGQ, q_bf16, k_new_bf16, v_new_bf16, k_pool, v_pool, seg_table, nullptr, nullptr,
                     nullptr, block_tables_dev, seq_lens_dev, max_seqlen, batch, num_q_heads, num_kv_heads, head_dim,
                     block_size, max_blocks_per_seq, num_blocks, out_bf16, workspace, workspace_bytes, cuda_stream,
                     window, sinks);
}

dgq_status dgq_paged_decode_attn_bf16_window(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                                             const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                                             const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                                             const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                                             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                             int32_t block_size, int32_t window, int32_t sinks, void *out_bf16,
                                             void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!window_ok(window, sinks)) return DGQ_ERR_INVALID_ARG;
    return attn_impl(dgq::kFormatBf16Cache, q_bf16, k_new_bf16, v_new_bf16, static_cast<const uint8_t *>(k_src_bf16),
                     static_cast<const uint8_t *>(v_src_bf16), nullptr, nullptr, nullptr, nullptr,
                     src_block_tables_dev, seq_lens_dev, max_seqlen, batch, num_q_heads, num_kv_heads, head_dim,
                     block_size, max_src_blocks_per_seq, num_src_blocks, out_bf16, workspace, workspace_bytes,
                     cuda_stream, window, sinks);
}

dgq_status dgq_paged_decode_attn_block8(int32_t format, const void *q_bf16, const void *k_new_bf16,
                                        const void *v_new_bf16, const uint8_t *k_pool, const uint8_t *v_pool,
                                        const float *k_scales, const float *v_scales, const int32_t *block_tables_dev,
                                        const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t block_size, int32_t max_blocks_per_seq, int32_t num_blocks,
                                        int32_t window, int32_t sinks, void *out_bf16, void *workspace,
                                        size_t workspace_bytes, void *cuda_stream)
{
    if (format != DGQ_BLOCK8_INT8 && format != DGQ_BLOCK8_E4M3) return DGQ_ERR_INVALID_ARG;
    if (!(window == 0 && sinks == 0) && !window_ok(window, sinks)) return DGQ_ERR_INVALID_ARG;
    if (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)) return DGQ_ERR_INVALID_ARG;
    return attn_impl(format == DGQ_BLOCK8_E4M3 ? dgq::kFormatBlockE4m3 : dgq::kFormatBlockInt8, q_bf16, k_new_bf16,
                     v_new_bf16, k_pool, v_pool, nullptr, nullptr, k_scales, v_scales, block_tables_dev, seq_lens_dev,
                     max_seqlen, batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                     num_blocks, out_bf16, workspace, workspace_bytes, cuda_stream, window, sinks);
}

namespace {
dgq_status attn_impl(int32_t format, const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                     const uint8_t *k_pool, const uint8_t *v_pool, const dgq_seg_record *seg_table,
                     const dgq_seg_record *v_seg_table, const float *k_group_params, const float *v_group_params,
                     const int32_t *block_tables_dev, const int32_t *seq_lens_dev, int32_t max_seqlen, int32_t batch,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t max_blocks_per_seq, int32_t num_blocks, void *out_bf16, void *workspace,
                     size_t workspace_bytes, void *cuda_stream, int32_t window, int32_t sinks)
{
    if (format == DGQ_FORMAT_FIXED64 && (!k_group_params || !v_group_params || !aligned16(k_group_params) ||
                                         !aligned16(v_group_params)))
        return DGQ_ERR_INVALID_ARG;
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || max_seqlen < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq <= 0)
        return DGQ_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads) return DGQ_ERR_INVALID_ARG;
    const int32_t G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DGQ_ERR_UNSUPPORTED;
    if ((int64_t)max_seqlen > (int64_t)max_blocks_per_seq * block_size) return DGQ_ERR_INVALID_ARG;
    const int64_t chunks = (int64_t)batch * num_kv_heads * ((max_seqlen + 63) / 64 + 1);
    if (chunks >= INT32_MAX || (int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (!q_bf16 || !k_new_bf16 || !v_new_bf16 || !k_pool || !v_pool ||
        (!seg_table && format < dgq::kFormatBf16Cache) || !block_tables_dev || !seq_lens_dev || !out_bf16)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(q_bf16) || !aligned16(k_new_bf16) || !aligned16(v_new_bf16) || !aligned16(k_pool) ||
        !aligned16(v_pool) || !aligned16(seg_table) || !aligned16(out_bf16) || !aligned16(block_tables_dev) ||
        !aligned16(seq_lens_dev))
        return DGQ_ERR_INVALID_ARG;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < dgq::attn_layout(batch, num_q_heads, num_kv_heads, nsm).total)
        return DGQ_ERR_WORKSPACE;
    bool map_failed = false;
    cudaError_t e = dgq::launch_attn(format, q_bf16, k_new_bf16, v_new_bf16, k_pool, v_pool, seg_table,
                                     v_seg_table, k_group_params, v_group_params, block_tables_dev, seq_lens_dev,
                                     max_seqlen, batch, num_q_heads, num_kv_heads, block_size, max_blocks_per_seq,
                                     num_blocks, held(window), held(sinks), out_bf16, workspace, nsm, &map_failed,
                                     static_cast<cudaStream_t>(cuda_stream));
    if (map_failed) return DGQ_ERR_INVALID_ARG;
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}
}  // namespace

size_t dgq_prefill_workspace_size(int32_t batch, int32_t num_kv_heads)
{
    if (batch <= 0 || num_kv_heads <= 0) return 0;
    return dgq::prefill_workspace_bytes(batch, num_kv_heads);
}

namespace {

// Checks shared by the two prefill calls (source, sizes, statistics array, workspace).
dgq_status prefill_checks(const void *k_src, const void *v_src, int32_t num_src_blocks, const int32_t *src_bt,
                          int32_t max_src_blocks, int32_t batch, int32_t max_seqlen, int32_t num_kv_heads,
                          int32_t head_dim, int32_t block_size, const void *stats, int32_t max_windows,
                          const void *workspace, size_t workspace_bytes)
{
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || max_seqlen < 0 || num_kv_heads <= 0 || num_src_blocks <= 0 ||
        max_src_blocks <= 0)
        return DGQ_ERR_INVALID_ARG;
    if ((int64_t)max_seqlen > (int64_t)max_src_blocks * block_size) return DGQ_ERR_INVALID_ARG;
    if (max_windows < (max_seqlen + DGQ_WINDOW - 1) / DGQ_WINDOW || max_windows <= 0) return DGQ_ERR_INVALID_ARG;
    const int64_t windows = (int64_t)batch * num_kv_heads * max_windows;
    if (windows >= INT32_MAX || (int64_t)num_src_blocks * num_kv_heads * block_size >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (!k_src || !v_src || !src_bt || !stats) return DGQ_ERR_INVALID_ARG;
    if (!aligned16(k_src) || !aligned16(v_src) || !aligned16(src_bt) || !aligned16(stats))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq::prefill_workspace_bytes(batch, num_kv_heads))
        return DGQ_ERR_WORKSPACE;
    return DGQ_OK;
}

}  // namespace

dgq_status dgq_prefill_chunk_stats(const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                                   const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                                   const int32_t *chunk_begin_dev, const int32_t *chunk_end_dev, int32_t batch,
                                   int32_t max_seqlen, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   float *window_stats, int32_t max_windows, int32_t flags, void *workspace,
                                   size_t workspace_bytes, void *cuda_stream)
{
    if (flags & ~DGQ_PREFILL_V_VARIANCE) return DGQ_ERR_INVALID_ARG;
    dgq_status st = prefill_checks(k_src_bf16, v_src_bf16, num_src_blocks, src_block_tables_dev,
                                   max_src_blocks_per_seq, batch, max_seqlen, num_kv_heads, head_dim, block_size,
                                   window_stats, max_windows, workspace, workspace_bytes);
    if (st != DGQ_OK) return st;
    if (!chunk_begin_dev || !chunk_end_dev || !aligned16(chunk_begin_dev) || !aligned16(chunk_end_dev))
        return DGQ_ERR_INVALID_ARG;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const dgq::SourceDesc src = {k_src_bf16, v_src_bf16, 0, src_block_tables_dev, max_src_blocks_per_seq,
                                 num_src_blocks};
    bool map_failed = false;
    const cudaError_t e = dgq::launch_prefill_stats(src, chunk_begin_dev, chunk_end_dev, batch, max_seqlen,
                                                    num_kv_heads, block_size, window_stats, max_windows,
                                                    (flags & DGQ_PREFILL_V_VARIANCE) != 0, workspace, nsm,
                                                    &map_failed, static_cast<cudaStream_t>(cuda_stream));
    if (map_failed) return DGQ_ERR_INVALID_ARG;
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

dgq_status dgq_prefill_finish(const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                              const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                              const int32_t *seq_lens_dev, int32_t batch, int32_t max_seqlen, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, const float *window_stats, int32_t max_windows,
                              const int32_t *block_tables_dev, int32_t max_blocks_per_seq, uint8_t *k_pool,
                              uint8_t *v_pool, int32_t num_blocks, dgq_seg_record *seg_table,
                              dgq_seg_record *v_seg_table, const dgq_compress_options *options, void *workspace,
                              size_t workspace_bytes, void *cuda_stream)
{
    return dgq_prefill_finish_ex(k_src_bf16, v_src_bf16, num_src_blocks, src_block_tables_dev,
                                 max_src_blocks_per_seq, seq_lens_dev, batch, max_seqlen, num_kv_heads, head_dim,
                                 block_size, window_stats, max_windows, block_tables_dev, max_blocks_per_seq, k_pool,
                                 v_pool, num_blocks, seg_table, v_seg_table, options, nullptr, 0, workspace,
                                 workspace_bytes, cuda_stream);
}

dgq_status dgq_prefill_finish_ex(const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                                 const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                                 const int32_t *seq_lens_dev, int32_t batch, int32_t max_seqlen,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 const float *window_stats, int32_t max_windows, const int32_t *block_tables_dev,
                                 int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                                 dgq_seg_record *seg_table, dgq_seg_record *v_seg_table,
                                 const dgq_compress_options *options, const int32_t *pair_flags,
                                 int32_t flag_mask, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (v_seg_table && !aligned16(v_seg_table)) return DGQ_ERR_INVALID_ARG;
    if (pair_flags && !aligned16(pair_flags)) return DGQ_ERR_INVALID_ARG;
    dgq::GroupSettings gs = {DGQ_MAX_SEG, 0.0f};
    if (options) {
        if (options->max_groups < 1 || options->max_groups > DGQ_MAX_SEG || !(options->min_var >= 0.0f) ||
            !(options->min_var <= 3.4e38f))
            return DGQ_ERR_INVALID_ARG;
        gs.max_groups = options->max_groups;
        gs.min_var = options->min_var;
    }
    dgq_status st = prefill_checks(k_src_bf16, v_src_bf16, num_src_blocks, src_block_tables_dev,
                                   max_src_blocks_per_seq, batch, max_seqlen, num_kv_heads, head_dim, block_size,
                                   window_stats, max_windows, workspace, workspace_bytes);
    if (st != DGQ_OK) return st;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0 ||
        (int64_t)max_seqlen > (int64_t)max_blocks_per_seq * block_size ||
        (int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX)
        return DGQ_ERR_INVALID_ARG;
    if (!seq_lens_dev || !block_tables_dev || !k_pool || !v_pool || !seg_table) return DGQ_ERR_INVALID_ARG;
    if (!aligned16(seq_lens_dev) || !aligned16(block_tables_dev) || !aligned16(k_pool) || !aligned16(v_pool) ||
        !aligned16(seg_table))
        return DGQ_ERR_INVALID_ARG;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const dgq::SourceDesc src = {k_src_bf16, v_src_bf16, 0, src_block_tables_dev, max_src_blocks_per_seq,
                                 num_src_blocks};
    bool map_failed = false;
    const cudaError_t e = dgq::launch_prefill_finish(
        src, seq_lens_dev, batch, max_seqlen, num_kv_heads, block_size, window_stats, max_windows, block_tables_dev,
        max_blocks_per_seq, k_pool, v_pool, num_blocks, seg_table, v_seg_table, gs, pair_flags, flag_mask,
        workspace, nsm, &map_failed, static_cast<cudaStream_t>(cuda_stream));
    if (map_failed) return DGQ_ERR_INVALID_ARG;
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

size_t dgq_encode_format_workspace_size(int32_t batch, int32_t num_kv_heads)
{
    if (batch <= 0 || num_kv_heads <= 0) return 0;
    return dgq::format_workspace_bytes(batch, num_kv_heads);
}

dgq_status dgq_encode_format(int32_t format, const void *k_bf16, const void *v_bf16, int32_t total_tokens,
                             const int32_t *cu_seqlens_dev, int32_t batch, int32_t max_seqlen, int32_t num_kv_heads,
                             int32_t head_dim, int32_t block_size, const int32_t *block_tables_dev,
                             int32_t max_blocks_per_seq, uint8_t *k_pool, uint8_t *v_pool, int32_t num_blocks,
                             dgq_seg_record *seg_table, float *k_group_params, float *v_group_params,
                             void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (format != DGQ_FORMAT_FIXED64 && format != DGQ_FORMAT_SYM_INT8 && format != DGQ_FORMAT_FP8_E4M3)
        return DGQ_ERR_INVALID_ARG;
    if (format == DGQ_FORMAT_FIXED64 && (!k_group_params || !v_group_params || !aligned16(k_group_params) ||
                                         !aligned16(v_group_params)))
        return DGQ_ERR_INVALID_ARG;
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || max_seqlen < 0 || total_tokens < 0 || num_kv_heads <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq <= 0)
        return DGQ_ERR_INVALID_ARG;
    if ((int64_t)max_seqlen > (int64_t)max_blocks_per_seq * block_size) return DGQ_ERR_INVALID_ARG;
    // grid: one CTA column per (request, head) pair, one row per 256 tokens
    if ((int64_t)batch * num_kv_heads >= INT32_MAX || (max_seqlen + 255) / 256 > 65535 ||
        (int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (!k_bf16 || !v_bf16 || !cu_seqlens_dev || !block_tables_dev || !k_pool || !v_pool || !seg_table)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(k_bf16) || !aligned16(v_bf16) || !aligned16(k_pool) || !aligned16(v_pool) ||
        !aligned16(seg_table) || !aligned16(cu_seqlens_dev) || !aligned16(block_tables_dev))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq::format_workspace_bytes(batch, num_kv_heads))
        return DGQ_ERR_WORKSPACE;
    const cudaError_t e = dgq::launch_format_encode(
        format, k_bf16, v_bf16, total_tokens, cu_seqlens_dev, batch, max_seqlen, num_kv_heads, block_size,
        block_tables_dev, max_blocks_per_seq, k_pool, v_pool, num_blocks, k_group_params, v_group_params, seg_table,
        workspace, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

dgq_status dgq_workspace_init(void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!workspace || workspace_bytes == 0) return DGQ_ERR_INVALID_ARG;
    cudaError_t e = cudaMemsetAsync(workspace, 0, workspace_bytes, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

dgq_status dgq_workspace_error(const void *workspace, void *cuda_stream, int32_t *device_error)
{
    if (!workspace || !device_error) return DGQ_ERR_INVALID_ARG;
    uint32_t word = 0;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return DGQ_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return DGQ_ERR_CUDA;
    *device_error = (int32_t)word;
    return word ? DGQ_ERR_DEVICE : DGQ_OK;
}

// ---- prompt attention -------------------------------------------------------------------

size_t dgq_prompt_attn_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads)
{
    if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return 0;
    return dgq::prompt_workspace_bytes(batch, num_q_heads, num_kv_heads, nsm);
}

namespace {
// Checks and launch shared by the packed and the paged entry point (bt null: packed).
dgq_status prompt_impl(const void *q, const void *k, const void *v, int32_t total_q, int32_t total_kv,
                       const int32_t *cu_q, const int32_t *kv, bool paged, const int32_t *bt, int32_t block_size,
                       int32_t max_blocks, int32_t num_blocks, int32_t batch, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, void *out, void *workspace, size_t workspace_bytes,
                       void *cuda_stream, int32_t window = 0, int32_t sinks = 0)
{
    if (head_dim != DGQ_HEAD_DIM || (paged && !block_size_ok(block_size))) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || total_q < 0 || total_kv < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads)
        return DGQ_ERR_INVALID_ARG;
    const int32_t G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DGQ_ERR_UNSUPPORTED;
    // rows of all heads are counted in 32 bits, and a request's keys stay below 2^30
    if ((int64_t)total_q * num_q_heads >= INT32_MAX || (int64_t)total_kv * num_kv_heads >= INT32_MAX ||
        total_q > (1 << 30) || total_kv > (1 << 30))
        return DGQ_ERR_UNSUPPORTED;
    if (paged) {
        if (num_blocks <= 0 || max_blocks <= 0 || !bt || !aligned16(bt)) return DGQ_ERR_INVALID_ARG;
        if ((int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX ||
            (int64_t)max_blocks * block_size > (1 << 30))
            return DGQ_ERR_UNSUPPORTED;
    }
    // an empty buffer has no address
    if ((!q && total_q) || (!out && total_q) || ((!k || !v) && (paged || total_kv)) || !cu_q || !kv)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(cu_q) || !aligned16(kv))
        return DGQ_ERR_INVALID_ARG;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < dgq::prompt_workspace_bytes(batch, num_q_heads, num_kv_heads, nsm))
        return DGQ_ERR_WORKSPACE;
    if (total_q == 0) return DGQ_OK;
    bool map_failed = false;
    const cudaError_t e = dgq::launch_prompt(q, k, v, total_q, total_kv, cu_q, kv, paged ? bt : nullptr, block_size,
                                             max_blocks, num_blocks, batch, num_q_heads, num_kv_heads, held(window),
                                             held(sinks), out, workspace, nsm, &map_failed, static_cast<cudaStream_t>(cuda_stream));
    if (map_failed) return DGQ_ERR_INVALID_ARG;
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}
}  // namespace

dgq_status dgq_prompt_attn(const void *q_bf16, const void *k_bf16, const void *v_bf16, int32_t total_q,
                           int32_t total_kv, const int32_t *cu_q_dev, const int32_t *cu_kv_dev, int32_t batch,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void *out_bf16,
                           void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    return prompt_impl(q_bf16, k_bf16, v_bf16, total_q, total_kv, cu_q_dev, cu_kv_dev, false, nullptr, 0, 0, 0, batch,
                       num_q_heads, num_kv_heads, head_dim, out_bf16, workspace, workspace_bytes, cuda_stream);
}

dgq_status dgq_prompt_attn_paged(const void *q_bf16, int32_t total_q, const int32_t *cu_q_dev, const void *k_src_bf16,
                                 const void *v_src_bf16, int32_t num_src_blocks, const int32_t *src_block_tables_dev,
                                 int32_t max_src_blocks_per_seq, const int32_t *seq_lens_dev, int32_t batch,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 void *out_bf16, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    return prompt_impl(q_bf16, k_src_bf16, v_src_bf16, total_q, 0, cu_q_dev, seq_lens_dev, true, src_block_tables_dev,
                       block_size, max_src_blocks_per_seq, num_src_blocks, batch, num_q_heads, num_kv_heads, head_dim,
                       out_bf16, workspace, workspace_bytes, cuda_stream);
}

dgq_status dgq_prompt_attn_window(const void *q_bf16, const void *k_bf16, const void *v_bf16, int32_t total_q,
                                  int32_t total_kv, const int32_t *cu_q_dev, const int32_t *cu_kv_dev, int32_t batch,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t window,
                                  int32_t sinks, void *out_bf16, void *workspace, size_t workspace_bytes,
                                  void *cuda_stream)
{
    if (!window_ok(window, sinks)) return DGQ_ERR_INVALID_ARG;
    return prompt_impl(q_bf16, k_bf16, v_bf16, total_q, total_kv, cu_q_dev, cu_kv_dev, false, nullptr, 0, 0, 0, batch,
                       num_q_heads, num_kv_heads, head_dim, out_bf16, workspace, workspace_bytes, cuda_stream, window,
                       sinks);
}

dgq_status dgq_prompt_attn_paged_window(const void *q_bf16, int32_t total_q, const int32_t *cu_q_dev,
                                        const void *k_src_bf16, const void *v_src_bf16, int32_t num_src_blocks,
                                        const int32_t *src_block_tables_dev, int32_t max_src_blocks_per_seq,
                                        const int32_t *seq_lens_dev, int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t window,
                                        int32_t sinks, void *out_bf16, void *workspace, size_t workspace_bytes,
                                        void *cuda_stream)
{
    if (!window_ok(window, sinks)) return DGQ_ERR_INVALID_ARG;
    return prompt_impl(q_bf16, k_src_bf16, v_src_bf16, total_q, 0, cu_q_dev, seq_lens_dev, true, src_block_tables_dev,
                       block_size, max_src_blocks_per_seq, num_src_blocks, batch, num_q_heads, num_kv_heads, head_dim,
                       out_bf16, workspace, workspace_bytes, cuda_stream, window, sinks);
}

// ---- tables from lengths, rows by slot ----------------------------------------------------

size_t dgq_extend_tables_workspace_size(void) { return 256; }  // the workspace header alone

dgq_status dgq_extend_tables(const int32_t *seq_lens_dev, const int32_t *new_lens_dev, int32_t batch,
                             int32_t block_size, int32_t num_blocks, const int32_t *free_ids_dev, int32_t num_free,
                             const int32_t *free_used_dev, int32_t *block_tables_dev, int32_t max_blocks_per_seq,
                             int32_t *slots_dev, int32_t total_slots, int32_t *cu_new_dev, int32_t *seq_lens_out_dev,
                             int32_t *free_used_out_dev, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || num_blocks <= 0 || max_blocks_per_seq <= 0 || num_free < 0 || total_slots < 0)
        return DGQ_ERR_INVALID_ARG;
    // slots, and the positions of a request, are 32-bit
    if ((int64_t)num_blocks * block_size >= INT32_MAX || (int64_t)max_blocks_per_seq * block_size > (1 << 30))
        return DGQ_ERR_UNSUPPORTED;
    // an empty buffer has no address
    if (!seq_lens_dev || !new_lens_dev || (num_free > 0 && !free_ids_dev) || !free_used_dev || !block_tables_dev ||
        (total_slots > 0 && !slots_dev) || !cu_new_dev || !seq_lens_out_dev || !free_used_out_dev)
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(seq_lens_dev) || !aligned16(new_lens_dev) || !aligned16(free_ids_dev) || !aligned16(free_used_dev) ||
        !aligned16(block_tables_dev) || !aligned16(slots_dev) || !aligned16(cu_new_dev) ||
        !aligned16(seq_lens_out_dev) || !aligned16(free_used_out_dev))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_extend_tables_workspace_size())
        return DGQ_ERR_WORKSPACE;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const dgq::ExtendArgs a = {seq_lens_dev,     new_lens_dev, free_ids_dev,       free_used_dev, block_tables_dev,
                               slots_dev,        cu_new_dev,   seq_lens_out_dev,   free_used_out_dev, batch,
                               block_size,       max_blocks_per_seq, num_blocks,   num_free,      total_slots};
    const cudaError_t e = dgq::launch_extend_tables(a, workspace, nsm, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

namespace {
// Checks of rows that are written by slot (T tokens, k_stride and v_stride elements apart).
dgq_status rows_checks(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int32_t T, int32_t num_kv_heads,
                       int32_t head_dim, const int32_t *slots, const void *k_pool, const void *v_pool,
                       int32_t num_blocks, int32_t block_size, const void *workspace, size_t workspace_bytes)
{
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (T < 0 || num_kv_heads <= 0 || num_blocks <= 0) return DGQ_ERR_INVALID_ARG;
    // rows in the pools, and 16-byte vectors of the tokens, are counted in 32 bits
    if ((int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX || (int64_t)T * num_kv_heads * 16 >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (T > 1 && (k_stride < (int64_t)num_kv_heads * DGQ_HEAD_DIM || v_stride < (int64_t)num_kv_heads * DGQ_HEAD_DIM ||
                  (k_stride & 7) || (v_stride & 7)))
        return DGQ_ERR_INVALID_ARG;
    if ((T > 0 && (!k || !v || !slots)) || !k_pool || !v_pool) return DGQ_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots) || !aligned16(k_pool) || !aligned16(v_pool))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < 256) return DGQ_ERR_WORKSPACE;
    return DGQ_OK;
}
}  // namespace

dgq_status dgq_write_slots(const void *k_bf16, const void *v_bf16, int64_t k_token_stride, int64_t v_token_stride,
                           int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, const int32_t *slots_dev,
                           void *k_pages_bf16, void *v_pages_bf16, int32_t num_blocks, int32_t block_size,
                           void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    const dgq_status st = rows_checks(k_bf16, v_bf16, k_token_stride, v_token_stride, num_tokens, num_kv_heads, head_dim,
                                      slots_dev, k_pages_bf16, v_pages_bf16, num_blocks, block_size, workspace,
                                      workspace_bytes);
    if (st != DGQ_OK || num_tokens == 0) return st;
    const cudaError_t e = dgq::launch_write_slots(k_bf16, v_bf16, k_token_stride, v_token_stride, num_tokens,
                                                  num_kv_heads, block_size, slots_dev, k_pages_bf16, v_pages_bf16,
                                                  num_blocks, workspace, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

// ---- 8-bit cache with a scale per block and head ------------------------------------------

size_t dgq_block8_workspace_size(void) { return 256; }  // the workspace header alone

dgq_status dgq_store_block8(int32_t format, const void *k_bf16, const void *v_bf16, int64_t k_token_stride,
                            int64_t v_token_stride, int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                            const int32_t *slots_dev, uint8_t *k_pool, uint8_t *v_pool, float *k_scales,
                            float *v_scales, int32_t num_blocks, int32_t block_size, void *workspace,
                            size_t workspace_bytes, void *cuda_stream)
{
    if (format != DGQ_BLOCK8_INT8 && format != DGQ_BLOCK8_E4M3) return DGQ_ERR_INVALID_ARG;
    const dgq_status st = rows_checks(k_bf16, v_bf16, k_token_stride, v_token_stride, num_tokens, num_kv_heads, head_dim,
                                      slots_dev, k_pool, v_pool, num_blocks, block_size, workspace, workspace_bytes);
    if (st != DGQ_OK) return st;
    if (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)) return DGQ_ERR_INVALID_ARG;
    if (num_tokens == 0) return DGQ_OK;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const cudaError_t e = dgq::launch_store_block8(
        format == DGQ_BLOCK8_E4M3, k_bf16, v_bf16, k_token_stride, v_token_stride, num_tokens, num_kv_heads, block_size,
        slots_dev, k_pool, v_pool, k_scales, v_scales, num_blocks, workspace, nsm, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

dgq_status dgq_load_block8(int32_t format, const uint8_t *k_pool, const uint8_t *v_pool, const float *k_scales,
                           const float *v_scales, int32_t num_blocks, int32_t block_size,
                           const int32_t *block_tables_dev, int32_t max_blocks_per_seq, const int32_t *cu_kv_dev,
                           int32_t batch, int32_t num_kv_heads, int32_t head_dim, void *k_bf16, void *v_bf16,
                           int32_t total_kv, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (format != DGQ_BLOCK8_INT8 && format != DGQ_BLOCK8_E4M3) return DGQ_ERR_INVALID_ARG;
    if (head_dim != DGQ_HEAD_DIM || !block_size_ok(block_size)) return DGQ_ERR_UNSUPPORTED;
    if (batch <= 0 || batch > kMaxBatch || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || total_kv < 0)
        return DGQ_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= INT32_MAX || (int64_t)total_kv * num_kv_heads >= INT32_MAX)
        return DGQ_ERR_UNSUPPORTED;
    if (!k_pool || !v_pool || !k_scales || !v_scales || !block_tables_dev || !cu_kv_dev ||
        (total_kv > 0 && (!k_bf16 || !v_bf16)))
        return DGQ_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_scales) || !aligned16(v_scales) ||
        !aligned16(block_tables_dev) || !aligned16(cu_kv_dev) || !aligned16(k_bf16) || !aligned16(v_bf16))
        return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_block8_workspace_size()) return DGQ_ERR_WORKSPACE;
    if (total_kv == 0) return DGQ_OK;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const cudaError_t e = dgq::launch_load_block8(
        format == DGQ_BLOCK8_E4M3, k_pool, v_pool, k_scales, v_scales, num_blocks, block_tables_dev, max_blocks_per_seq,
        cu_kv_dev, batch, num_kv_heads, block_size, k_bf16, v_bf16, total_kv, workspace, nsm,
        static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

// ---- pages ------------------------------------------------------------------------------

size_t dgq_copy_pages_workspace_size(void) { return 256; }  // the workspace header alone

dgq_status dgq_copy_pages(void *const *arrays, int32_t num_arrays, int64_t page_bytes, int32_t num_pages,
                          const int32_t *pairs_dev, int32_t num_pairs, void *workspace, size_t workspace_bytes,
                          void *cuda_stream)
{
    if (num_arrays < 0 || num_pairs < 0 || page_bytes <= 0 || (page_bytes & 15) || num_pages <= 0)
        return DGQ_ERR_INVALID_ARG;
    // units of 4 KB in a page are counted in 32 bits, bytes of an array and units of a call in 64
    if (page_bytes > ((int64_t)1 << 40) || page_bytes > INT64_MAX / num_pages ||
        (int64_t)num_pairs > ((int64_t)1 << 50) / (page_bytes / 4096 + 1))
        return DGQ_ERR_UNSUPPORTED;
    if ((num_arrays > 0 && !arrays) || (num_pairs > 0 && !pairs_dev) || !aligned16(pairs_dev))
        return DGQ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num_arrays; ++i)
        if (!arrays[i] || !aligned16(arrays[i])) return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_copy_pages_workspace_size())
        return DGQ_ERR_WORKSPACE;
    if (num_arrays == 0 || num_pairs == 0) return DGQ_OK;
    const cudaError_t e = dgq::launch_copy_pages(arrays, num_arrays, page_bytes, num_pages, pairs_dev, num_pairs,
                                                 workspace, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

dgq_status dgq_remap_tables(const int32_t *tables_dev, int64_t num_entries, const int32_t *remap_dev,
                            int32_t num_pages, int32_t *out_dev, void *workspace, size_t workspace_bytes,
                            void *cuda_stream)
{
    if (num_entries < 0 || num_pages <= 0) return DGQ_ERR_INVALID_ARG;
    if (num_entries > 0 && (!tables_dev || !remap_dev || !out_dev)) return DGQ_ERR_INVALID_ARG;
    if (!aligned16(tables_dev) || !aligned16(remap_dev) || !aligned16(out_dev)) return DGQ_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < dgq_copy_pages_workspace_size())
        return DGQ_ERR_WORKSPACE;
    if (num_entries == 0) return DGQ_OK;
    int nsm = 0;
    if (device_sm_count(&nsm) != 0) return DGQ_ERR_CUDA;
    const cudaError_t e = dgq::launch_remap_tables(tables_dev, num_entries, remap_dev, num_pages, out_dev, workspace,
                                                   nsm, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? DGQ_OK : DGQ_ERR_CUDA;
}

// ---- host block pool --------------------------------------------------------------------

// A block is free (no reference) or held by one reference per table row (or caller) that names it.
// All storage is taken at creation, so no later call allocates or throws.
struct dgq_pool {
    int32_t num_blocks;
    std::vector<int32_t> free_list;  // stack of free ids, capacity num_blocks
    std::vector<int32_t> refs;       // references per block, 0 when free
    std::vector<uint8_t> mark;       // all 0 between calls
};

dgq_pool *dgq_pool_create(int32_t num_blocks)
{
    if (num_blocks <= 0) return nullptr;
    dgq_pool *p = new (std::nothrow) dgq_pool;
    if (!p) return nullptr;
    try {
        p->num_blocks = num_blocks;
        p->free_list.resize(num_blocks);
        p->refs.assign(num_blocks, 0);
        p->mark.assign(num_blocks, 0);
    } catch (...) {  // (no exception leaves a C entry)
        delete p;
        return nullptr;
    }
    for (int32_t i = 0; i < num_blocks; ++i) p->free_list[i] = num_blocks - 1 - i;  // pops 0, 1, 2, ...
    return p;
}

void dgq_pool_destroy(dgq_pool *pool) { delete pool; }

namespace {

bool pool_live(const dgq_pool *pool, int32_t id) { return id >= 0 && id < pool->num_blocks && pool->refs[id] > 0; }

int32_t pool_take(dgq_pool *pool)  // one free block, its first reference (the list is not empty)
{
    const int32_t id = pool->free_list.back();
    pool->free_list.pop_back();
    pool->refs[id] = 1;
    return id;
}

// Every id live and none named twice.
bool pool_ids_ok(dgq_pool *pool, const int32_t *ids, int32_t n)
{
    int32_t i = 0;
    bool ok = true;
    for (; i < n && ok; ++i) {
        if (!pool_live(pool, ids[i]) || pool->mark[ids[i]]) {
            ok = false;
            break;
        }
        pool->mark[ids[i]] = 1;
    }
    for (int32_t j = 0; j < i; ++j) pool->mark[ids[j]] = 0;
    return ok;
}

}  // namespace

dgq_status dgq_pool_alloc(dgq_pool *pool, int32_t n, int32_t *out_ids)
{
    if (!pool || n < 0 || (n > 0 && !out_ids)) return DGQ_ERR_INVALID_ARG;
    if ((size_t)n > pool->free_list.size()) return DGQ_ERR_POOL_EXHAUSTED;
    for (int32_t i = 0; i < n; ++i) out_ids[i] = pool_take(pool);
    return DGQ_OK;
}

dgq_status dgq_pool_free(dgq_pool *pool, const int32_t *ids, int32_t n)
{
    if (!pool || n < 0 || (n > 0 && !ids)) return DGQ_ERR_INVALID_ARG;
    if (!pool_ids_ok(pool, ids, n)) return DGQ_ERR_INVALID_ARG;  // validated first: nothing is freed on error
    for (int32_t i = 0; i < n; ++i)
        if (--pool->refs[ids[i]] == 0) pool->free_list.push_back(ids[i]);
    return DGQ_OK;
}

dgq_status dgq_pool_share(dgq_pool *pool, const int32_t *ids, int32_t n)
{
    if (!pool || n < 0 || (n > 0 && !ids)) return DGQ_ERR_INVALID_ARG;
    if (!pool_ids_ok(pool, ids, n)) return DGQ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i)
        if (pool->refs[ids[i]] == INT32_MAX) return DGQ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) ++pool->refs[ids[i]];
    return DGQ_OK;
}

int32_t dgq_pool_num_free(const dgq_pool *pool) { return pool ? (int32_t)pool->free_list.size() : -1; }

int32_t dgq_pool_references(const dgq_pool *pool, int32_t id)
{
    return pool && id >= 0 && id < pool->num_blocks ? pool->refs[id] : -1;
}

dgq_status dgq_pool_alloc_table_row(dgq_pool *pool, int32_t len, int32_t block_size, int32_t *table, int32_t row,
                                    int32_t max_blocks_per_seq)
{
    if (!pool || !table || len < 0 || row < 0 || max_blocks_per_seq <= 0 || block_size <= 0)
        return DGQ_ERR_INVALID_ARG;
    const int32_t n = (int32_t)(((int64_t)len + block_size - 1) / block_size);
    if (n > max_blocks_per_seq) return DGQ_ERR_INVALID_ARG;
    int32_t *dst = table + (int64_t)row * max_blocks_per_seq;
    dgq_status s = dgq_pool_alloc(pool, n, dst);
    if (s != DGQ_OK) return s;
    for (int32_t i = n; i < max_blocks_per_seq; ++i) dst[i] = 0;
    return DGQ_OK;
}

dgq_status dgq_pool_fork_row(dgq_pool *pool, int32_t len, int32_t block_size, int32_t *table, int32_t src_row,
                             int32_t dst_row, int32_t max_blocks_per_seq, int32_t *out_pair, int32_t *num_pairs)
{
    if (!pool || !table || !out_pair || !num_pairs || len < 0 || src_row < 0 || dst_row < 0 || src_row == dst_row ||
        max_blocks_per_seq <= 0 || block_size <= 0)
        return DGQ_ERR_INVALID_ARG;
    const int32_t n = (int32_t)(((int64_t)len + block_size - 1) / block_size), whole = len / block_size;
    if (n > max_blocks_per_seq) return DGQ_ERR_INVALID_ARG;
    const int32_t *src = table + (int64_t)src_row * max_blocks_per_seq;
    int32_t *dst = table + (int64_t)dst_row * max_blocks_per_seq;
    if (!pool_ids_ok(pool, src, n)) return DGQ_ERR_INVALID_ARG;
    if (n > whole && pool->free_list.empty()) return DGQ_ERR_POOL_EXHAUSTED;
    const dgq_status s = dgq_pool_share(pool, src, whole);
    if (s != DGQ_OK) return s;
    for (int32_t i = 0; i < whole; ++i) dst[i] = src[i];
    *num_pairs = 0;
    if (n > whole) {
        out_pair[0] = src[whole];
        out_pair[1] = dst[whole] = pool_take(pool);
        *num_pairs = 1;
    }
    for (int32_t i = n; i < max_blocks_per_seq; ++i) dst[i] = 0;
    return DGQ_OK;
}

dgq_status dgq_pool_own_row(dgq_pool *pool, int32_t *table, int32_t row, int32_t max_blocks_per_seq,
                            int32_t first_block, int32_t num_row_blocks, int32_t *out_pairs, int32_t *num_pairs)
{
    if (!pool || !table || !num_pairs || row < 0 || max_blocks_per_seq <= 0 || first_block < 0 ||
        num_row_blocks < 0 || first_block > max_blocks_per_seq - num_row_blocks || (num_row_blocks > 0 && !out_pairs))
        return DGQ_ERR_INVALID_ARG;
    int32_t *ids = table + (int64_t)row * max_blocks_per_seq + first_block;
    if (!pool_ids_ok(pool, ids, num_row_blocks)) return DGQ_ERR_INVALID_ARG;
    int32_t shared = 0;
    for (int32_t i = 0; i < num_row_blocks; ++i) shared += pool->refs[ids[i]] > 1;
    if ((size_t)shared > pool->free_list.size()) return DGQ_ERR_POOL_EXHAUSTED;
    int32_t n = 0;
    for (int32_t i = 0; i < num_row_blocks; ++i) {
        if (pool->refs[ids[i]] == 1) continue;
        const int32_t id = pool_take(pool);
        out_pairs[2 * n] = ids[i];
        out_pairs[2 * n + 1] = id;
        ++n;
        --pool->refs[ids[i]];
        ids[i] = id;
    }
    *num_pairs = n;
    return DGQ_OK;
}

dgq_status dgq_pool_free_row(dgq_pool *pool, int32_t *table, int32_t row, int32_t max_blocks_per_seq,
                             int32_t num_row_blocks)
{
    if (!pool || !table || row < 0 || max_blocks_per_seq <= 0 || num_row_blocks < 0 ||
        num_row_blocks > max_blocks_per_seq)
        return DGQ_ERR_INVALID_ARG;
    int32_t *ids = table + (int64_t)row * max_blocks_per_seq;
    const dgq_status s = dgq_pool_free(pool, ids, num_row_blocks);
    if (s != DGQ_OK) return s;
    for (int32_t i = 0; i < max_blocks_per_seq; ++i) ids[i] = 0;
    return DGQ_OK;
}

dgq_status dgq_pool_compact(dgq_pool *pool, int32_t *remap, int32_t *out_pairs, int32_t *num_pairs)
{
    if (!pool || !remap || !num_pairs || (pool->num_blocks > 1 && !out_pairs)) return DGQ_ERR_INVALID_ARG;
    const int32_t live = pool->num_blocks - (int32_t)pool->free_list.size();
    int32_t n = 0, hole = 0;
    for (int32_t id = 0; id < pool->num_blocks; ++id) remap[id] = id;
    for (int32_t id = live; id < pool->num_blocks; ++id) {  // ascending ids into ascending holes
        if (pool->refs[id] == 0) continue;
        while (pool->refs[hole] != 0) ++hole;
        out_pairs[2 * n] = id;
        out_pairs[2 * n + 1] = hole;
        ++n;
        remap[id] = hole;
        pool->refs[hole] = pool->refs[id];
        pool->refs[id] = 0;
    }
    for (int32_t i = 0; i < pool->num_blocks - live; ++i) pool->free_list[i] = pool->num_blocks - 1 - i;
    *num_pairs = n;
    return DGQ_OK;
}

}  // extern "C"
