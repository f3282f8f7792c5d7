// dgq_prompt.cu -- causal grouped-query attention of a prompt (or of a chunk of it behind a history)
// over bf16 K and V, packed rows or paged (sm_103a).
//
// Request b has n = cu_q[b+1] - cu_q[b] query rows and m keys; query row i sits at position
// m - n + i and sees the keys t <= m - n + i:
//   out[i] = sum_t softmax_t(q_i . k_t / sqrt(128)) v_t, zeros where the row sees no key (m < n).
// The G query heads of a KV head are packed into the rows of one product: row r of a tile is token
// r / G, head r % G, so a K and V tile is read once for the whole group.
//
// First form: one CTA of four warps per 64 packed rows of a KV head, keys in tiles of 64 through
// shared memory, mma.sync m16n8k16, online softmax in the log2 domain.
#include "dgq_device.cuh"
#include "dgq.h"
#include "dgq_launch.h"

#include <cuda_bf16.h>
#include <stdint.h>

namespace dgq {

constexpr float kPromptScale = 0.12751743074570180f;  // log2(e) / sqrt(128)
constexpr int kPmRows = 64, kPmKeys = 64;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    const int32_t *cu_q, *kv;  // kv: cu_kv (packed) or sequence lengths (paged)
    const int32_t *bt;         // null: packed
    WsHeader *hdr;
    int32_t B, Hq, Hkv, G, total_q, total_kv, bs, max_blocks, num_blocks;
};

struct PromptSeq {
    int32_t q0, n, kv0, m;  // first query row, query rows, first key row (packed), keys
};

// Request b's rows, held inside the buffers (flagged when they were not).
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs &a, int32_t b, bool flag)
{
    PromptSeq s;
    const int32_t q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    s.q0 = min(max(q0, 0), a.total_q);
    const int32_t e = min(max(q1, s.q0), a.total_q);
    s.n = e - s.q0;
    bool bad = s.q0 != q0 || e != q1;
    if (a.bt) {
        const int32_t m = __ldg(a.kv + b);
        s.kv0 = 0;
        s.m = min(max(m, 0), a.max_blocks * a.bs);
        bad |= s.m != m;
    } else {
        const int32_t k0 = __ldg(a.kv + b), k1 = __ldg(a.kv + b + 1);
        s.kv0 = min(max(k0, 0), a.total_kv);
        const int32_t ke = min(max(k1, s.kv0), a.total_kv);
        s.m = ke - s.kv0;
        bad |= s.kv0 != k0 || ke != k1;
    }
    if (bad && flag) record_error(a.hdr, kErrBadLength);
    return s;
}

__device__ __forceinline__ void pm_mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float pm_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__global__ void __launch_bounds__(128) prompt_simple_kernel(PromptArgs a)
{
    __shared__ __align__(16) uint16_t sk[kPmKeys][kD + 8], sv[kPmKeys][kD + 8];
    __shared__ int32_t s_b, s_unit;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, cq = lane & 3;
    const int32_t h = blockIdx.y, G = a.G, tok_per = kPmRows / G;
    if (tid == 0) {
        int32_t u = blockIdx.x, b = 0;
        for (; b < a.B; ++b) {
            const int32_t nu = (prompt_seq(a, b, true).n + tok_per - 1) / tok_per;
            if (u < nu) break;
            u -= nu;
        }
        s_b = b;
        s_unit = u;
    }
    __syncthreads();
    const int32_t b = s_b;
    if (b >= a.B) return;
    const PromptSeq s = prompt_seq(a, b, false);
    const int32_t t0 = s_unit * tok_per, off = s.m - s.n;
    // this lane's rows: 16 warp + r and + 8
    int32_t tok[2], hd[2], lim[2];
    const uint16_t *qrow[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int row = 16 * warp + r + 8 * e;
        tok[e] = t0 + row / G;
        hd[e] = h * G + row % G;
        const bool ok = row < tok_per * G && tok[e] < s.n;
        lim[e] = ok ? min(s.m, off + tok[e] + 1) : 0;  // keys the row sees
        if (!ok) tok[e] = -1;
        qrow[e] = a.q + ((int64_t)(s.q0 + max(tok[e], 0)) * a.Hq + hd[e]) * kD;
    }
    uint32_t qf[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            qf[k][e] = *reinterpret_cast<const uint32_t *>(qrow[e & 1] + 16 * k + 2 * cq + 8 * (e >> 1));
    float o[16][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    const int32_t keys = min(s.m, off + min(s.n, t0 + tok_per));
    for (int32_t j0 = 0; j0 < keys; j0 += kPmKeys) {
        __syncthreads();
        for (int i = tid; i < kPmKeys * 16; i += 128) {  // 16-byte columns; rows past the end as zeros
            const int row = i >> 4, col = i & 15;
            const int32_t t = j0 + row;
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (t < s.m) {
                int64_t kr;
                if (a.bt) {
                    int32_t blk = __ldg(a.bt + (int64_t)b * a.max_blocks + pow2_div(t, a.bs));
                    if ((uint32_t)blk >= (uint32_t)a.num_blocks) {
                        record_error(a.hdr, kErrBadBlock);
                        blk = 0;
                    }
                    kr = ((int64_t)blk * a.Hkv + h) * a.bs + pow2_mod(t, a.bs);
                } else {
                    kr = (int64_t)(s.kv0 + t) * a.Hkv + h;
                }
                x = __ldg(reinterpret_cast<const uint4 *>(a.k + kr * kD) + col);
                y = __ldg(reinterpret_cast<const uint4 *>(a.v + kr * kD) + col);
            }
            *reinterpret_cast<uint4 *>(&sk[row][col * 8]) = x;
            *reinterpret_cast<uint4 *>(&sv[row][col * 8]) = y;
        }
        __syncthreads();
        float z[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            z[nt][0] = z[nt][1] = z[nt][2] = z[nt][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint16_t *kp = &sk[8 * nt + r][16 * k + 2 * cq];
                pm_mma(z[nt], qf[k], *reinterpret_cast<const uint32_t *>(kp),
                       *reinterpret_cast<const uint32_t *>(kp + 8));
            }
        }
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t t = j0 + 8 * nt + 2 * cq + (e & 1);
                z[nt][e] = t < lim[e >> 1] ? z[nt][e] * kPromptScale : -INFINITY;
                mt[e >> 1] = fmaxf(mt[e >> 1], z[nt][e]);
            }
        float al[2], mu[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 1));
            mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 2));
            const float mn = fmaxf(mx[e], mt[e]);
            mu[e] = mn == -INFINITY ? 0.0f : mn;
            al[e] = pm_ex2(mx[e] - mu[e]);
            mx[e] = mn;
            sum[e] *= al[e];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= al[e >> 1];
        uint32_t p[8][2];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = pm_ex2(z[nt][2 * e] - mu[e]), y = pm_ex2(z[nt][2 * e + 1] - mu[e]);
                const __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
                p[nt][e] = *reinterpret_cast<const uint32_t *>(&w);
                sum[e] += x + y;
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t pa[4] = {p[2 * k][0], p[2 * k][1], p[2 * k + 1][0], p[2 * k + 1][1]};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 16 * k + 2 * cq, d = 8 * i + r;
                const uint32_t b0 = (uint32_t)sv[row][d] | ((uint32_t)sv[row + 1][d] << 16);
                const uint32_t b1 = (uint32_t)sv[row + 8][d] | ((uint32_t)sv[row + 9][d] << 16);
                pm_mma(o[i], pa, b0, b1);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        if (tok[e] < 0) continue;
        const float inv = sum[e] > 0.0f ? 1.0f / sum[e] : 0.0f;
        uint16_t *orow = a.out + ((int64_t)(s.q0 + tok[e]) * a.Hq + hd[e]) * kD;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
            *reinterpret_cast<__nv_bfloat162 *>(orow + 8 * i + 2 * cq) = w;
        }
    }
}

size_t prompt_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int nsm)
{
    (void)B;
    (void)Hq;
    (void)Hkv;
    (void)nsm;
    return sizeof(WsHeader);
}

cudaError_t launch_prompt(const void *q, const void *k, const void *v, int32_t total_q, int32_t total_kv,
                          const int32_t *cu_q, const int32_t *kv, const int32_t *bt, int32_t bs, int32_t max_blocks,
                          int32_t num_blocks, int32_t B, int32_t Hq, int32_t Hkv, void *out, void *ws, int nsm,
                          bool *map_failed, cudaStream_t stream)
{
    *map_failed = false;
    (void)nsm;
    PromptArgs a;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.out = static_cast<uint16_t *>(out);
    a.cu_q = cu_q;
    a.kv = kv;
    a.bt = bt;
    a.hdr = static_cast<WsHeader *>(ws);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.total_q = total_q;
    a.total_kv = total_kv;
    a.bs = bs;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    const int32_t tok_per = kPmRows / a.G;
    const int32_t units = total_q / tok_per + B;  // upper bound: every request rounds up once
    prompt_simple_kernel<<<dim3((unsigned)units, (unsigned)Hkv), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dgq
