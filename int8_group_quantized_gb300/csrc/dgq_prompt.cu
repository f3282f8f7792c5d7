// dgq_prompt.cu -- causal grouped-query attention of a prompt (or of a chunk of it behind a history)
// over bf16 K and V, packed rows or paged (sm_103a).
//
// Request b has n = cu_q[b+1] - cu_q[b] query rows and m keys; query row i sits at position
// m - n + i and sees the keys t <= m - n + i:
//   out[i] = sum_t softmax_t(q_i . k_t / sqrt(128)) v_t, zeros where the row sees no key (m < n).
//
// What bounds it.  4 * 128 flop per (row, key) pair against 512 bytes per key and KV head: the tensor
// cores for prompts (one prompt of 16384 tokens, 32 query and 8 KV heads: 2.2 Tflop for 336 MB), HBM
// for a few rows behind a long history.  Measured on a GB300: 1.23 ms for that prompt, 1788 TFLOP/s,
// 96% of a cuBLAS product's burst rate (1.34 to 1.36 ms, 95 to 97% of the sustained rate, in a long run
// under the power cap); 188 us for eight prompts of 2048 (208 there); 86 to 89 us for sixteen short turns
// over 438 MB of cache.
//
// GPU design.
//  * Rows: the G query heads of a KV head are packed into the rows of one product (row r of a tile is
//    token r / G, head r % G), so a K and V tile is read once for the whole group.  A unit is two
//    tiles of 128 rows (256 / G tokens of one KV head).
//  * Products: S = Q K^T and O += P V on the fifth-generation tensor cores (tcgen05.mma, 128 x 128 x 16
//    per instruction, fp32 accumulators in tensor memory).  Tensor memory holds S and O of both tiles
//    (4 x 128 columns, all of it); P, rounded to bf16, overwrites the S it came from and is the A
//    operand of the second product, so no weight passes through shared memory.  V is read as it lies
//    (keys by values), a transposed B operand.
//  * Roles: warps 0-3 and 4-7 are the softmax of tile 0 and of tile 1, one row per thread; warp 8 loads
//    (TMA, a ring of four 32 KB K or V tiles under the 128-byte swizzle; five measured the same) and
//    hands the pieces of work to the others; one thread of warp 9 issues every product.  While one
//    tile's softmax runs, the tensor cores work on the other's products.  (A product warp for each
//    tile was slower, 1.78 against 1.52 ms: their products interleave, both tiles finish together and
//    the tensor cores wait for both.  So was a warpgroup of its own for writing results.)
//  * The code of all roles has to stay in the instruction cache, and there is next to no L1 left for
//    spilled registers: unrolling the wait loops (200 KB of code) cost 25% on ragged batches, 200
//    bytes of spills 30%.  The warp index goes through a shuffle so that the compiler knows the roles'
//    branches are uniform: the products' operands then stay in uniform registers (1.40 -> 1.30 ms).
//  * Softmax: online, log2 domain, the reference maximum moving only when a tile exceeds it by 8 (lazy
//    rescaling: O in tensor memory is then multiplied in place; the softmax threads may do that
//    between products because S of the next key tile is complete only after O's product is).
//    (The one-pass softmax is Milakov and Gimelshein's, 2018; two row tiles in turn, P in the place of S and
//    the lazy maximum are known from published attention kernels of this hardware generation.)
//  * Work where a CTA's share (one per SM) is at least kPmQueued times the longest unit: the load warps
//    draw whole units from a counter, requests in their order and a request's longest unit first, the next
//    number while a unit is loaded.  All CTAs then work in few requests at a time, whose K and V stay in
//    L2; which CTA has a unit changes no result.  The last request's units decide how evenly CTAs end: a
//    prompt's short ones level them out, units of one length leave up to one of them, and a short chunk
//    behind a long history at the list's end leaves its units to few CTAs alone.  Against slices (below),
//    us with launch, calls on their own: 199 -> 188 for eight prompts of 2048, 195 -> 180 for eight chunks
//    of 512 behind 3584; thirty prompts of 2048 and 64 tokens behind 16320 in front of them 748 -> 659, at
//    their end 746 -> 811; thirteen and 64 tokens behind 8128 330 -> 299 and 330 -> 371.
//  * Else the units lie in one flat list by cost, a unit costing the keys it sees plus a constant, and
//    each CTA takes an equal slice, which may begin and end inside a unit, at a key tile.  A unit cut
//    that way leaves its parts' maxima, sums and unnormalised O in the workspace, and a merge kernel
//    chained with programmatic dependent launch folds them in order (bitwise repeatable on a given
//    GPU).  Cuts within kPmSnap key tiles of a unit's end move there.
//  * What cannot be seen: columns past a row's limit get weight 0; V rows behind a request's end are
//    zeroed in shared memory, so that values of other requests or of unused slots (NaN too) never
//    meet a weight.
//  * Every wait is bounded: one that runs out records an error and its role leaves, after which the others'
//    waits run out too.
#include "dgq_device.cuh"
#include "dgq.h"
#include "dgq_launch.h"

#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

namespace dgq {

constexpr float kPmScale = 0.12751743074570180f;  // log2(e) / sqrt(128)
constexpr float kPmLazy = 8.0f / kPmScale;        // the maximum moves when exceeded by 8 in the log2 domain
// A weight is 2^(x s - fl(m s)), so the largest one is not 1 but 2^e with e the rounding of m s: the same factor
// in numerator and sum, until from |m| = 2^31 on it leaves the range of fp32 (|e| <= 16 below).  There a power
// of two stands for s, with which m s is exact; scores that differ do so by 128 or more, so that with either
// factor any weight but the largest is below 2^-16, and with it below what P's bf16 can add to it.
constexpr float kPmFar = 2147483648.0f;
constexpr int kPmTile = 128;                      // rows of a tile, keys of a key tile
constexpr int kPmStages = 4;
constexpr int kPmTileBytes = kPmTile * kD * 2;    // 32 KB: two halves of 64 columns, [row][64] each
constexpr int kPmHalf = kPmTileBytes / 2;
constexpr int kPmThreads = 320;  // two softmax warpgroups, a load warp, a product warp
constexpr int kPmLoadWarp = 8, kPmMmaWarp = 9;
// A unit's fixed cost, in keys, and what a key tile costs where only tile 0 has rows (it takes 0.76 to 0.85
// of the time of both).  Sixteen short turns behind up to 32768, us with launch: 128 -> 106, 160 -> 100,
// 192 -> 102; all key tiles alike 108.
constexpr int kPmUnitCost = 160, kPmLoneTile = 104;
// Key tiles: no part of a cut unit is smaller.  The same turns: 1 -> 101, 2 -> 100, 4 -> 102.
constexpr int kPmSnap = 2;
// Shares from which on units are drawn from a counter.  464 units of one length (58 requests, 3.05 to a
// CTA) take as long as in slices, 124 us with launch; at two, 2 prompts of 2048 do, 77 us.
constexpr int kPmQueued = 3;
constexpr int kPmRows = 2 * kPmTile;              // packed rows of a unit
// A wait ends after this many polls.  One that finds its barrier open took 7776 cycles (4 us), which makes a
// second of them; how long a poll suspends is up to the hardware, so the time is not a promise.
constexpr uint32_t kPmWaitPolls = 1u << 18;

// Tensor-memory columns of the 512 a CTA takes: S (and P) of tile 0 and 1, O of tile 0 and 1.
constexpr uint32_t kPmColS = 0, kPmColO = 256;

struct PromptArgs {
    uint16_t *out;
    const int32_t *cu_q, *kv;  // kv: cu_kv (packed) or sequence lengths (paged)
    const int32_t *bt;         // null: packed
    WsHeader *hdr;
    int4 *head;    // per CTA: the unit its slice ends inside of and begins (x: 1 + slot parity, or 0)
    int32_t *cont; // per CTA: 1 its first piece continues a unit, 2 and ends it there
    float2 *ml;    // per slot and row: maximum and sum
    float *part;   // per slot: O [256][128], unnormalised
    int32_t B, Hq, Hkv, G, lg, total_q, total_kv, bs, max_blocks, num_blocks;
};

struct PromptMaps {
    CUtensorMap q, k, v;
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

// ---- the flat list of units ---------------------------------------------------------------------

// A position in the list: request, KV head, unit, key tile.
struct PromptPos {
    int32_t b, h, i, j;
};

__device__ __forceinline__ bool same_unit(const PromptPos &x, const PromptPos &y)
{
    return x.b == y.b && x.h == y.h && x.i == y.i;
}

__device__ __forceinline__ int32_t prompt_units(const PromptSeq &s, int32_t U) { return (s.n + U - 1) >> (__ffs(U) - 1); }

// Keys that the tokens before `tok` of the request see (the last of them sees all of these).
__device__ __forceinline__ int32_t keys_before(const PromptSeq &s, int32_t tok)
{
    return max(0, s.m - s.n + min(tok, s.n));
}

__device__ __forceinline__ int32_t key_tiles(int32_t keys) { return (keys + kPmTile - 1) / kPmTile; }

// Cost of a head's first i units (the last one not among them): kPmUnitCost each and the keys of its
// last token, max(0, off + x U) for unit x = 1 .. i.
__device__ __forceinline__ int64_t unit_cost(const PromptSeq &s, int32_t U, int32_t i)
{
    const int32_t off = s.m - s.n;
    const int64_t x0 = off >= 0 ? 0 : min(i, -off >> (__ffs(U) - 1));  // units that see no key
    const int64_t c = (int64_t)i - x0;
    return (int64_t)i * kPmUnitCost + c * off + U * (((int64_t)i * (i + 1) - x0 * (x0 + 1)) / 2);
}

// A head's last unit sees all keys; where it has rows in tile 0 only, a key tile costs kPmLoneTile.
__device__ __forceinline__ bool lone_tile(const PromptSeq &s, int32_t U, int32_t nu) { return s.n - (nu - 1) * U <= U / 2; }

// Cost of a head with nu units.
__device__ __forceinline__ int64_t head_cost(const PromptSeq &s, int32_t U, int32_t nu)
{
    if (nu == 0) return 0;
    const int64_t last = lone_tile(s, U, nu) ? (uint64_t)s.m * kPmLoneTile / kPmTile : s.m;
    return unit_cost(s, U, nu - 1) + kPmUnitCost + last;
}

__device__ __forceinline__ PromptSeq seq_of_lane(const PromptSeq &s, int l)
{
    return PromptSeq{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.n, l),
                     __shfl_sync(0xffffffffu, s.kv0, l), __shfl_sync(0xffffffffu, s.m, l)};
}

// The unit behind p (the whole warp: empty requests are passed 32 at a time); R: requests up to the last one
// with rows.  (One at a time up to the end, the last block of eight requests padded to 256 finished 14 us
// after the others.)
__device__ __forceinline__ void next_unit(const PromptArgs &a, int32_t U, int32_t R, int lane, PromptPos &p, PromptSeq &s)
{
    p.j = 0;
    if (++p.i < prompt_units(s, U)) return;
    p.i = 0;
    if (++p.h < a.Hkv) return;
    p.h = 0;
    for (++p.b; p.b < R; p.b += 32) {
        PromptSeq t = {0, 0, 0, 0};
        if (p.b + lane < R) t = prompt_seq(a, p.b + lane, false);
        const uint32_t hit = __ballot_sync(0xffffffffu, t.n > 0);
        if (hit) {
            s = seq_of_lane(t, __ffs(hit) - 1);
            p.b += __ffs(hit) - 1;
            return;
        }
    }
    p.b = a.B;
}

// The units drawn one by one, a request's longest first: the requests in a window of 32, one per lane.
struct PromptQueue {
    PromptSeq s;    // this lane's request
    int64_t upto;   // units of the window's requests up to it
    int64_t base;   // units before the window
    int32_t first;  // the window's first request
};

__device__ __forceinline__ void queue_window(const PromptArgs &a, int32_t U, int32_t R, int lane, PromptQueue &w)
{
    w.s = PromptSeq{0, 0, 0, 0};
    if (w.first + lane < R) w.s = prompt_seq(a, w.first + lane, false);
    w.upto = (int64_t)prompt_units(w.s, U) * a.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w.upto, o);
        if (lane >= o) w.upto += y;
    }
}

// Unit number `ticket` and its request, or false: there are not so many (the whole warp; tickets only rise).
__device__ __forceinline__ bool queue_unit(const PromptArgs &a, int32_t U, int32_t R, int lane, PromptQueue &w,
                                           int64_t ticket, PromptPos &p, PromptSeq &s)
{
    for (;;) {
        const uint32_t hit = __ballot_sync(0xffffffffu, w.base + w.upto > ticket);
        if (hit) {
            const int l = __ffs(hit) - 1;
            s = seq_of_lane(w.s, l);
            const int32_t back = (int32_t)(w.base + __shfl_sync(0xffffffffu, w.upto, l) - ticket) - 1;  // from the request's end
            p.b = w.first + l;
            p.i = back / a.Hkv;
            p.h = back - p.i * a.Hkv;
            p.j = 0;
            return true;
        }
        w.base += __shfl_sync(0xffffffffu, w.upto, 31);
        w.first += 32;
        if (w.first >= R) return false;
        queue_window(a, U, R, lane, w);
    }
}

// The last of n positions from 0 on where `yes` holds (it does at 0, and nowhere behind a position where it
// does not): 32 are looked at together.
template <typename F>
__device__ __forceinline__ int32_t last_where(int32_t n, int lane, F yes)
{
    int32_t lo = 0;
    while (n > 1) {
        const int32_t step = (n - 1) / 32 + 1, x = lane * step;
        const int32_t c = __popc(__ballot_sync(0xffffffffu, x < n && yes(lo + x))) - 1;
        lo += c * step;
        n = min(step, n - c * step);
    }
    return lo;
}

// The unit and key tile at cost position pos (pre: cost prefix over requests, [B + 1]); the whole warp.
__device__ PromptPos cut_at(const PromptArgs &a, int32_t U, int32_t R, int64_t pos, const int64_t *pre, int lane)
{
    PromptPos p = {a.B, 0, 0, 0};
    if (pos >= pre[a.B]) return p;
    p.b = last_where(R, lane, [&](int32_t b) { return pre[b] <= pos; });
    PromptSeq s = prompt_seq(a, p.b, false);  // has units: the next prefix is larger
    const int32_t nu = prompt_units(s, U);
    const int64_t per_head = head_cost(s, U, nu);
    int64_t r = pos - pre[p.b];
    p.h = (int32_t)__fdividef((float)r, (float)per_head);  // off by one at most below a million heads
    r -= p.h * per_head;
    for (; r < 0; r += per_head) --p.h;
    for (; r >= per_head; r -= per_head) ++p.h;
    const int32_t lo = last_where(nu, lane, [&](int32_t i) { return unit_cost(s, U, i) <= r; });
    p.i = lo;
    r -= unit_cost(s, U, lo) + kPmUnitCost;
    const int32_t tiles = key_tiles(keys_before(s, (lo + 1) * U));
    int32_t j = r > 0 ? (int32_t)r / (lo == nu - 1 && lone_tile(s, U, nu) ? kPmLoneTile : kPmTile) : 0;  // (r <= m < 2^31)
    if (j > tiles - kPmSnap) {
        if (j >= kPmSnap || r > 0) next_unit(a, U, R, lane, p, s);
        return p;
    }
    p.j = j < kPmSnap ? 0 : j;
    return p;
}

// ---- tcgen05 ------------------------------------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// 32 columns of the warp's 32 lanes: thread l receives lane l's columns.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// D (fp32, 128 x 128) (+)= A B, 16 deep, bf16 operands; B n-by-k (K-major) in shared memory.
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
// the same with B k-by-n as it lies (MN-major: bit 16)
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// Shared-memory operand descriptors of a pair of [128][64] halves under the 128-byte swizzle: address
// and strides in units of 16 bytes, version 1 (bit 46), swizzle mode 2 (bit 61); 8-row groups 1024
// bytes apart.  Only the low word differs between operands: the address and the other stride, which
// K-major operands do not use and MN-major ones take as the distance of their 64-column atoms.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return (addr >> 4) | ((uint32_t)(kPmHalf >> 4) << 16); }

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t atmem, uint32_t blo, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(atmem), "r"(blo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void tma_tile_4d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_tile_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Whether the phase of that parity is complete (1 or 0): after a short wait, and without waiting.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}

// Offset of k-step k (16 columns) in a K-major operand, in descriptor units.
__device__ __forceinline__ constexpr uint32_t kstep(int k) { return ((k >> 2) * kPmHalf + (k & 3) * 32) >> 4; }

// 16 bytes to global memory where `yes` (a predicated store: no branch).
__device__ __forceinline__ void st_if(void *p, const uint4 &v, bool yes)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((uint32_t)yes)
                 : "memory");
}

// ---- small arithmetic -----------------------------------------------------------------------------

__device__ __forceinline__ float pm_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float pm_rcp(float x)  // to one unit in the last place
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint32_t pm_pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// ---- the kernel -----------------------------------------------------------------------------------

// A piece as the load warp hands it to the other roles, through a ring of kPmItems entries.
struct PromptItem {
    int32_t e0, e1;  // key tiles of tile 0 and 1 (both < 0: no more pieces)
    int32_t see;     // keys of the piece that the unit's first token sees: token i of it sees `see` + i
    int32_t toks;    // the request's tokens from the unit's first on
    int32_t row;     // row of that token in q and out
    int32_t h;       // KV head
    int32_t slot;    // where its part goes, or -1: a whole unit
    int32_t pad;
};
static_assert(sizeof(PromptItem) == 32, "eight words, one per lane");
constexpr int kPmItems = 4;

struct PromptBars {
    uint64_t item_full[kPmItems], item_empty[kPmItems];
    PromptItem items[kPmItems];
    uint64_t full[kPmStages], empty[kPmStages];
    uint64_t q_full[2], s_full[2], p_most[2], p_ready[2], o_full[2];
    uint64_t q_empty, v_part, drain;
    uint32_t tmem;
    PromptPos cut[2];
    int64_t wsum[kPmThreads / 32];
    int32_t wmax[kPmThreads / 32], wlast[kPmThreads / 32];
};

constexpr int kPmTurn = 32 * 128;  // a softmax warp's buffer for turning rows
constexpr size_t kPmSmem = (size_t)(2 + kPmStages) * kPmTileBytes + 8 * kPmTurn + sizeof(PromptBars);
static_assert(kPmSmem <= 232448, "shared memory of a CTA");
static_assert((size_t)(kMaxCallBatch + 1) * 8 <= (size_t)kPmStages * kPmTileBytes, "the request prefix uses the ring");

// Bounded wait, with one answer for the warp.  False: the wait ran out; the caller leaves, and whoever
// waits for it runs out in turn.
__device__ __forceinline__ bool pm_wait(uint32_t bar, uint32_t parity, WsHeader *hdr)
{
#pragma unroll 1
    for (uint32_t i = 0; i < kPmWaitPolls; ++i)
        if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    record_error(hdr, kErrFullWait);
    return false;
}

// A unit's tiles in the piece [j0, j1): per tile the key tiles to go through, and its keys.
struct PromptPiece {
    int32_t j1;        // end of the piece
    int32_t e0, e1;    // key tiles of tile 0, 1 inside the piece (from j0)
    int32_t steps;     // key tiles loaded
};

__device__ __forceinline__ PromptPiece piece_of(const PromptSeq &s, const PromptPos &p, const PromptPos &end, int32_t U)
{
    PromptPiece z;
    const int32_t half = U / 2, tok = p.i * U;
    const int32_t k0 = keys_before(s, tok + half), k1 = keys_before(s, tok + U);
    const bool two = tok + half < s.n;  // tile 1 has rows
    z.j1 = same_unit(p, end) ? end.j : key_tiles(k1);
    z.e0 = max(0, min(z.j1, key_tiles(k0)) - p.j);
    z.e1 = two ? max(0, z.j1 - p.j) : 0;
    z.steps = max(z.e0, z.e1);
    return z;
}

__device__ __forceinline__ bool before(const PromptPos &x, const PromptPos &end)
{
    if (x.b != end.b) return x.b < end.b;
    if (x.h != end.h) return x.h < end.h;
    if (x.i != end.i) return x.i < end.i;
    return x.j < end.j;
}

__global__ void __launch_bounds__(kPmThreads, 1) prompt_kernel(const PromptArgs a, const __grid_constant__ PromptMaps maps)
{
    extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle repeats every 1024 bytes)
    PromptBars *sb = reinterpret_cast<PromptBars *>(smem + (2 + kPmStages) * kPmTileBytes + 8 * kPmTurn);
    const uint32_t sq = smem_u32(smem), sring = sq + 2 * kPmTileBytes;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be
    const int32_t G = a.G, lg = a.lg, U = kPmRows >> lg;

    pdl_launch_dependents();  // the merge may be scheduled while this kernel runs

    if (tid < 3) prefetch_tensormap(tid == 0 ? &maps.q : (tid == 1 ? &maps.k : &maps.v));
    // ---- this CTA's slice of the flat list, or whether units are handed out one by one
    bool queued;
    int32_t requests;  // up to the last one with rows
    {
        int64_t *pre = reinterpret_cast<int64_t *>(smem + 2 * kPmTileBytes);  // the ring is not in use yet
        int64_t carry = 0;
        int32_t longest = 0;
        requests = 0;
        for (int32_t base = 0; base < a.B; base += kPmThreads) {
            const int32_t b = base + tid;
            int64_t c = 0;
            if (b < a.B) {
                const PromptSeq s = prompt_seq(a, b, blockIdx.x == 0);
                c = a.Hkv * head_cost(s, U, prompt_units(s, U));
                if (s.n > 0) {
                    longest = max(longest, s.m);
                    requests = b + 1;
                }
            }
            int64_t x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) sb->wsum[warp] = x;
            __syncthreads();
            int64_t before_warp = 0, all = 0;
#pragma unroll
            for (int w = 0; w < kPmThreads / 32; ++w) {
                if (w < warp) before_warp += sb->wsum[w];
                all += sb->wsum[w];
            }
            if (b < a.B) pre[b] = carry + before_warp + x - c;
            carry += all;
            __syncthreads();
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        requests = __reduce_max_sync(0xffffffffu, requests);
        if (lane == 0) {
            sb->wmax[warp] = longest;
            sb->wlast[warp] = requests;
        }
        if (tid == 0) {
            pre[a.B] = carry;
            for (int i = 0; i < kPmStages; ++i) {
                mbar_init(&sb->full[i], 1);
                mbar_init(&sb->empty[i], 1);
            }
            for (int t = 0; t < 2; ++t) {
                mbar_init(&sb->q_full[t], 1);
                mbar_init(&sb->s_full[t], 1);
                mbar_init(&sb->p_most[t], 4);
                mbar_init(&sb->p_ready[t], 4);
                mbar_init(&sb->o_full[t], 1);
            }
            for (int i = 0; i < kPmItems; ++i) {
                mbar_init(&sb->item_full[i], 1);
                mbar_init(&sb->item_empty[i], 9);  // eight softmax warps and the product warp
            }
            mbar_init(&sb->q_empty, 1);
            mbar_init(&sb->v_part, 1);
            mbar_init(&sb->drain, 1);
            fence_barrier_init();
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kPmThreads / 32; ++w) {
            longest = max(longest, sb->wmax[w]);
            requests = max(requests, sb->wlast[w]);
        }
        queued = ((int64_t)longest + kPmUnitCost) * (kPmQueued * gridDim.x) <= carry;
        if (queued) {
            if (lane == 0 && warp < 2) sb->cut[warp] = PromptPos{warp ? a.B : 0, 0, 0, 0};
        } else if (warp < 2) {
            // carry * c / n in steps of 2^-20 (monotone, exact at c = n, no 64-bit division: one took 400 cycles)
            const int64_t f = (uint32_t)((blockIdx.x + warp) << 20) / gridDim.x;
            const PromptPos c = cut_at(a, U, requests, (carry >> 20) * f + (((carry & 0xfffff) * f) >> 20), pre, lane);
            if (lane == 0) sb->cut[warp] = c;
        }
        __syncthreads();
    }
    const PromptPos begin = sb->cut[0], end = sb->cut[1];
    const bool work = before(begin, end);  // (queued: any)
    if (tid == 0) {  // read by the merge
        const bool one = same_unit(begin, end);
        int4 head = make_int4(0, 0, 0, 0);
        if (work && end.j > 0 && !(one && begin.j > 0)) head = make_int4(one ? 1 : 2, end.b, end.h, end.i);
        a.head[blockIdx.x] = head;
        a.cont[blockIdx.x] = work && begin.j > 0 ? (one ? 1 : 2) : 0;
        if (blockIdx.x == 0) a.hdr->path = queued ? kPathPromptDrawn : kPathPromptSliced;  // (tests read it)
    }
    if (!work) return;  // the whole CTA: no barrier follows for it
    if (warp == kPmMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&sb->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb->tmem;

    uint32_t ni = 0;  // items taken
    auto next_item = [&](PromptItem &z) -> bool {
        const uint32_t i = ni % kPmItems;
        if (!pm_wait(smem_u32(&sb->item_full[i]), (ni / kPmItems) & 1u, a.hdr)) return false;
        const int32_t w = reinterpret_cast<const int32_t *>(&sb->items[i])[lane & 7];
        z.e0 = __shfl_sync(0xffffffffu, w, 0);
        z.e1 = __shfl_sync(0xffffffffu, w, 1);
        z.see = __shfl_sync(0xffffffffu, w, 2);
        z.toks = __shfl_sync(0xffffffffu, w, 3);
        z.row = __shfl_sync(0xffffffffu, w, 4);
        z.h = __shfl_sync(0xffffffffu, w, 5);
        z.slot = __shfl_sync(0xffffffffu, w, 6);
        if (lane == 0) mbar_arrive(&sb->item_empty[i]);
        ++ni;
        return z.e0 >= 0;
    };

    if (warp == kPmLoadWarp) {
        // ======================================== pieces and their loads
        PromptPos pos = begin;
        PromptSeq s;
        PromptQueue queue;
        uint32_t ticket = 0;  // (lane 0)
        bool more = true;
        if (queued) {
            queue.base = 0;
            queue.first = 0;
            queue_window(a, U, requests, lane, queue);
            more = queue_unit(a, U, requests, lane, queue, blockIdx.x, pos, s);
        } else {
            s = prompt_seq(a, pos.b, false);
        }
        auto advance = [&]() {
            if (queued) {
                more = queue_unit(a, U, requests, lane, queue, (int64_t)gridDim.x + __shfl_sync(0xffffffffu, ticket, 0), pos, s);
            } else {
                next_unit(a, U, requests, lane, pos, s);
                more = before(pos, end);
            }
        };
        auto hand_out = [&](const PromptItem &z) -> bool {
            const uint32_t i = ni % kPmItems;
            if (ni >= kPmItems && !pm_wait(smem_u32(&sb->item_empty[i]), (ni / kPmItems - 1) & 1u, a.hdr))
                return false;
            if (lane == 0) {
                sb->items[i] = z;
                mbar_arrive(&sb->item_full[i]);
            }
            ++ni;
            return true;
        };
        fence_proxy_async_smem();  // the prefix was read from the ring by ordinary loads
        const int32_t pages = a.bt ? kPmTile / a.bs : 0;  // pages of a key tile
        uint32_t it = 0, nv = 0;
        uint32_t nq0 = 0, nq1 = 0;  // Q tiles loaded
        bool ok = true, v_flight = false;
        uint32_t q_loaded = 0;  // pieces with a Q load
        // a unit's Q, behind its first K: its buffer is free once the last unit's last S is done
        auto load_q = [&](const PromptPiece &z) -> bool {
            if (q_loaded > 0 && !pm_wait(smem_u32(&sb->q_empty), (q_loaded - 1) & 1u, a.hdr)) return false;
            ++q_loaded;
            if (lane == 0) {
                const int32_t tok = s.q0 + pos.i * U;
                if (z.e0 > 0) {
                    ++nq0;
                    mbar_arrive_expect_tx(&sb->q_full[0], kPmTileBytes);
                    tma_tile_4d(sq, &maps.q, 0, pos.h * G, tok, 0, &sb->q_full[0]);
                }
                if (z.e1 > 0) {
                    ++nq1;
                    mbar_arrive_expect_tx(&sb->q_full[1], kPmTileBytes);
                    tma_tile_4d(sq + kPmTileBytes, &maps.q, 0, pos.h * G, tok + U / 2, 0, &sb->q_full[1]);
                }
            }
            return true;
        };
        for (bool first = true; ok && more; advance(), first = false) {
            if (queued && lane == 0) ticket = atomicAdd(&a.hdr->tickets, 1u);  // of the next unit
            const PromptPiece z = piece_of(s, pos, end, U);
            const int32_t toks = s.n - pos.i * U, row0 = s.q0 + pos.i * U;
            if (z.steps == 0) {  // rows that see no key
                for (int32_t x = lane; x < min(U, toks) * G * 16; x += 32) {
                    const int32_t r = x >> 4;
                    reinterpret_cast<uint4 *>(a.out + ((int64_t)(row0 + (r >> lg)) * a.Hq + pos.h * G + (r & (G - 1))) * kD)[x & 15] =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            const bool partial = pos.j > 0 || (same_unit(pos, end) && end.j > 0);
            if (!hand_out(PromptItem{z.e0, z.e1, s.m - s.n + 1 + pos.i * U - pos.j * kPmTile, toks, row0, pos.h,
                                     partial ? 2 * (int32_t)blockIdx.x + (first ? 0 : 1) : -1, 0})) {
                ok = false;
                break;
            }
            // lane l copies half l % 2 of page l / 2 of the key tile
            auto block_of = [&](int32_t j) -> int32_t {
                int32_t blk = 0;
                const int32_t t = j * kPmTile + (lane >> 1) * a.bs;
                if (lane < 2 * pages && t < s.m) {
                    blk = __ldg(a.bt + (int64_t)pos.b * a.max_blocks + pow2_div(t, a.bs));
                    if ((uint32_t)blk >= (uint32_t)a.num_blocks) {  // not a block of the cache: flagged,
                        record_error(a.hdr, kErrBadBlock);          // and block 0 read instead
                        blk = 0;
                    }
                }
                return blk;
            };
            int32_t blk = a.bt ? block_of(pos.j) : 0;
            for (int32_t j = pos.j; j < pos.j + z.steps; ++j) {
                const int32_t valid = min(kPmTile, s.m - j * kPmTile);  // keys of the tile
                const int32_t blk_next = a.bt && j + 1 < pos.j + z.steps ? block_of(j + 1) : 0;
                const int32_t used = a.bt ? (valid + a.bs - 1) / a.bs : 0;
                const uint32_t bytes = a.bt ? (uint32_t)used * a.bs * kD * 2 : (uint32_t)kPmTileBytes;
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t st = it % kPmStages, dst = sring + st * kPmTileBytes;
                    if (it >= kPmStages && !pm_wait(smem_u32(&sb->empty[st]), (it / kPmStages - 1) & 1u, a.hdr)) {
                        ok = false;
                        break;
                    }
                    const CUtensorMap *map = kv ? &maps.v : &maps.k;
                    const bool part = kv == 1 && valid < kPmTile;  // V rows to clear behind the end
                    uint64_t *bar = part ? &sb->v_part : &sb->full[st];
                    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (a.bt) {
                        if (lane < 2 * used) {
                            const int32_t row = (blk * a.Hkv + pos.h) * a.bs;
                            tma_tile_2d(dst + (lane & 1) * kPmHalf + (lane >> 1) * a.bs * 128, map, (lane & 1) * 64, row,
                                        bar);
                        }
                    } else if (lane == 0) {
                        tma_tile_4d(dst, map, 0, s.kv0 + j * kPmTile, pos.h, 0, bar);
                    }
                    v_flight = part;
                    if (part) {
                        if (!pm_wait(smem_u32(&sb->v_part), nv & 1u, a.hdr)) {
                            ok = false;
                            break;
                        }
                        ++nv;
                        v_flight = false;
                        uint8_t *t = smem + 2 * kPmTileBytes + st * kPmTileBytes;
                        for (int32_t x = valid * 8 + lane; x < kPmTile * 8; x += 32) {
                            *reinterpret_cast<uint4 *>(t + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4 *>(t + kPmHalf + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sb->full[st]);
                    }
                    ++it;
                    if (kv == 0 && j == pos.j && !load_q(z)) {
                        ok = false;
                        break;
                    }
                }
                if (!ok) break;
                blk = blk_next;
            }
        }
        if (ok) ok = hand_out(PromptItem{-1, -1, 0, 0, 0, 0, -1, 0});
        if (!ok && lane == 0) {  // a wait ran out: no copy may still be in flight when the CTA ends
            auto drain = [](uint64_t *bar, uint32_t parity) {
#pragma unroll 1
                for (uint32_t i = 0; i < kPmWaitPolls && !mbar_try_wait(bar, parity); ++i) {}
            };
            for (uint32_t k = it > kPmStages ? it - kPmStages : 0; k < it; ++k)
                drain(&sb->full[k % kPmStages], (k / kPmStages) & 1u);
            if (nq0 > 0) drain(&sb->q_full[0], (nq0 - 1) & 1u);
            if (nq1 > 0) drain(&sb->q_full[1], (nq1 - 1) & 1u);
            if (v_flight) drain(&sb->v_part, nv & 1u);
        }
        __syncwarp();
    } else if (warp == kPmMmaWarp) {
        // ======================================== products: the warp walks, one lane issues
        // Two products fit into the tensor cores' queue, so whatever the warp does between the last
        // product of a turn and the first of the next leaves them idle.  A turn is one tile's O += P V
        // of key tile j and S = Q K^T of key tile j + 1; the barriers that the next turn needs are
        // polled between this turn's products, and waited for only when a poll found them open.
        // (Operands go through a shuffle so that the compiler sees them uniform over the warp.)
        uint32_t st = 0, ph = 0;        // ring stage and parity of the next K tile
        uint32_t qpar = 0, ppar = 0;    // bit t: parity of the next Q and P tile of tile t
        bool ok = true;
        const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t q_desc = __shfl_sync(0xffffffffu, desc_k(sq), 0);
        const uint32_t k_desc = desc_k(sring), v_desc = desc_mn(sring);
        const uint32_t full0 = smem_u32(&sb->full[0]), empty0 = smem_u32(&sb->empty[0]);
        auto wait = [&](uint32_t bar, uint32_t parity) { return pm_wait(bar, parity, a.hdr); };
        auto wrap = [](uint32_t x) { return x >= kPmStages ? x - kPmStages : x; };
        for (PromptItem z; ok && next_item(z);) {
            const int32_t steps = max(z.e0, z.e1);
            // S of the first key tile
            if (!wait(full0 + 8 * st, ph)) break;
            uint32_t kb = __shfl_sync(0xffffffffu, k_desc + st * (kPmTileBytes >> 4), 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if ((t ? z.e1 : z.e0) == 0) continue;
                if (!wait(smem_u32(&sb->q_full[t]), (qpar >> t) & 1u)) { ok = false; break; }
                qpar ^= 1u << t;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ss(base + kPmColS + t * 128, q_desc + t * (kPmTileBytes >> 4) + kstep(k), kb + kstep(k),
                                  kIdescQK, k > 0);
                    tc_commit(smem_u32(&sb->s_full[t]));
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) {
                tc_commit(empty0 + 8 * st);
                if (steps == 1) tc_commit(smem_u32(&sb->q_empty));
            }
            __syncwarp();
            // stage and parity of V of key tile j, and of K of the next
            uint32_t sv = wrap(st + 1), sk = wrap(st + 2);
            uint32_t hv = ph ^ (sv < st), hk = ph ^ (sk < st);
            uint32_t vb = __shfl_sync(0xffffffffu, v_desc + sv * (kPmTileBytes >> 4), 0);
            kb = __shfl_sync(0xffffffffu, k_desc + sk * (kPmTileBytes >> 4), 0);
            uint32_t got = 0;  // bit 0: V and K of the next step are known to be there, bit 1 + t: P of tile t
            for (int32_t j = 0; j < steps; ++j) {
                const bool more = j + 1 < steps;
                if (!(got & 1u) && (!wait(full0 + 8 * sv, hv) || (more && !wait(full0 + 8 * sk, hk)))) { ok = false; break; }
                const uint32_t acc = __shfl_sync(0xffffffffu, j > 0 ? 1u : 0u, 0);
                uint32_t vn = 0, kn = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int32_t e = t ? z.e1 : z.e0;
                    if (j >= e) continue;
                    const uint32_t pbar = smem_u32(&sb->p_ready[t]), par = (ppar >> t) & 1u;
                    if (!(got & (2u << t)) && !wait(smem_u32(&sb->p_most[t]), par)) { ok = false; break; }
                    tc_fence_after();
                    uint32_t g = 0;
                    if (elect_one()) {
                        // keys 96 .. 127 and 0 .. 63, then 64 .. 95, as the softmax stores them
#pragma unroll
                        for (int i = 0; i < 6; ++i) {
                            const int k = (i + 6) & 7;
                            tc_mma_ts(base + kPmColO + t * 128, base + kPmColS + t * 128 + k * 8, vb + k * (2048 >> 4),
                                      kIdescPV, i > 0 ? 1u : acc);
                        }
                        g = bar_test(pbar, par);
                    }
                    if (!__any_sync(0xffffffffu, g) && !wait(pbar, par)) { ok = false; break; }
                    tc_fence_after();
                    g = 0;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 4; k < 6; ++k)
                            tc_mma_ts(base + kPmColO + t * 128, base + kPmColS + t * 128 + k * 8, vb + k * (2048 >> 4),
                                      kIdescPV, 1u);
                        const bool last = t == 1 || j >= z.e1;  // the step's last turn
                        if (last) {
                            vn = wrap(sv + 2);
                            kn = wrap(sk + 2);
                            g = bar_test(full0 + 8 * vn, hv ^ (vn < sv)) & (j + 2 < steps ? bar_test(full0 + 8 * kn, hk ^ (kn < sk)) : 1u);
                        }
                        if (j + 1 < e) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                tc_mma_ss(base + kPmColS + t * 128, q_desc + t * (kPmTileBytes >> 4) + kstep(k), kb + kstep(k),
                                          kIdescQK, k > 0);
                                if (k == 6) g |= bar_test(smem_u32(&sb->p_most[t ^ 1]), (ppar >> (t ^ 1)) & 1u) << (1 + (t ^ 1));
                            }
                            tc_commit(smem_u32(&sb->s_full[t]));
                        } else {
                            tc_commit(smem_u32(&sb->o_full[t]));
                        }
                        if (last) {
                            tc_commit(empty0 + 8 * sv);
                            if (more) tc_commit(empty0 + 8 * sk);
                            if (j + 2 == steps) tc_commit(smem_u32(&sb->q_empty));
                            vn = v_desc + vn * (kPmTileBytes >> 4);
                            kn = k_desc + kn * (kPmTileBytes >> 4);
                        }
                    }
                    ppar ^= 1u << t;
                    got = __reduce_or_sync(0xffffffffu, g);
                }
                if (!ok) break;
                vb = __reduce_or_sync(0xffffffffu, vn);
                kb = __reduce_or_sync(0xffffffffu, kn);
                const uint32_t v2 = wrap(sv + 2), k2 = wrap(sk + 2);
                hv ^= v2 < sv;
                hk ^= k2 < sk;
                sv = v2;
                sk = k2;
            }
            if (!ok) break;
            // the piece took 2 steps tiles: the next K tile follows the last V, one before sv
            const uint32_t s1 = sv == 0 ? kPmStages - 1 : sv - 1;
            ph = hv ^ (s1 > sv);
            st = s1;
        }
        // the ring's last releases have no reader: wait for every product before the CTA ends
        if (elect_one()) tc_commit(smem_u32(&sb->drain));
        __syncwarp();
#pragma unroll 1
        for (uint32_t i = 0; i < kPmWaitPolls && !mbar_try_wait(&sb->drain, 0); ++i) {}
        __syncwarp();
    } else {
        // ======================================== softmax: tile t, this thread's row
        const int t = warp >> 2;
        const int32_t row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kPmColS + t * 128, to = tmem + lanes + kPmColO + t * 128;
        const int32_t rtok = t * (U / 2) + (row >> lg);
        uint8_t *turn = smem + (2 + kPmStages) * kPmTileBytes + warp * kPmTurn;
        uint32_t ns = 0, no = 0;  // S tiles and O tiles taken
        bool ok = true;
        for (PromptItem z; ok && next_item(z);) {
            const int32_t e = t ? z.e1 : z.e0;
            const bool has_row = rtok < z.toks;
            // columns from this key tile on that the row sees (a row without a token, whose result nobody
            // takes, sees all: it must not send the warp through the hiding of columns)
            int32_t left = has_row ? z.see + rtok : 1 << 30;
            float m = -INFINITY, l = 0.0f;
            for (int32_t j = 0; j < e; ++j, left -= kPmTile) {
                if (!pm_wait(smem_u32(&sb->s_full[t]), ns & 1u, a.hdr)) { ok = false; break; }
                ++ns;
                tc_fence_after();
                const int32_t low = __reduce_min_sync(0xffffffffu, left);  // columns that all rows of the warp see
                // the row's maximum; the first 64 scores stay in registers, the others are read again
                // below (in tensor memory P overwrites the first 64 columns only)
                uint32_t x[64], y[32];
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto hide = [&](uint32_t *v, int c0) {  // 32 columns from c0 on, where some row does not see them all
                    if (low >= c0 + 32) return;
                    const int32_t n = left - c0;
                    const uint32_t keep = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(keep & (1u << c))) v[c] = 0xff800000u;  // -inf
                };
                auto maxima = [&](const uint32_t *v, int n) {
#pragma unroll
                    for (int c = 0; c < n; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[i] = max3(mx[i], __uint_as_float(v[c + 2 * i]), __uint_as_float(v[c + 2 * i + 1]));
                };
                tc_ld32(ts, x);
                tc_ld32(ts + 32, x + 32);
                tc_wait_ld();
                tc_ld32(ts + 64, y);
                hide(x, 0);
                hide(x + 32, 32);
                maxima(x, 64);
                tc_wait_ld();
                hide(y, 64);
                maxima(y, 32);
                tc_ld32(ts + 96, y);
                tc_wait_ld();
                hide(y, 96);
                maxima(y, 32);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool need = top > m + kPmLazy;
                float alpha = 1.0f;
                if (need) {
                    alpha = pm_ex2((m - top) * kPmScale);  // 0 from -inf
                    m = top;
                    l *= alpha;
                }
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    // O holds the earlier key tiles, complete before this S was
                    const uint64_t al = pack2(alpha, alpha);
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[16];
                        tc_ld16(to + 16 * c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float lo, hi;
                            unpack2(mul2(pack2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), al), lo, hi);
                            o[i] = __float_as_uint(lo);
                            o[i + 1] = __float_as_uint(hi);
                        }
                        tc_st16(to + 16 * c, o);
                    }
                }
                const float sc = fabsf(m) < kPmFar ? kPmScale : 0.125f;
                const float ref = m == -INFINITY ? 0.0f : -m * sc;
                const uint64_t sc2 = pack2(sc, sc), ref2 = pack2(ref, ref);
                uint64_t sum[2] = {0ull, 0ull};
                auto weights = [&](const uint32_t *v, int c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float lo, hi;
                        unpack2(fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, ref2), lo, hi);
                        lo = pm_ex2(lo);
                        hi = pm_ex2(hi);
                        sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(lo, hi));
                        p[i >> 1] = pm_pack_bf16(lo, hi);
                    }
                    tc_st16(ts + c / 2, p);
                };
                // three quarters of P first (y still holds columns 96 .. 127), announced on their own
                weights(y, 96);
                tc_ld32(ts + 64, y);
                weights(x, 0);
                weights(x + 32, 32);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sb->p_most[t]);
                tc_wait_ld();
                hide(y, 64);
                weights(y, 64);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sb->p_ready[t]);
                float lo, hi;
                unpack2(add2(sum[0], sum[1]), lo, hi);
                l += lo + hi;
            }
            if (!ok) break;
            // ---- the piece's end: the rows, or their part for the merge.  A thread has a row, so the warp
            // turns them through shared memory: eight lanes write 128 bytes of one row.  (Stored as they
            // lie, 16 bytes of 32 rows at a time, a tile took 4000 cycles.)
            const bool partial = z.slot >= 0;
            if (e > 0) {
                if (!pm_wait(smem_u32(&sb->o_full[t]), no & 1u, a.hdr)) break;
                ++no;
                tc_fence_after();
            }
            const int64_t prow = (int64_t)z.slot * kPmRows + t * kPmTile + (warp & 3) * 32;
            if (partial && has_row) __stcg(a.ml + prow + lane, make_float2(m, l));
            const float inv = l > 0.0f ? pm_rcp(l) : 0.0f;  // (a row that sees no key: its O is 0 too)
            uint8_t *mine = turn + lane * 128;  // 16-byte unit u of row r lies at unit u ^ r % 8
            const int u = lane & 7;
            if (!partial) {
                // this lane writes rows r0 + 4k, two steps of which are a whole number of tokens apart
                const int32_t r0 = (warp & 3) * 32 + (lane >> 3), tok0 = t * (U / 2) + (r0 >> lg);
                const int32_t tok_odd = 4 >> lg, tok_two = 8 >> lg;
                const int64_t row_odd = lg < 3 ? (int64_t)tok_odd * a.Hq * kD : 4 * kD, row_two = (int64_t)tok_two * a.Hq * kD;
                const uint8_t *from = turn + (lane >> 3) * 128;
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t o[32];
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        if ((v & 3) == 0) {
                            if (e > 0) {
                                tc_ld32(to + c + 8 * v, o);
                                tc_wait_ld();
                            } else {  // no key tile
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = 0u;
                            }
                        }
                        const int k = 8 * (v & 3);
                        uint4 w;
                        w.x = pm_pack_bf16(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv);
                        w.y = pm_pack_bf16(__uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
                        w.z = pm_pack_bf16(__uint_as_float(o[k + 4]) * inv, __uint_as_float(o[k + 5]) * inv);
                        w.w = pm_pack_bf16(__uint_as_float(o[k + 6]) * inv, __uint_as_float(o[k + 7]) * inv);
                        *reinterpret_cast<uint4 *>(mine + ((v ^ (lane & 7)) << 4)) = w;
                    }
                    __syncwarp();
                    uint4 w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        w[k] = *reinterpret_cast<const uint4 *>(from + k * 512 + ((u ^ ((4 * k + (lane >> 3)) & 7)) << 4));
                    uint16_t *out = a.out + (int64_t)((z.row + tok0) * a.Hq + z.h * G + (r0 & (G - 1))) * kD + u * 8 + c;
                    int32_t tok = tok0;
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        st_if(out, w[k], tok < z.toks);
                        st_if(out + row_odd, w[k + 1], tok + tok_odd < z.toks);
                        out += row_two;
                        tok += tok_two;
                    }
                }
            } else if (e > 0) {
                float *part = a.part + (prow + (lane >> 3)) * kD + u * 4;
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t o[32];
                    tc_ld32(to + c, o);
                    tc_wait_ld();
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        *reinterpret_cast<uint4 *>(mine + ((v ^ (lane & 7)) << 4)) =
                            make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    __syncwarp();
#pragma unroll 4
                    for (int k = 0; k < 8; ++k) {
                        const int r = 4 * k + (lane >> 3);
                        st_if(part + 4 * k * kD + c, *reinterpret_cast<const uint4 *>(turn + r * 128 + ((u ^ (r & 7)) << 4)),
                              t * (U / 2) + (((warp & 3) * 32 + r) >> lg) < z.toks);
                    }
                }
            }
            tc_fence_before();  // the reads of O above come before the next piece's first product
        }
    }
    __syncthreads();
    if (queued && tid == 0 && atomicAdd(&a.hdr->ended_ctas, 1u) + 1u == gridDim.x) {  // the last one: for the next call
        a.hdr->tickets = 0u;
        a.hdr->ended_ctas = 0u;
    }
    if (warp == kPmMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Merge of the units cut between CTAs: block (c, part) folds 32 rows of the unit whose first part is
// CTA c's last piece, in CTA order; a warp takes four rows, four columns per lane, and has the parts
// of kPmMergeDepth CTAs in flight.  Bound by the latency of its dependent reads, which grows with the
// parts of a unit (one per CTA at most): sixteen short turns behind up to 32768 tokens 11.1 us on its own,
// 7 us behind the last block when chained (eight rows a warp with one part in flight took 20 to 55).
constexpr int kPmMergeParts = 8, kPmMergeWarps = 8, kPmMergeDepth = 8;
constexpr int kPmMaxCtas = 1024;  // (c << 20 fits 32 bits in the slice search)

__global__ void __launch_bounds__(kPmMergeWarps * 32) prompt_merge_kernel(const PromptArgs a, int32_t ctas)
{
    __shared__ int32_t slots[kPmMaxCtas], s_count;
    pdl_wait_primary();
    const int4 head = __ldcg(a.head + blockIdx.x);
    if (head.x == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t G = a.G, U = kPmRows >> a.lg;
    if (warp == 0) {  // the unit's parts: this CTA's, then the next CTAs' first pieces up to the unit's end
        int32_t count = 1;
        if (lane == 0) slots[0] = 2 * blockIdx.x + (head.x - 1);
        for (int32_t c0 = blockIdx.x + 1; c0 < ctas; c0 += 32) {
            const int32_t c = c0 + lane;
            const int32_t flag = c < ctas ? __ldcg(a.cont + c) : 0;
            const uint32_t ends = __ballot_sync(0xffffffffu, flag == 2);
            const uint32_t upto = ends ? (ends & (0u - ends)) * 2u - 1u : 0xffffffffu;
            const uint32_t have = __ballot_sync(0xffffffffu, flag != 0) & upto;  // (a CTA may have no piece)
            if ((have >> lane) & 1u) slots[count + __popc(have & ((1u << lane) - 1u))] = 2 * c;
            count += __popc(have);
            if (ends) break;
        }
        if (lane == 0) s_count = count;
    }
    __syncthreads();
    const int32_t count = s_count;
    const PromptSeq s = prompt_seq(a, head.y, false);
    constexpr int kRows = kPmRows / kPmMergeParts / kPmMergeWarps;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int32_t row = blockIdx.y * (kPmRows / kPmMergeParts) + i * kPmMergeWarps + warp;
        const int32_t tok = head.w * U + (row >> a.lg);
        if (tok >= s.n) continue;
        float M = -INFINITY, L = 0.0f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t k0 = 0; k0 < count; k0 += kPmMergeDepth) {
            float2 ml[kPmMergeDepth];
            float4 o[kPmMergeDepth];
#pragma unroll
            for (int k = 0; k < kPmMergeDepth; ++k) {
                ml[k] = make_float2(-INFINITY, 0.0f);
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < count) {
                    const int64_t p = (int64_t)slots[k0 + k] * kPmRows + row;
                    ml[k] = __ldcg(a.ml + p);
                    o[k] = __ldcg(reinterpret_cast<const float4 *>(a.part + p * kD) + lane);
                }
            }
#pragma unroll
            for (int k = 0; k < kPmMergeDepth; ++k) {
                if (ml[k].x == -INFINITY) continue;  // no key of the part is seen by the row: it wrote no O
                const float Mn = fmaxf(M, ml[k].x);
                const float fo = M == -INFINITY ? 0.0f : pm_ex2((M - Mn) * kPmScale);
                const float fn = pm_ex2((ml[k].x - Mn) * kPmScale);
                L = L * fo + ml[k].y * fn;
                O.x = O.x * fo + o[k].x * fn;
                O.y = O.y * fo + o[k].y * fn;
                O.z = O.z * fo + o[k].z * fn;
                O.w = O.w * fo + o[k].w * fn;
                M = Mn;
            }
        }
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        uint2 w;
        w.x = pm_pack_bf16(O.x * inv, O.y * inv);
        w.y = pm_pack_bf16(O.z * inv, O.w * inv);
        reinterpret_cast<uint2 *>(a.out + ((int64_t)(s.q0 + tok) * a.Hq + head.z * G + (row & (G - 1))) * kD)[lane] = w;
    }
}

// ---- host -------------------------------------------------------------------------------------------

namespace {
struct PromptLayout {
    size_t off_head, off_cont, off_ml, off_part, total;
};
PromptLayout prompt_layout(int nsm)
{
    PromptLayout l;
    size_t off = sizeof(WsHeader);
    l.off_head = off;
    off = (off + (size_t)nsm * sizeof(int4) + 255) & ~size_t(255);
    l.off_cont = off;
    off = (off + (size_t)nsm * sizeof(int32_t) + 255) & ~size_t(255);
    l.off_ml = off;
    off += (size_t)nsm * 2 * kPmRows * sizeof(float2);
    l.off_part = off;
    off += (size_t)nsm * 2 * kPmRows * kD * sizeof(float);
    l.total = off;
    return l;
}
}  // namespace

size_t prompt_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int nsm)
{
    (void)B;
    (void)Hq;
    (void)Hkv;
    return prompt_layout(nsm).total;
}

cudaError_t launch_prompt(const void *q, const void *k, const void *v, int32_t total_q, int32_t total_kv,
                          const int32_t *cu_q, const int32_t *kv, const int32_t *bt, int32_t bs, int32_t max_blocks,
                          int32_t num_blocks, int32_t B, int32_t Hq, int32_t Hkv, void *out, void *ws, int nsm,
                          bool *map_failed, cudaStream_t stream)
{
    *map_failed = true;
    const int32_t G = Hq / Hkv;
    if (nsm > kPmMaxCtas) nsm = kPmMaxCtas;
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    PromptMaps maps;
    {
        // a tile's rows as two halves of 64 columns: (column, head, token, half) for Q, (column, token,
        // head, half) for packed K and V; (column, row) of one half of a page for the paged cache
        const cuuint32_t one[4] = {1, 1, 1, 1};
        const cuuint64_t qd[4] = {64, (cuuint64_t)Hq, (cuuint64_t)total_q, 2};
        const cuuint64_t qs[3] = {256, (cuuint64_t)Hq * 256, 128};
        const cuuint32_t qb[4] = {64, (cuuint32_t)G, (cuuint32_t)(kPmTile / G), 2};
        if (enc(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), qd, qs, qb, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
        const void *src[2] = {k, v};
        CUtensorMap *dst[2] = {&maps.k, &maps.v};
        for (int i = 0; i < 2; ++i) {
            CUresult r;
            if (bt) {
                const cuuint64_t d[2] = {kD, (cuuint64_t)num_blocks * Hkv * bs};
                const cuuint64_t st[1] = {256};
                const cuuint32_t box[2] = {64, (cuuint32_t)bs};
                r = enc(dst[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(src[i]), d, st, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            } else {
                // no keys at all: a map of one row that no copy reads
                const cuuint64_t d[4] = {64, (cuuint64_t)(total_kv > 0 ? total_kv : 1), (cuuint64_t)Hkv, 2};
                const cuuint64_t st[3] = {(cuuint64_t)Hkv * 256, 256, 128};
                const cuuint32_t box[4] = {64, kPmTile, 1, 2};
                r = enc(dst[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(total_kv > 0 ? src[i] : q), d, st,
                        box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            }
            if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
        }
    }
    *map_failed = false;

    const PromptLayout l = prompt_layout(nsm);
    char *base = static_cast<char *>(ws);
    PromptArgs a;
    a.out = static_cast<uint16_t *>(out);
    a.cu_q = cu_q;
    a.kv = kv;
    a.bt = bt;
    a.hdr = reinterpret_cast<WsHeader *>(base);
    a.head = reinterpret_cast<int4 *>(base + l.off_head);
    a.cont = reinterpret_cast<int32_t *>(base + l.off_cont);
    a.ml = reinterpret_cast<float2 *>(base + l.off_ml);
    a.part = reinterpret_cast<float *>(base + l.off_part);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.lg = __builtin_ctz((unsigned)G);  // (G is 1, 2, 4 or 8)
    a.total_q = total_q;
    a.total_kv = total_kv;
    a.bs = bs;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;

    static thread_local int limit_dev = -1;  // the shared-memory limit is raised once per device and host thread
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != limit_dev) {
        e = cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPmSmem);
        if (e != cudaSuccess) return e;
        limit_dev = dev;
    }
    prompt_kernel<<<(unsigned)nsm, kPmThreads, kPmSmem, stream>>>(a, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // no request has a unit that may be cut: nothing to merge
    if ((bt ? (int64_t)max_blocks * bs : (int64_t)total_kv) <= (2 * kPmSnap - 1) * kPmTile) return cudaSuccess;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nsm, kPmMergeParts);
    cfg.blockDim = dim3(kPmMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_merge_kernel, a, (int32_t)nsm);
}

}  // namespace dgq
