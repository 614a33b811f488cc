// Device and host helpers that the decode-step operators' sources share (lora_step.hip,
// lora_quant.hip, lora_sample.hip): 16-bit data, launches, the attention's split of rows over workgroups
// and the join of split rows, and the host's checks of arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "lora_internal.hpp"
#include "lora_step.h"

// As in the add-on's kernels, every fused multiply-add is an explicit __builtin_fmaf.
#pragma clang fp contract(off)

namespace lora {
namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------ launching
template <typename Kernel, typename... A>
void launch(Kernel kernel, dim3 grid, int threads, size_t lds, hipStream_t s, const A &...a)
{
    hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, s, a...);
}

int launch_status(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_E_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return LORA_OK;
}

// ------------------------------------------------------------------------ 16-bit data
struct F16 {
    typedef _Float16 elem;
};
struct BF16 {
    typedef __bf16 elem;
};
template <typename T>
using vec8 = typename T::elem __attribute__((ext_vector_type(8)));

template <typename T>
__device__ inline void unpack8(const uint4 &r, float (&f)[8])
{
    const vec8<T> v = __builtin_bit_cast(vec8<T>, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
}

// Rounds to nearest even.
template <typename T>
__device__ inline uint4 pack8(const float (&f)[8])
{
    vec8<T> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (typename T::elem)f[e];
    return __builtin_bit_cast(uint4, v);
}

__device__ inline uint4 load16(const void *base, int64_t elem)
{
    return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + elem);
}
__device__ inline void store16(void *base, int64_t elem, const uint4 &v)
{
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = v;
}

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
// With STREAM, a streaming store, for what is larger than the caches.
template <bool STREAM>
__device__ inline void store16(void *base, int64_t elem, const uint4 &v)
{
    if (STREAM)
        __builtin_nontemporal_store(__builtin_bit_cast(u4_t, v),
                                    reinterpret_cast<u4_t *>(static_cast<uint16_t *>(base) + elem));
    else store16(base, elem, v);
}

// Outputs of a call larger than this, the L2s of all XCDs together, are written with
// streaming stores: lines that the next call cannot find there anyway no longer displace
// what is being read.  Measured: rotary append of 4001 rows in the 70B layout (82 MB
// written) 41.7 -> 27.2 us, of 12,907 rows in the 7B layout (317 MB) 122 -> 114; residual
// norm of 12,907 rows of 4096 (211 MB) 74.7 -> 71.2.  Smaller outputs stay in the L2s for
// the call that reads them.
constexpr int64_t kStreamBytes = 32 << 20;

// ------------------------------------------------------------------------ attention
struct AttnArgs {
    int32_t n_rows, q_heads, kv_heads, head_dim, n_req, max_blocks, window, shift;
    int32_t group, head_tiles;  // query heads per key/value head; its 16-head tiles
    int32_t shares;             // workgroups per head tile
    float scale;
    void *out;
    const void *q;
    int64_t ldo, ldq, ld_table;
    const int32_t *table, *kv_len, *req;
    float *lse;
    uint32_t *count;          // arrivals of split rows' parts (zero between calls)
    float *part_ml, *part_o;  // their (m, l) and unnormalised sums
};

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// How a kernel splits its rows.
template <int WAVES, int TILE, int MIN_SHARE, int ROW_TILES, int ALIGN, bool SOLO, int BATCH, int ONCE>
struct AttnLine {
    static constexpr int kBatch = BATCH;         // parts that a join loads at a time
    static constexpr int kOnce = ONCE;           // parts that are joined in one step; more in groups of kAttnJoin first
    static constexpr int kAlign = ALIGN;         // a row's first tile begins at a multiple of this (a power of two)
    static constexpr bool kSolo = SOLO;          // a wavefront has a share of its own, and not its workgroup
    static constexpr int kWaves = SOLO ? 1 : WAVES;  // wavefronts that work on one
    static constexpr int kTile = TILE;           // tokens a wavefront takes at a time
    static constexpr int kMinShare = MIN_SHARE;  // tiles a workgroup takes at least: one per wavefront
    static constexpr int kRowTiles = ROW_TILES;  // what starting and finishing a row costs, in tiles
};
constexpr int kAttnJoin = 16;        // parts joined at a time
constexpr int kAttnMaxTiles = 4096;  // key/value heads x 16-head tiles of one launch
constexpr int kAttnCUs = 256;
constexpr int32_t kAttnMaxSpan = 1 << 30;  // tokens of a table row: positions and steps past them fit 32 bits
// Arrival counters: two part slots per workgroup, and at most 4 workgroups per CU or one
// per head tile.  They lie first in a workspace, at one size for every shape, so calls of
// different shapes sharing a workspace never put sums where another finds its counters.
constexpr size_t kAttnCounters = 2 * (4 * kAttnCUs + kAttnMaxTiles);

// Visible tokens [first, first + span) of row i (from a multiple of kAlign on); span -1: the row is not active, or none.
struct RowSpan {
    int32_t req, first, span;
};

template <typename LINE>
__device__ inline RowSpan row_span(const AttnArgs &a, int32_t i)
{
    const int32_t at = min(i, a.n_rows - 1);  // loads without a branch, so many can be in flight
    const int32_t n = a.kv_len[at], r = a.req ? a.req[at] : at;
    const bool on = i < a.n_rows && n >= 0 && n <= a.max_blocks << a.shift && r >= 0 && r < a.n_req;
    const int32_t first = a.window > 0 && n > a.window ? (n - a.window) & -LINE::kAlign : 0;
    return RowSpan{r, first, on ? n - first : -1};
}

// The schedule of a launch, found by every workgroup from the lengths on the device.  Each
// active row costs its visible tokens in tiles (at least one) and kRowTiles
// more; the rows' costs are laid end to end, and workgroup w takes [w share, (w + 1) share)
// of them: parts of one or more rows, the same amount of work in every workgroup whatever
// the lengths.  Row i's tiles lie at [tile0, tile0 + tiles) of that line.
struct RowWork {
    int32_t row, tile0, tiles;
    RowSpan rs;
};

template <typename LINE>
__device__ inline int32_t row_tiles(const RowSpan &rs)
{
    return rs.span < 0 ? 0 : rs.span <= LINE::kTile ? 1 : (rs.span - 1) / LINE::kTile + 1;
}

// Inclusive prefix sum over the wavefront: within rows of sixteen lanes, then across them.
__device__ inline int32_t wave_scan(int32_t v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

// A wavefront's walk over the rows of a launch, 64 of them in its lanes at a time.
template <typename LINE>
struct RowWalk {
    int32_t base;   // the lanes hold rows base .. base + 63
    RowSpan rs;     // lane's row
    int32_t tiles;

    __device__ inline void load(const AttnArgs &a, int32_t b)
    {
        base = b;
        rs = row_span<LINE>(a, b + (int32_t)(threadIdx.x & 63));
        tiles = row_tiles<LINE>(rs);
    }
    __device__ inline RowWork row(int lane, int32_t tile0) const
    {
        return RowWork{base + lane, tile0, __builtin_amdgcn_readlane(tiles, lane),
                       RowSpan{__builtin_amdgcn_readlane(rs.req, lane), __builtin_amdgcn_readlane(rs.first, lane),
                               __builtin_amdgcn_readlane(rs.span, lane)}};
    }
    // The next active row behind row r, at position tile0 of the line (row n_rows: none).
    __device__ inline RowWork after(const AttnArgs &a, int32_t r, int32_t tile0)
    {
        uint64_t on = r + 1 - base < 64 ? __ballot(tiles > 0) & (~(uint64_t)0 << (r + 1 - base)) : 0;
        while (!on && base + 64 < a.n_rows) {
            load(a, base + 64);
            on = __ballot(tiles > 0);
        }
        return on ? row(__builtin_ctzll(on), tile0) : RowWork{a.n_rows, 0, 0, RowSpan{0, 0, -1}};
    }
};

// The first row with work at or behind position w * share (row n_rows: none), the share and
// the line's length.  Every wavefront finds it for itself, so nothing waits on a barrier;
// the host has checked that the line fits 32 bits.
template <typename LINE>
__device__ inline RowWork first_row(const AttnArgs &a, int32_t w, RowWalk<LINE> &walk, int32_t &share, int32_t &total)
{
    const int lane = threadIdx.x & 63;
    walk.load(a, 0);
    int32_t sum = walk.tiles > 0 ? walk.tiles + LINE::kRowTiles : 0;
#pragma unroll 8
    for (int32_t c = 64; c < a.n_rows; c += 64) {
        const int32_t t = row_tiles<LINE>(row_span<LINE>(a, c + lane));
        sum += t > 0 ? t + LINE::kRowTiles : 0;
    }
    total = __builtin_amdgcn_readlane(wave_scan(sum), 63);
    share = max((total + a.shares - 1) / a.shares, LINE::kMinShare);
    const int64_t begin = (int64_t)w * share;
    int32_t at0 = 0;
    while (begin < total) {
        const int32_t cost = walk.tiles > 0 ? walk.tiles + LINE::kRowTiles : 0, end = at0 + wave_scan(cost);
        const uint64_t here = __ballot(end - cost <= begin && begin < end);
        if (here) {
            const int l = __builtin_ctzll(here);
            return walk.row(l, __builtin_amdgcn_readlane(end - walk.tiles, l));
        }
        at0 = __builtin_amdgcn_readlane(end, 63);
        if (walk.base + 64 >= a.n_rows) break;
        walk.load(a, walk.base + 64);
    }
    return RowWork{a.n_rows, 0, 0, RowSpan{0, 0, -1}};
}

__device__ inline f4_t mfma(const vec8<F16> &x, const vec8<F16> &y, const f4_t &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
}
__device__ inline f4_t mfma(const vec8<BF16> &x, const vec8<BF16> &y, const f4_t &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}

// A weight p in [0, 2^kBias] as two 16-bit parts, hi + lo, both cut off (never rounded up)
// and neither 0, so that hi * v + lo * v is what p * v is for an infinite v too.  fp16 keeps
// 22 bits (the bias lifts weights out of its subnormals, whose step is 2^-38 of the largest
// weight; a weight of 0 counts as two such steps), bf16 16 bits: both far below the
// rounding of the output.  The steps add up: n tokens of weights near or below them put an
// fp16 output off by up to n 2^-37 max |v|, 2^-20 max |v| at 131,072 tokens, half an fp16
// step of it (2^-11) at 2^26.
template <typename T>
struct Weight;
template <>
struct Weight<F16> {
    static constexpr float kBias = 14.f;
    static __device__ inline void split(float p0, float p1, uint32_t &hi, uint32_t &lo)
    {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 h = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(p0, p1));
        hi = at_least(__builtin_bit_cast(uint32_t, h));
        lo = at_least(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(p0 - (float)h[0], p1 - (float)h[1])));
    }
    static __device__ inline uint32_t at_least(uint32_t x)
    {
        typedef unsigned short u2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2, x), u2{1, 1}));
    }
};
template <>
struct Weight<BF16> {
    static constexpr float kBias = 0.f;
    static __device__ inline void split(float p0, float p1, uint32_t &hi, uint32_t &lo)
    {
        const uint32_t a = __builtin_bit_cast(uint32_t, p0), b = __builtin_bit_cast(uint32_t, p1);
        const float r0 = p0 - __builtin_bit_cast(float, a & 0xffff0000u), r1 = p1 - __builtin_bit_cast(float, b & 0xffff0000u);
        hi = at_least((a >> 16) | (b & 0xffff0000u));
        lo = at_least((__builtin_bit_cast(uint32_t, r0) >> 16) | (__builtin_bit_cast(uint32_t, r1) & 0xffff0000u));
    }
    static __device__ inline uint32_t at_least(uint32_t x)
    {
        typedef unsigned short u2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2, x), u2{0x80, 0x80}));
    }
};

// Four columns of a finished row: sum / l, rounded once; an empty row is 0.
template <typename T>
__device__ inline void write_row(const AttnArgs &a, int64_t row, int64_t head, int d, const f4_t &sum, float m, float l)
{
    typedef typename T::elem E;
    typedef E e4 __attribute__((ext_vector_type(4)));
    const bool none = l == 0.f;
    e4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (E)(none ? 0.f : sum[e] / l);
    *reinterpret_cast<e4 *>(static_cast<E *>(a.out) + row * a.ldo + head * a.head_dim + d) = r;
    if (a.lse && d == 0)
        a.lse[row * a.q_heads + head] = none ? -INFINITY : (m + (__builtin_log2f(l) - Weight<T>::kBias)) * kLn2;
}

// A split row's sums pass between workgroups of different XCDs, whose L2s are not coherent:
// they are stored and loaded device-coherently (relaxed atomics of device scope, which the
// hardware takes past the local L2), ordered by the waits in last_arrival.  Fences of
// device scope instead write back and invalidate a whole L2 each: measured on the 7B
// decode batch, 393 us against 120.
__device__ inline void put_part(float *p, float x, float y)
{
    const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, y) << 32 | __builtin_bit_cast(uint32_t, x);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float2 get_part(const float *p)
{
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}

// Waits for those that work on one share.
template <typename LINE>
__device__ inline void line_sync()
{
    if constexpr (LINE::kSolo) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        __syncthreads();
    }
}

// True in the workgroup (or, alone, wavefront) that is the n-th to come here with this counter, which is then 0
// again.  Every wavefront waits for its own stores to complete before the workgroup
// counts itself, so the last one's loads find all parts.
template <typename LINE>
__device__ inline bool last_arrival(uint32_t *count, int n)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (LINE::kSolo) {
        uint32_t before = 0;
        if ((threadIdx.x & 63) == 0) {
            before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (before == (uint32_t)(n - 1)) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        const bool last = __builtin_amdgcn_readfirstlane(before) == (uint32_t)(n - 1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        return last;
    } else {
        __shared__ bool last;
        __syncthreads();
        if (threadIdx.x == 0) {
            last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
            if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        return last;
    }
}

// Slot of part p of a row whose first part is in workgroup w0: a workgroup has one slot for
// the row it found begun and one for the row it leaves unfinished.
__device__ inline int32_t part_slot(int32_t w0, int32_t p) { return p == 0 ? 2 * w0 + 1 : 2 * (w0 + p); }

// Adds n parts (part0, part0 + step, ...) of a split row's heads, in that order, into part0's
// slot, or with `finish` into the row.
template <typename T, typename LINE>
__device__ inline void join_parts(const AttnArgs &a, int32_t row, int32_t w0, int64_t head0, int heads, int part0,
                                  int step, int n, bool finish)
{
    __shared__ float2 joined_all[LINE::kSolo ? 16 : 1][16];  // (a workgroup has sixteen wavefronts at most)
    float2 *const joined = joined_all[LINE::kSolo ? threadIdx.x >> 6 : 0];
    constexpr int kBatch = LINE::kBatch;
    const int cols = a.head_dim / 4, tid = LINE::kSolo ? threadIdx.x & 63 : threadIdx.x;
    for (int i0 = 0; i0 < heads * cols; i0 += 64 * LINE::kWaves) {
        const int i = i0 + tid;
        const bool on = i < heads * cols;
        const int h = on ? i / cols : 0, d = on ? 4 * (i - h * cols) : 0;
        // kBatch parts at a time, all their loads in flight together
        float m = -INFINITY, l = 0.f;
        f4_t sum = f4_t{0.f, 0.f, 0.f, 0.f};
        for (int p0 = 0; p0 < n; p0 += kBatch) {
            float2 v[kBatch], x[kBatch], y[kBatch];
#pragma unroll
            for (int p = 0; p < kBatch; ++p) {
                const int64_t at = (int64_t)part_slot(w0, part0 + min(p0 + p, n - 1) * step) * a.q_heads + head0 + h;
                v[p] = get_part(&a.part_ml[2 * at]);
                x[p] = get_part(&a.part_o[at * a.head_dim + d]);
                y[p] = get_part(&a.part_o[at * a.head_dim + d + 2]);
            }
            float mx = m;
#pragma unroll
            for (int p = 0; p < kBatch; ++p) mx = __builtin_fmaxf(mx, v[p].x);
            const float base = mx == -INFINITY ? 0.f : mx, keep = __builtin_amdgcn_exp2f(m - base);
            l *= keep;
            sum *= keep;
            m = mx;
#pragma unroll
            for (int p = 0; p < kBatch; ++p) {
                const bool in = p0 + p < n;  // past the end the last part is read again, and not added
                const float f = __builtin_amdgcn_exp2f(v[p].x - base);
                l = in ? __builtin_fmaf(v[p].y, f, l) : l;
                const f4_t more = sum + f4_t{x[p].x, x[p].y, y[p].x, y[p].y} * f;
                sum = in ? more : sum;
            }
        }
        if (!on) continue;
        if (finish) {
            write_row<T>(a, row, head0 + h, d, sum, m, l);
        } else {
            const int64_t slot = (int64_t)part_slot(w0, part0) * a.q_heads + head0 + h;
            put_part(&a.part_o[slot * a.head_dim + d], sum[0], sum[1]);  // these columns are read by this lane only
            put_part(&a.part_o[slot * a.head_dim + d + 2], sum[2], sum[3]);
            if (d == 0) joined[h] = make_float2(m, l);
        }
    }
    if (finish) return;
    line_sync<LINE>();  // every lane has read its heads' (m, l) of part0
    if (tid < heads)
        put_part(&a.part_ml[2 * ((int64_t)part_slot(w0, part0) * a.q_heads + head0 + tid)], joined[tid].x, joined[tid].y);
}

// The part `part` of a split row is stored: of every kAttnJoin parts, the workgroup that
// arrives last adds them up in order into the first one's slot; of those sums, the last
// arrival adds all and writes the row.  Who that is does not change what is added in which
// order.
template <typename T, typename LINE>
__device__ inline void join_row(const AttnArgs &a, int32_t row, int32_t w0, int32_t parts, int32_t part, int per_share,
                                int rest, int64_t head0, int heads)
{
    const int width = parts <= LINE::kOnce ? parts : kAttnJoin;
    const int group0 = part / width * width, n_groups = (parts + width - 1) / width;
    const int in_group = min(width, parts - group0);
    if (!last_arrival<LINE>(a.count + (int64_t)part_slot(w0, group0) * per_share + rest, in_group)) return;
    join_parts<T, LINE>(a, row, w0, head0, heads, group0, 1, in_group, n_groups == 1);
    // (part 1 leads no group, so its counter is free for the groups)
    if (n_groups == 1 || !last_arrival<LINE>(a.count + (int64_t)part_slot(w0, 1) * per_share + rest, n_groups)) return;
    join_parts<T, LINE>(a, row, w0, head0, heads, 0, kAttnJoin, n_groups, true);
}

int32_t attn_tiles(int32_t q_heads, int32_t kv_heads)
{
    return (int32_t)std::min<int64_t>((int64_t)kv_heads * ((q_heads / kv_heads + 15) / 16), INT32_MAX);
}

// ------------------------------------------------------------------------ host checks
int page_shift(int32_t page_size)
{
    if (page_size < 1 || page_size > LORA_KV_MAX_PAGE || (page_size & (page_size - 1))) return -1;
    return __builtin_ctz((unsigned)page_size);
}

int check_type(int32_t type)
{
    if (type != LORA_TYPE_F16 && type != LORA_TYPE_BF16) return fail(LORA_E_UNSUPPORTED, "unknown type %d", type);
    return LORA_OK;
}

int check_matrix(const void *p, int64_t ld, int64_t cols, const char *name)
{
    if (!p) return fail(LORA_E_NULL, "%s is NULL", name);
    if (!aligned16(p)) return fail(LORA_E_ALIGN, "%s must be 16-byte aligned", name);
    if (ld < cols) return fail(LORA_E_SHAPE, "leading dimension of %s = %lld < %lld", name, (long long)ld, (long long)cols);
    if (ld % 8) return fail(LORA_E_ALIGN, "leading dimension of %s = %lld is not a multiple of 8", name, (long long)ld);
    return LORA_OK;
}

// An output and another matrix of n_rows rows of 16-bit elements share no element, unless
// they are the very same one and `same_ok`.  Column slices of one product (equal leading
// dimensions) may lie between each other's rows.
int check_apart(const void *out, int64_t ldo, int64_t cols_o, const void *in, int64_t ldi, int64_t cols_i,
                int64_t n_rows, bool same_ok, const char *what)
{
    if (!out || !in) return LORA_OK;
    if (same_ok && out == in && ldo == ldi) return LORA_OK;
    const int64_t o = (int64_t)reinterpret_cast<uintptr_t>(out), i = (int64_t)reinterpret_cast<uintptr_t>(in);
    if (o >= i + 2 * ((n_rows - 1) * ldi + cols_i) || i >= o + 2 * ((n_rows - 1) * ldo + cols_o)) return LORA_OK;
    if (ldo == ldi) {
        const int64_t d = (i - o) / 2 % ldo, off = d < 0 ? d + ldo : d;  // in's first column, counted from out's
        if (off >= cols_o && off + cols_i <= ldo) return LORA_OK;
    }
    return fail(LORA_E_SHAPE, "%s overlap", what);
}

// A launch of one workgroup per row has at most 2^32 - 1 threads along its rows, which may be rounded up by `more`.
int check_rows(int32_t n_rows, int threads, int more = 0)
{
    if (((int64_t)n_rows + more) * threads > UINT32_MAX)
        return fail(LORA_E_UNSUPPORTED, "%d rows of %d threads are too many for one launch", n_rows, threads);
    return LORA_OK;
}

// A rotary embedding of heads of head_dim columns.
int check_rope(const lora_rope *rope, int32_t head_dim)
{
    if (!rope) return fail(LORA_E_NULL, "rope descriptor is NULL");
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > head_dim)
        return fail(LORA_E_SHAPE, "rot_dim = %d is not a multiple of 16 in 0..head_dim = %d", rope->rot_dim, head_dim);
    if (rope->n_axes < 1 || rope->n_axes > LORA_ROPE_MAX_AXES)
        return fail(LORA_E_SHAPE, "n_axes = %d outside 1..%d", rope->n_axes, LORA_ROPE_MAX_AXES);
    if ((rope->interleaved != 0 && rope->interleaved != 1) || rope->reserved != 0)
        return fail(LORA_E_SHAPE, "interleaved = %d, reserved = %d", rope->interleaved, rope->reserved);
    return LORA_OK;
}

// An append's other arguments; the pointers only where there are rows.
int check_append(int32_t n_rows, int32_t q_heads, const void *q_out, int64_t ldqo, const void *q, int64_t ldq,
                 const void *k, int64_t ldk, const void *v, int64_t ldv, const lora_rope *rope, const int32_t *positions,
                 int64_t ld_pos, const int32_t *slots, int32_t kv_heads, int32_t head_dim)
{
    int st;
    if (n_rows < 0 || q_heads < 0) return fail(LORA_E_SHAPE, "n_rows = %d, q_heads = %d", n_rows, q_heads);
    if ((int64_t)q_heads + kv_heads > 1 << 20)
        return fail(LORA_E_UNSUPPORTED, "%d query and %d key/value heads", q_heads, kv_heads);
    if (n_rows == 0) return LORA_OK;
    const int64_t kv_cols = (int64_t)kv_heads * head_dim, cols = (int64_t)q_heads * head_dim;
    if (q_heads > 0) {
        if ((st = check_matrix(q, ldq, cols, "q"))) return st;
        if ((st = check_matrix(q_out, ldqo, cols, "q_out"))) return st;
    }
    if ((st = check_matrix(k, ldk, kv_cols, "k"))) return st;
    if ((st = check_matrix(v, ldv, kv_cols, "v"))) return st;
    if (q_heads > 0) {
        if ((st = check_apart(q_out, ldqo, cols, q, ldq, cols, n_rows, true, "q_out and q"))) return st;
        if ((st = check_apart(q_out, ldqo, cols, k, ldk, kv_cols, n_rows, false, "q_out and k"))) return st;
        if ((st = check_apart(q_out, ldqo, cols, v, ldv, kv_cols, n_rows, false, "q_out and v"))) return st;
    }
    if (!slots) return fail(LORA_E_NULL, "slots is NULL");
    if (rope->rot_dim > 0) {
        if (!positions || !rope->inv_freq) return fail(LORA_E_NULL, "positions and inv_freq are required");
        if (ld_pos < n_rows) return fail(LORA_E_SHAPE, "ld_pos = %lld < %d rows", (long long)ld_pos, n_rows);
    }
    return LORA_OK;
}

// An attention's arguments beside its cache; the pointers only where there are rows.
int check_attention(int32_t n_rows, int32_t q_heads, const void *out, int64_t ldo, const void *q, int64_t ldq,
                    int32_t n_req, const int32_t *block_table, int64_t ld_table, int32_t max_blocks,
                    const int32_t *kv_len, float scale, int32_t window, const float *lse, const void *work,
                    size_t work_bytes, int32_t kv_heads, int32_t head_dim, int32_t page_size, size_t need)
{
    int st;
    if (n_rows < 0 || n_req < 0) return fail(LORA_E_SHAPE, "n_rows = %d, n_req = %d", n_rows, n_req);
    if (q_heads < 1 || q_heads % kv_heads)
        return fail(LORA_E_SHAPE, "q_heads = %d is not a multiple of kv_heads = %d", q_heads, kv_heads);
    if (max_blocks < 1 || ld_table < max_blocks || (int64_t)max_blocks * page_size > kAttnMaxSpan)
        return fail(LORA_E_SHAPE, "max_blocks = %d of %d tokens, ld_table = %lld", max_blocks, page_size, (long long)ld_table);
    if (window < 0) return fail(LORA_E_SHAPE, "window = %d", window);
    if (!std::isfinite(scale)) return fail(LORA_E_SHAPE, "scale is not finite");
    if ((int64_t)n_rows * q_heads > (int64_t)1 << 30)
        return fail(LORA_E_SHAPE, "%d rows of %d heads are too many for one launch", n_rows, q_heads);
    if (attn_tiles(q_heads, kv_heads) > kAttnMaxTiles)
        return fail(LORA_E_UNSUPPORTED, "%d key/value heads of %d query heads", kv_heads, q_heads);
    if (n_rows == 0) return LORA_OK;
    const int64_t cols = (int64_t)q_heads * head_dim;
    if ((st = check_matrix(q, ldq, cols, "q"))) return st;
    if ((st = check_matrix(out, ldo, cols, "out"))) return st;
    if ((st = check_apart(out, ldo, cols, q, ldq, cols, n_rows, false, "out and q"))) return st;
    if (!kv_len || (n_req > 0 && !block_table)) return fail(LORA_E_NULL, "kv_len and block_table are required");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) return fail(LORA_E_ALIGN, "lse must be 4-byte aligned");
    if (!work) return fail(LORA_E_NULL, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(work) & 255) return fail(LORA_E_ALIGN, "workspace must be 256-byte aligned");
    if (work_bytes < need) return fail(LORA_E_SHAPE, "workspace of %zu bytes < %zu for %d rows", work_bytes, need, n_rows);
    return LORA_OK;
}

// The kernel's arguments of a call that passed the checks, for at most `most` shares.
template <typename LINE>
int fill_attention(AttnArgs &a, int32_t n_rows, int32_t q_heads, void *out, int64_t ldo, const void *q, int64_t ldq,
                   int32_t n_req, const int32_t *block_table, int64_t ld_table, int32_t max_blocks,
                   const int32_t *kv_len, const int32_t *req, float scale, int32_t window, float *lse, void *work,
                   int32_t kv_heads, int32_t head_dim, int32_t page_size, int32_t most)
{
    a.n_rows = n_rows;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.n_req = n_req;
    a.max_blocks = max_blocks;
    a.window = window;
    a.shift = page_shift(page_size);
    a.group = q_heads / kv_heads;
    a.head_tiles = (a.group + 15) / 16;
    // no row is longer than its table or the window, and no share shorter than kMinShare
    const int64_t span = std::min<int64_t>((int64_t)max_blocks * page_size, window > 0 ? (int64_t)window + LINE::kAlign - 1 : INT32_MAX);
    const int64_t line = n_rows * ((span + LINE::kTile - 1) / LINE::kTile + LINE::kRowTiles);
    if (line > INT32_MAX - most)  // (rounded up to whole shares)
        return fail(LORA_E_UNSUPPORTED, "%d rows of up to %lld tokens", n_rows, (long long)span);
    a.shares = (int32_t)std::min<int64_t>(most, (line + LINE::kMinShare - 1) / LINE::kMinShare);
    a.scale = scale;
    a.out = out;
    a.q = q;
    a.ldo = ldo;
    a.ldq = ldq;
    a.ld_table = ld_table;
    a.table = block_table;
    a.kv_len = kv_len;
    a.req = req;
    a.lse = lse;
    a.count = static_cast<uint32_t *>(work);
    a.part_o = reinterpret_cast<float *>(a.count + kAttnCounters);
    a.part_ml = a.part_o + 2 * (size_t)most * q_heads * head_dim;
    return LORA_OK;
}

// Workgroups of `per` shares each.
dim3 attention_grid(const AttnArgs &a, int per = 1)
{
    const int32_t pairs = (a.shares * a.kv_heads + per - 1) / per;
    return dim3((unsigned)(a.head_tiles > 1 ? (pairs + 7) / 8 * 8 * a.head_tiles : pairs));
}

}  // namespace
}  // namespace lora
