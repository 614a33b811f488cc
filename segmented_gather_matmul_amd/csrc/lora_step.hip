// HIP kernels (gfx950 / CDNA4) and launchers of the decode-step operators beside the
// add-on: the step plan, rotary positions with the append to the paged cache, attention
// over that cache, and the residual add with its norms (lora_step.h).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "lora_launch.hpp"
#include "lora_step.h"

// As in the add-on's kernels, every fused multiply-add is an explicit __builtin_fmaf.
#pragma clang fp contract(off)

namespace lora {
namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));

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

// ------------------------------------------------------------------------ step plan
struct PlanArgs {
    lora_kv_pages pg;
    lora_kv_plan_out out;
    const int32_t *kv_len, *new_len, *req_slot;
    int32_t shift;    // log2(page_size)
    int32_t maps;     // the first kernel writes the token maps too
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanMapsHere = 4096;  // token rows up to which the planning workgroup writes the maps itself

// One request of a plan; `bad` holds its LORA_KV_* bits.
struct PlanReq {
    int32_t len, add, had, grown, given, bad;
    int64_t end;
};

__device__ inline PlanReq plan_req(const PlanArgs &a, int r)
{
    PlanReq q{};
    if (r >= a.pg.n_req) return q;
    q.len = a.kv_len[r];
    const int32_t nl = a.new_len[r];
    if (q.len < 0 || nl < -1) {
        q.bad = LORA_KV_INVALID;
        return q;
    }
    q.add = nl > 0 ? nl : 0;
    const int64_t end = (int64_t)q.len + q.add;
    if (end > (int64_t)a.pg.max_blocks << a.shift) q.bad = LORA_KV_TOO_LONG;
    const int64_t mask = ((int64_t)1 << a.shift) - 1;
    q.had = (int32_t)((q.len + mask) >> a.shift);
    if (nl < 0) {
        q.given = q.had;
    } else {
        q.end = end;
        q.grown = (int32_t)(((end + mask) >> a.shift) - q.had);
    }
    return q;
}

// Exclusive prefix of v over the workgroup, and the total, in 32 bits.
__device__ inline int32_t block_scan(int32_t v, int32_t *wave_sums, int32_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t up = __shfl_up(s, d);
        if (lane >= d) s += up;
    }
    __syncthreads();  // wave_sums may still be read from the call before
    if (lane == 63) wave_sums[wave] = s;
    __syncthreads();
    int32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        const int32_t x = wave_sums[w];
        before += w < wave ? x : 0;
        all += x;
    }
    total = all;
    return before + s - v;
}

// Last index i in [0, n) with off[i] <= k (off[0] <= k, off non-decreasing).
__device__ inline int last_at_most(const int32_t *off, int n, int32_t k)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ inline void plan_map_row(const PlanArgs &a, int32_t t, int32_t r, int32_t pos, int32_t page)
{
    const lora_kv_plan_out &o = a.out;
    const bool ok = r >= 0 && page >= 0 && page < a.pg.num_pages;  // a table entry that is no page: no slot
    o.tok_req[t] = r;
    o.tok_pos[t] = pos;
    o.slots[t] = ok ? (page << a.shift) | (pos & ((1 << a.shift) - 1)) : -1;
    if (o.idx) o.idx[t] = r < 0 || !a.req_slot ? -1 : a.req_slot[r];
}

// The plan proper, in one workgroup: totals and checks over all requests first (all or
// nothing), then, 1024 requests at a time, the pages of ended requests onto the free
// list, and after all of those the pages of growing ones off it.  A chunk's work is spread over
// the workgroup by page and by token, each found by a binary search in the chunk's
// prefix sums.
__global__ __launch_bounds__(kPlanThreads) void lora_kv_plan_kernel(PlanArgs a)
{
    __shared__ int32_t wave_sums[kPlanWaves];
    __shared__ int64_t sums[kPlanWaves][3];
    __shared__ int32_t bits;
    __shared__ int32_t off[kPlanThreads], had_s[kPlanThreads], off_tok[kPlanThreads], len_s[kPlanThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t n = a.pg.n_req;
    if (tid == 0) bits = 0;
    __syncthreads();
    // totals
    int64_t tokens = 0, taken = 0, given = 0;
    int32_t bad = 0;
    for (int32_t r = tid; r < n; r += kPlanThreads) {
        const PlanReq q = plan_req(a, r);
        bad |= q.bad;
        tokens += q.add;
        taken += q.grown;
        given += q.given;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        tokens += __shfl_xor(tokens, d);
        taken += __shfl_xor(taken, d);
        given += __shfl_xor(given, d);
        bad |= __shfl_xor(bad, d);
    }
    if (lane == 0) {
        sums[wave][0] = tokens;
        sums[wave][1] = taken;
        sums[wave][2] = given;
        if (bad) atomicOr(&bits, bad);
    }
    const int32_t top0 = *a.pg.free_top;
    __syncthreads();
    tokens = taken = given = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        tokens += sums[w][0];
        taken += sums[w][1];
        given += sums[w][2];
    }
    bad = bits;
    if (top0 < 0 || top0 > a.pg.num_pages || top0 + given > a.pg.num_pages) bad |= LORA_KV_INVALID;
    if (taken > top0 + given) bad |= LORA_KV_NO_PAGES;
    if (tokens > a.out.max_tokens) bad |= LORA_KV_TOO_MANY;
    if (tid == 0) {
        const int64_t most = INT32_MAX;
        a.out.status[0] = bad;
        a.out.status[1] = (int32_t)(tokens < most ? tokens : most);
        a.out.status[2] = (int32_t)(taken < most ? taken : most);
        a.out.status[3] = (int32_t)(given < most ? given : most);
        a.out.free_top[0] = bad ? top0 : (int32_t)(top0 + given - taken);
        a.out.q_ptr[n] = bad ? 0 : (int32_t)tokens;
    }
    if (bad) {
        for (int32_t r = tid; r < n; r += kPlanThreads) {
            a.out.kv_end[r] = a.kv_len[r];
            a.out.q_ptr[r] = 0;
        }
        if (a.maps)
            for (int32_t t = tid; t < a.out.max_tokens; t += kPlanThreads) plan_map_row(a, t, -1, -1, 0);
        return;
    }
    // pages of ended requests go on top of the free list
    if (given > 0) {
        int32_t at = top0;
        for (int32_t c = 0; c < n; c += kPlanThreads) {
            const PlanReq q = plan_req(a, c + tid);
            int32_t total;
            const int32_t before = block_scan(q.given, wave_sums, total);
            off[tid] = before;
            __syncthreads();
            for (int32_t k = tid; k < total; k += kPlanThreads) {
                const int i = last_at_most(off, kPlanThreads, k);
                a.pg.free_pages[at + k] = a.pg.block_table[(int64_t)(c + i) * a.pg.ld_table + (k - off[i])];
            }
            at += total;
        }
        __syncthreads();  // the list is read below by other threads of this workgroup
    }
    // growing requests and the token maps
    int32_t at = (int32_t)(top0 + given) - 1, row0 = 0;
    for (int32_t c = 0; c < n; c += kPlanThreads) {
        const PlanReq q = plan_req(a, c + tid);
        int32_t pages, rows;
        const int32_t before = block_scan(q.grown, wave_sums, pages);
        const int32_t before_tok = block_scan(q.add, wave_sums, rows);
        off[tid] = before;
        had_s[tid] = q.had;
        off_tok[tid] = before_tok;
        len_s[tid] = q.len;
        if (c + tid < n) {
            a.out.q_ptr[c + tid] = row0 + before_tok;
            a.out.kv_end[c + tid] = (int32_t)q.end;
        }
        __syncthreads();
        for (int32_t k = tid; k < pages; k += kPlanThreads) {
            const int i = last_at_most(off, kPlanThreads, k);
            a.pg.block_table[(int64_t)(c + i) * a.pg.ld_table + had_s[i] + (k - off[i])] = a.pg.free_pages[at - k];
        }
        if (a.maps) {
            for (int32_t k = tid; k < rows; k += kPlanThreads) {
                const int i = last_at_most(off_tok, kPlanThreads, k);
                const int32_t pos = len_s[i] + (k - off_tok[i]), b = pos >> a.shift;
                const int32_t page = b < had_s[i] ? a.pg.block_table[(int64_t)(c + i) * a.pg.ld_table + b]
                                                  : a.pg.free_pages[at - (off[i] + b - had_s[i])];
                plan_map_row(a, row0 + k, c + i, pos, page);
            }
        }
        at -= pages;
        row0 += rows;
        __syncthreads();
    }
    if (a.maps)
        for (int32_t t = row0 + tid; t < a.out.max_tokens; t += kPlanThreads) plan_map_row(a, t, -1, -1, 0);
}

// Token maps of a step with many rows, one row per thread, from what the plan left: q_ptr
// (searched), kv_end and the table.
__global__ __launch_bounds__(256) void lora_kv_maps_kernel(PlanArgs a)
{
    const int32_t t = blockIdx.x * 256 + threadIdx.x;
    if (t >= a.out.max_tokens) return;
    const int32_t n = a.pg.n_req;
    if (n == 0 || t >= a.out.q_ptr[n]) {
        plan_map_row(a, t, -1, -1, 0);
        return;
    }
    const int32_t r = last_at_most(a.out.q_ptr, n, t);
    const int32_t pos = a.out.kv_end[r] - (a.out.q_ptr[r + 1] - t);
    plan_map_row(a, t, r, pos, a.pg.block_table[(int64_t)r * a.pg.ld_table + (pos >> a.shift)]);
}

// ------------------------------------------------------------------------ rotary positions and append
struct AppendArgs {
    int32_t q_heads, kv_heads, head_dim, rot, n_axes, units_rot, units_v;
    void *q_out;
    const void *q, *k, *v;
    int64_t ldqo, ldq, ldk, ldv;
    const float *inv_freq;
    const int32_t *axis, *pos, *slots;
    int64_t ld_pos;
    lora_kv_cache c;
    int32_t shift;
};

// cos and sin of position * inv_freq: the product is exact in 64 bits (31 + 24 bits), so
// reducing it to turns in 64 bits leaves the angle right to 2^-22 turns or better at any
// 32-bit position.
__device__ inline float2 turn_of(int32_t pos, float inv_freq)
{
    const double turns = (double)pos * (double)inv_freq * 0.15915494309189533577;
    const float half_turns = (float)(2.0 * (turns - rint(turns)));
    float2 cs;
    cs.y = sinpif(half_turns);
    cs.x = cospif(half_turns);
    return cs;
}

// One workgroup per token row: the row's cos and sin go to LDS once, and every thread then
// moves 16-byte chunks; a chunk pair (x[i..], x[i + rot/2..]) or, interleaved, one chunk
// holds whole rotation pairs.
template <typename T, bool INTER>
__global__ __launch_bounds__(256) void lora_rope_append_kernel(AppendArgs a)
{
    __shared__ float2 cs[LORA_KV_MAX_HEAD_DIM / 2];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int32_t slot = a.slots[t];
    if (slot < 0 || slot >= (int64_t)a.c.num_pages << a.shift) return;
    const int half = a.rot / 2;
    for (int i = tid; i < half; i += 256) {
        const int ax = a.axis ? a.axis[i] : 0;
        cs[i] = ax >= 0 && ax < a.n_axes ? turn_of(a.pos[ax * a.ld_pos + t], a.inv_freq[i]) : make_float2(1.f, 0.f);
    }
    __syncthreads();
    const int64_t cell = (int64_t)(slot >> a.shift) * a.c.page_stride +
                         (int64_t)(slot & ((1 << a.shift) - 1)) * a.c.token_stride;
    const int n_qk = (a.q_heads + a.kv_heads) * a.units_rot;
    const int n_all = n_qk + a.kv_heads * a.units_v;
    for (int u = tid; u < n_all; u += 256) {
        if (u >= n_qk) {
            const int h = (u - n_qk) / a.units_v, c = (u - n_qk) - h * a.units_v;
            store16(a.c.v, cell + h * a.c.head_stride + 8 * c, load16(a.v, t * a.ldv + h * a.head_dim + 8 * c));
            continue;
        }
        int h = u / a.units_rot;
        const int p = u - h * a.units_rot;
        const bool is_q = h < a.q_heads;
        if (!is_q) h -= a.q_heads;
        const void *src = is_q ? a.q : a.k;
        void *dst = is_q ? a.q_out : a.c.k;
        const int64_t from = t * (is_q ? a.ldq : a.ldk) + (int64_t)h * a.head_dim;
        const int64_t to = is_q ? t * a.ldqo + (int64_t)h * a.head_dim : cell + h * a.c.head_stride;
        float x[8], y[8];
        if (INTER) {
            const uint4 raw = load16(src, from + 8 * p);
            if (8 * p >= a.rot) {
                store16(dst, to + 8 * p, raw);
                continue;
            }
            unpack8<T>(raw, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 w = cs[4 * p + e];
                y[2 * e] = __builtin_fmaf(x[2 * e], w.x, -(x[2 * e + 1] * w.y));
                y[2 * e + 1] = __builtin_fmaf(x[2 * e], w.y, x[2 * e + 1] * w.x);
            }
            store16(dst, to + 8 * p, pack8<T>(y));
        } else {
            if (8 * p >= half) {  // a chunk that passes through
                const int c = half + 8 * p;
                store16(dst, to + c, load16(src, from + c));
                continue;
            }
            float b[8], z[8];
            unpack8<T>(load16(src, from + 8 * p), x);
            unpack8<T>(load16(src, from + half + 8 * p), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 w = cs[8 * p + e];
                y[e] = __builtin_fmaf(x[e], w.x, -(b[e] * w.y));
                z[e] = __builtin_fmaf(x[e], w.y, b[e] * w.x);
            }
            store16(dst, to + 8 * p, pack8<T>(y));
            store16(dst, to + half + 8 * p, pack8<T>(z));
        }
    }
}

// ------------------------------------------------------------------------ attention
struct AttnArgs {
    int32_t q_heads, kv_heads, head_dim, n_req, max_blocks, window, shift;
    float scale;
    void *out;
    const void *q;
    int64_t ldo, ldq, ld_table;
    const int32_t *table, *kv_len, *req;
    float *lse;
    lora_kv_cache c;
};

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// One workgroup per (row, head).  Sixteen lanes take a token: 16-byte chunks of its key
// against the query, summed over the lanes, then the softmax's running maximum and sum and
// the value's chunks; each group of sixteen lanes keeps its own, joined at the end in LDS.
template <typename T, int NC>
__global__ __launch_bounds__(256) void lora_paged_attention_kernel(AttnArgs a)
{
    __shared__ float sm[16], sl[16], so[16][LORA_KV_MAX_HEAD_DIM];
    const int tid = threadIdx.x, li = tid & 15, grp = tid >> 4;
    const int64_t row = blockIdx.x / a.q_heads;
    const int head = blockIdx.x % a.q_heads, kvh = head / (a.q_heads / a.kv_heads);
    const int32_t n = a.kv_len[row], r = a.req ? a.req[row] : (int32_t)row;
    if (n < 0 || n > (int64_t)a.max_blocks << a.shift || r < 0 || r >= a.n_req) return;
    const int chunks = a.head_dim / 8;
    float q[NC][8], o[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[c][e] = o[c][e] = 0.f;
        if (li + 16 * c < chunks)
            unpack8<T>(load16(a.q, row * a.ldq + (int64_t)head * a.head_dim + 8 * (li + 16 * c)), q[c]);
    }
    float m = -INFINITY, l = 0.f;
    const float sc = a.scale * kLog2e;
    const int32_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    for (int32_t t = first + grp; t < n; t += 16) {
        const int32_t page = a.table[(int64_t)r * a.ld_table + (t >> a.shift)];
        if (page < 0 || page >= a.c.num_pages) continue;
        const int64_t at = (int64_t)page * a.c.page_stride + (int64_t)(t & ((1 << a.shift) - 1)) * a.c.token_stride +
                           kvh * a.c.head_stride;
        float s = 0.f, x[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (li + 16 * c >= chunks) continue;
            float k[8];
            unpack8<T>(load16(a.c.k, at + 8 * (li + 16 * c)), k);
            unpack8<T>(load16(a.c.v, at + 8 * (li + 16 * c)), x[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(q[c][e], k[e], s);
        }
#pragma unroll
        for (int d = 1; d < 16; d *= 2) s += __shfl_xor(s, d, 16);
        s *= sc;
        const float mn = __builtin_fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        // a NaN score stays a NaN (fmax would drop it)
        const float p = __builtin_amdgcn_exp2f(s - base), f = __builtin_amdgcn_exp2f(m - base);
        m = mn;
        l = __builtin_fmaf(l, f, p);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (li + 16 * c >= chunks) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[c][e] = __builtin_fmaf(p, x[c][e], o[c][e] * f);
        }
    }
    if (li == 0) {
        sm[grp] = m;
        sl[grp] = l;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (li + 16 * c < chunks)
#pragma unroll
            for (int e = 0; e < 8; ++e) so[grp][8 * (li + 16 * c) + e] = o[c][e];
    __syncthreads();
    float mx = -INFINITY;
    for (int g = 0; g < 16; ++g) mx = __builtin_fmaxf(mx, sm[g]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float total = 0.f, f[16];
    for (int g = 0; g < 16; ++g) {
        f[g] = __builtin_amdgcn_exp2f(sm[g] - base);
        total = __builtin_fmaf(f[g], sl[g], total);
    }
    const bool none = total == 0.f;
    for (int d = tid; d < a.head_dim; d += 256) {
        float s = 0.f;
        for (int g = 0; g < 16; ++g) s = __builtin_fmaf(f[g], so[g][d], s);
        typename T::elem e = (typename T::elem)(none ? 0.f : s / total);
        static_cast<typename T::elem *>(a.out)[row * a.ldo + (int64_t)head * a.head_dim + d] = e;
    }
    if (a.lse && tid == 0) a.lse[row * a.q_heads + head] = none ? -INFINITY : (mx + __builtin_log2f(total)) * kLn2;
}

// ------------------------------------------------------------------------ residual add and norms
// Sum of v over the workgroup (same order for every launch of one size).
__device__ inline float block_sum(float v, float *wave_sums)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) wave_sums[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += wave_sums[w];
    return s;
}

// One workgroup per row; a thread keeps its NC chunks of eight elements in registers from
// the loads to the stores, so x and res are read once and res_out and y written once.
template <typename T, int NC>
__global__ __launch_bounds__(1024) void lora_residual_norm_kernel(lora_norm_args a)
{
    __shared__ float wave_sums[16];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int64_t row = blockIdx.x;
    const int chunks = a.hidden / 8;
    int32_t gi = -1;
    if (a.gate) {
        gi = a.gate_idx ? a.gate_idx[row] : 0;
        if (gi < -1 || gi >= a.n_gates) return;
    }
    float h[NC][8], p[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = p[i][e] = 0.f;
        const int c = tid + i * nt;
        if (c < chunks) {
            unpack8<T>(load16(a.res, row * a.ldr + 8 * c), h[i]);
            if (a.x) unpack8<T>(load16(a.x, row * a.ldx + 8 * c), p[i]);
        }
    }
    if (a.post_w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(p[i][e], p[i][e], ss);
        const float inv = 1.f / __builtin_sqrtf(block_sum(ss, wave_sums) / (float)a.hidden + a.eps);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + i * nt;
            if (c >= chunks) continue;
            float w[8];
            unpack8<T>(load16(a.post_w, 8 * c), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] = p[i][e] * inv * (w[e] + a.w_offset);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + i * nt;
        if (c >= chunks) continue;
        if (gi >= 0) {
            float g[8];
            unpack8<T>(load16(a.gate, gi * a.ldg + 8 * c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] *= g[e];
        }
        if (a.x)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = __builtin_fmaf(a.alpha, p[i][e], h[i][e]);
        if (a.res_out) store16(a.res_out, row * a.ldro + 8 * c, pack8<T>(h[i]));
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
    }
    if (!a.y) return;
    const float inv = 1.f / __builtin_sqrtf(block_sum(ss, wave_sums) / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + i * nt;
        if (c >= chunks) continue;
        float w[8], y[8];
        unpack8<T>(load16(a.w, 8 * c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[i][e] * inv * (w[e] + a.w_offset);
        store16(a.y, row * a.ldy + 8 * c, pack8<T>(y));
    }
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

int check_cache(const lora_kv_cache *c)
{
    if (!c) return fail(LORA_E_NULL, "cache descriptor is NULL");
    int st = check_type(c->type);
    if (st) return st;
    if (page_shift(c->page_size) < 0)
        return fail(LORA_E_SHAPE, "page_size = %d is not a power of two in 1..%d", c->page_size, LORA_KV_MAX_PAGE);
    if (c->num_pages < 1 || (int64_t)c->num_pages * c->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "num_pages = %d of %d tokens (1 page to 2^31 - 1 tokens)", c->num_pages, c->page_size);
    if (c->kv_heads < 1) return fail(LORA_E_SHAPE, "kv_heads = %d", c->kv_heads);
    if (c->head_dim < 8 || c->head_dim > LORA_KV_MAX_HEAD_DIM || c->head_dim % 8)
        return fail(LORA_E_SHAPE, "head_dim = %d is not a multiple of 8 in 8..%d", c->head_dim, LORA_KV_MAX_HEAD_DIM);
    if (c->reserved != 0) return fail(LORA_E_SHAPE, "reserved field must be 0");
    if (!c->k || !c->v) return fail(LORA_E_NULL, "cache needs k and v");
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(LORA_E_ALIGN, "cache k and v must be 16-byte aligned");
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride}) {
        if (s < c->head_dim || s > (int64_t)1 << 50)
            return fail(LORA_E_SHAPE, "cache stride %lld < head_dim = %d", (long long)s, c->head_dim);
        if (s % 8) return fail(LORA_E_ALIGN, "cache stride %lld is not a multiple of 8", (long long)s);
    }
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

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

int lora_kv_plan(void *stream, const lora_kv_pages *pages, const int32_t *kv_len, const int32_t *new_len,
                 const int32_t *req_slot, const lora_kv_plan_out *out)
{
    clear_error();
    if (!pages || !out) return fail(LORA_E_NULL, "pages and out are required");
    PlanArgs a{*pages, *out, kv_len, new_len, req_slot, 0, 0};
    a.shift = page_shift(pages->page_size);
    if (a.shift < 0)
        return fail(LORA_E_SHAPE, "page_size = %d is not a power of two in 1..%d", pages->page_size, LORA_KV_MAX_PAGE);
    if (pages->n_req < 0 || pages->num_pages < 1 || (int64_t)pages->num_pages * pages->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "n_req = %d, num_pages = %d of %d tokens", pages->n_req, pages->num_pages,
                    pages->page_size);
    if (pages->max_blocks < 1 || pages->ld_table < pages->max_blocks)
        return fail(LORA_E_SHAPE, "max_blocks = %d, ld_table = %lld", pages->max_blocks, (long long)pages->ld_table);
    if (out->max_tokens < 0 || out->reserved != 0)
        return fail(LORA_E_SHAPE, "max_tokens = %d, reserved = %d", out->max_tokens, out->reserved);
    if (!pages->free_pages || !pages->free_top || !out->status || !out->free_top || !out->q_ptr)
        return fail(LORA_E_NULL, "free_pages, free_top, status and q_ptr are required");
    if (pages->n_req > 0 && (!pages->block_table || !kv_len || !new_len || !out->kv_end))
        return fail(LORA_E_NULL, "block_table, kv_len, new_len and kv_end are required");
    if (out->max_tokens > 0 && (!out->tok_req || !out->tok_pos || !out->slots))
        return fail(LORA_E_NULL, "tok_req, tok_pos and slots are required");
    hipStream_t s = static_cast<hipStream_t>(stream);
    a.maps = out->max_tokens <= kPlanMapsHere;
    launch_args(lora_kv_plan_kernel, dim3(1), kPlanThreads, 0, s, a);
    if (!a.maps) launch_args(lora_kv_maps_kernel, dim3((unsigned)((out->max_tokens + 255ll) / 256)), 256, 0, s, a);
    return launch_status("step plan");
}

int lora_rope_append(void *stream, int32_t n_rows, int32_t q_heads, void *q_out, int64_t ldqo, const void *q,
                     int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const lora_rope *rope,
                     const int32_t *positions, int64_t ld_pos, const int32_t *slots, const lora_kv_cache *cache)
{
    clear_error();
    int st = check_cache(cache);
    if (st) return st;
    if (!rope) return fail(LORA_E_NULL, "rope descriptor is NULL");
    if (n_rows < 0 || q_heads < 0) return fail(LORA_E_SHAPE, "n_rows = %d, q_heads = %d", n_rows, q_heads);
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > cache->head_dim)
        return fail(LORA_E_SHAPE, "rot_dim = %d is not a multiple of 16 in 0..head_dim = %d", rope->rot_dim,
                    cache->head_dim);
    if (rope->n_axes < 1 || rope->n_axes > LORA_ROPE_MAX_AXES)
        return fail(LORA_E_SHAPE, "n_axes = %d outside 1..%d", rope->n_axes, LORA_ROPE_MAX_AXES);
    if ((rope->interleaved != 0 && rope->interleaved != 1) || rope->reserved != 0)
        return fail(LORA_E_SHAPE, "interleaved = %d, reserved = %d", rope->interleaved, rope->reserved);
    if ((int64_t)q_heads + cache->kv_heads > 1 << 20)
        return fail(LORA_E_UNSUPPORTED, "%d query and %d key/value heads", q_heads, cache->kv_heads);
    if (n_rows == 0) return LORA_OK;
    const int64_t kv_cols = (int64_t)cache->kv_heads * cache->head_dim;
    if (q_heads > 0) {
        if ((st = check_matrix(q, ldq, (int64_t)q_heads * cache->head_dim, "q"))) return st;
        if ((st = check_matrix(q_out, ldqo, (int64_t)q_heads * cache->head_dim, "q_out"))) return st;
    }
    if ((st = check_matrix(k, ldk, kv_cols, "k"))) return st;
    if ((st = check_matrix(v, ldv, kv_cols, "v"))) return st;
    if (q_heads > 0) {
        const int64_t cols = (int64_t)q_heads * cache->head_dim;
        if ((st = check_apart(q_out, ldqo, cols, q, ldq, cols, n_rows, true, "q_out and q"))) return st;
        if ((st = check_apart(q_out, ldqo, cols, k, ldk, kv_cols, n_rows, false, "q_out and k"))) return st;
        if ((st = check_apart(q_out, ldqo, cols, v, ldv, kv_cols, n_rows, false, "q_out and v"))) return st;
    }
    if (!slots) return fail(LORA_E_NULL, "slots is NULL");
    if (rope->rot_dim > 0) {
        if (!positions || !rope->inv_freq) return fail(LORA_E_NULL, "positions and inv_freq are required");
        if (ld_pos < n_rows) return fail(LORA_E_SHAPE, "ld_pos = %lld < %d rows", (long long)ld_pos, n_rows);
    }
    AppendArgs a{};
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.rot = rope->rot_dim;
    a.n_axes = rope->n_axes;
    a.units_rot = rope->interleaved ? cache->head_dim / 8 : cache->head_dim / 8 - rope->rot_dim / 16;
    a.units_v = cache->head_dim / 8;
    a.q_out = q_out;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldqo = ldqo;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.inv_freq = rope->inv_freq;
    a.axis = rope->axis;
    a.pos = positions;
    a.ld_pos = ld_pos;
    a.slots = slots;
    a.c = *cache;
    a.shift = page_shift(cache->page_size);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)n_rows);
    const bool bf = cache->type == LORA_TYPE_BF16;
    if (rope->interleaved) {
        if (bf) launch_args(lora_rope_append_kernel<BF16, true>, grid, 256, 0, s, a);
        else launch_args(lora_rope_append_kernel<F16, true>, grid, 256, 0, s, a);
    } else {
        if (bf) launch_args(lora_rope_append_kernel<BF16, false>, grid, 256, 0, s, a);
        else launch_args(lora_rope_append_kernel<F16, false>, grid, 256, 0, s, a);
    }
    return launch_status("rotary append");
}

size_t lora_paged_attention_bytes(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim)
{
    if (n_rows < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 8) return 0;
    return 256;
}

int lora_paged_attention(void *stream, int32_t n_rows, int32_t q_heads, void *out, int64_t ldo, const void *q,
                         int64_t ldq, const lora_kv_cache *cache, int32_t n_req, const int32_t *block_table,
                         int64_t ld_table, int32_t max_blocks, const int32_t *kv_len, const int32_t *req, float scale,
                         int32_t window, float *lse, void *work, size_t work_bytes)
{
    clear_error();
    int st = check_cache(cache);
    if (st) return st;
    if (n_rows < 0 || n_req < 0) return fail(LORA_E_SHAPE, "n_rows = %d, n_req = %d", n_rows, n_req);
    if (q_heads < 1 || q_heads % cache->kv_heads)
        return fail(LORA_E_SHAPE, "q_heads = %d is not a multiple of kv_heads = %d", q_heads, cache->kv_heads);
    if (max_blocks < 1 || ld_table < max_blocks || (int64_t)max_blocks * cache->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "max_blocks = %d, ld_table = %lld", max_blocks, (long long)ld_table);
    if (window < 0) return fail(LORA_E_SHAPE, "window = %d", window);
    if (!std::isfinite(scale)) return fail(LORA_E_SHAPE, "scale is not finite");
    if ((int64_t)n_rows * q_heads > (int64_t)1 << 30)
        return fail(LORA_E_SHAPE, "%d rows of %d heads are too many for one launch", n_rows, q_heads);
    if (n_rows == 0) return LORA_OK;
    if ((st = check_matrix(q, ldq, (int64_t)q_heads * cache->head_dim, "q"))) return st;
    if ((st = check_matrix(out, ldo, (int64_t)q_heads * cache->head_dim, "out"))) return st;
    const int64_t cols = (int64_t)q_heads * cache->head_dim;
    if ((st = check_apart(out, ldo, cols, q, ldq, cols, n_rows, false, "out and q"))) return st;
    if (!kv_len || (n_req > 0 && !block_table)) return fail(LORA_E_NULL, "kv_len and block_table are required");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) return fail(LORA_E_ALIGN, "lse must be 4-byte aligned");
    if (!work) return fail(LORA_E_NULL, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(work) & 255) return fail(LORA_E_ALIGN, "workspace must be 256-byte aligned");
    const size_t need = lora_paged_attention_bytes(n_rows, q_heads, cache->kv_heads, cache->head_dim);
    if (work_bytes < need) return fail(LORA_E_SHAPE, "workspace of %zu bytes < %zu for %d rows", work_bytes, need, n_rows);
    AttnArgs a{};
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.n_req = n_req;
    a.max_blocks = max_blocks;
    a.window = window;
    a.shift = page_shift(cache->page_size);
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
    a.c = *cache;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)(n_rows * q_heads));
    const bool bf = cache->type == LORA_TYPE_BF16, wide = cache->head_dim > 128;
    if (bf && wide) launch_args(lora_paged_attention_kernel<BF16, 2>, grid, 256, 0, s, a);
    else if (bf) launch_args(lora_paged_attention_kernel<BF16, 1>, grid, 256, 0, s, a);
    else if (wide) launch_args(lora_paged_attention_kernel<F16, 2>, grid, 256, 0, s, a);
    else launch_args(lora_paged_attention_kernel<F16, 1>, grid, 256, 0, s, a);
    return launch_status("paged attention");
}

int lora_residual_norm(void *stream, const lora_norm_args *args)
{
    clear_error();
    if (!args) return fail(LORA_E_NULL, "args is NULL");
    const lora_norm_args &a = *args;
    int st = check_type(a.type);
    if (st) return st;
    if (a.n_rows < 0) return fail(LORA_E_SHAPE, "n_rows = %d", a.n_rows);
    if (a.hidden < 8 || a.hidden > LORA_NORM_MAX_HIDDEN || a.hidden % 8)
        return fail(LORA_E_SHAPE, "hidden = %d is not a multiple of 8 in 8..%d", a.hidden, LORA_NORM_MAX_HIDDEN);
    if (a.reserved != 0) return fail(LORA_E_SHAPE, "reserved field must be 0");
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.alpha) || !std::isfinite(a.w_offset))
        return fail(LORA_E_SHAPE, "eps = %g, alpha = %g, w_offset = %g", a.eps, a.alpha, a.w_offset);
    if (!a.y && !a.res_out) return fail(LORA_E_NULL, "y and res_out are both NULL");
    if (!a.x && (a.post_w || a.gate)) return fail(LORA_E_NULL, "post_w and gate need x");
    if (!a.gate && a.gate_idx) return fail(LORA_E_NULL, "gate_idx without gate");
    if (a.n_rows == 0) return LORA_OK;
    if ((st = check_matrix(a.res, a.ldr, a.hidden, "res"))) return st;
    if (a.x && (st = check_matrix(a.x, a.ldx, a.hidden, "x"))) return st;
    if (a.y && (st = check_matrix(a.y, a.ldy, a.hidden, "y"))) return st;
    if (a.res_out && (st = check_matrix(a.res_out, a.ldro, a.hidden, "res_out"))) return st;
    if (a.y && (st = check_matrix(a.w, a.hidden, a.hidden, "w"))) return st;
    if (a.post_w && (st = check_matrix(a.post_w, a.hidden, a.hidden, "post_w"))) return st;
    const int64_t h = a.hidden, n = a.n_rows;
    if ((st = check_apart(a.res_out, a.ldro, h, a.res, a.ldr, h, n, true, "res_out and res"))) return st;
    if ((st = check_apart(a.res_out, a.ldro, h, a.x, a.ldx, h, n, false, "res_out and x"))) return st;
    if ((st = check_apart(a.y, a.ldy, h, a.x, a.ldx, h, n, true, "y and x"))) return st;
    if ((st = check_apart(a.y, a.ldy, h, a.res, a.ldr, h, n, false, "y and res"))) return st;
    if ((st = check_apart(a.y, a.ldy, h, a.res_out, a.ldro, h, n, false, "y and res_out"))) return st;
    if (a.gate) {
        if (a.n_gates < 1 || (!a.gate_idx && a.n_gates != 1))
            return fail(LORA_E_SHAPE, "n_gates = %d%s", a.n_gates, a.gate_idx ? "" : " without gate_idx");
        if ((st = check_matrix(a.gate, a.ldg, a.hidden, "gate"))) return st;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int chunks = a.hidden / 8;
    int threads = 64;
    while (threads < 1024 && threads < chunks) threads *= 2;
    const int nc = (chunks + threads - 1) / threads;
    const dim3 grid((unsigned)a.n_rows);
    const bool bf = a.type == LORA_TYPE_BF16;
#define LORA_NORM(NC)                                                                          \
    (bf ? launch_args(lora_residual_norm_kernel<BF16, NC>, grid, threads, 0, s, a)             \
        : launch_args(lora_residual_norm_kernel<F16, NC>, grid, threads, 0, s, a))
    if (nc <= 1) LORA_NORM(1);
    else if (nc <= 2) LORA_NORM(2);
    else if (nc <= 4) LORA_NORM(4);
    else LORA_NORM(8);
#undef LORA_NORM
    return launch_status("residual norm");
}

}  // extern "C"
