// HIP kernels (gfx950 / CDNA4) and launchers of the decode-step operators beside the
// add-on: the step plan, rotary positions with the append to the paged cache, attention
// over that cache, and the residual add with its norms (lora_step.h).
//
// Times in comments: what a kernel takes now is the median of its kernel trace; figures with
// an alternative or an earlier form beside them were taken together, as launches of a
// captured graph (the two ways differ by up to 0.5 us for the smallest kernels and by 5 %
// for the others).
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

// ------------------------------------------------------------------------ step plan
struct PlanArgs {
    lora_kv_pages pg;
    lora_kv_plan_out out;
    const int32_t *kv_len, *new_len, *req_slot;
    int32_t shift;   // log2(page_size)
    int32_t move;    // this launch moves the pages and writes the maps
    int32_t finish;  // this launch writes the lengths, offsets, free top and status
};

constexpr int kPlanThreads = 1024;  // requests planned at a time
constexpr int kPlanGroups = 256;    // workgroups of a launch at most: one per CU
constexpr int32_t kPlanMaxReq = 1 << 30;  // requests: the sum of two of their numbers fits 32 bits

// One request of a plan; `bad` holds its LORA_KV_* bits.
struct PlanReq {
    int32_t len, had;
    uint32_t add, grown, given;
    int32_t bad;
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
        q.grown = (uint32_t)(((end + mask) >> a.shift) - q.had);
    }
    return q;
}

// Inclusive prefix sum over the wavefront that stops at 2^32 - 1 (sums of that kind are
// associative, and one that large fits no list and no batch): within rows of sixteen
// lanes, then across them.
__device__ inline uint32_t wave_scan_sat(uint32_t v)
{
#define LORA_SCAN_STEP(ctrl, rows) \
    v = __builtin_elementwise_add_sat(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
    LORA_SCAN_STEP(0x111, 0xf);  // row_shr:1, 2, 4, 8
    LORA_SCAN_STEP(0x112, 0xf);
    LORA_SCAN_STEP(0x114, 0xf);
    LORA_SCAN_STEP(0x118, 0xf);
    LORA_SCAN_STEP(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
    LORA_SCAN_STEP(0x143, 0xc);  // row_bcast:31 into rows 2 and 3
#undef LORA_SCAN_STEP
    return v;
}

// Prefix sums of a chunk of requests and their totals: pages given back, pages taken, tokens.
struct PlanSums {
    uint32_t given, grown, add;        // before this thread's request
    uint32_t all_given, all_grown, all_add;
    int32_t bad;
};

template <int THREADS>
__device__ inline PlanSums plan_scan(const PlanReq &q, uint4 *wave_sums)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t g = wave_scan_sat(q.given), t = wave_scan_sat(q.grown), n = wave_scan_sat(q.add);
    int32_t bad = 0;
    for (int b = 1; b <= LORA_KV_INVALID; b *= 2) bad |= __any(q.bad & b) ? b : 0;
    PlanSums s{0, 0, 0, 0, 0, 0, 0};
    if (THREADS == 64) {
        s.all_given = __builtin_amdgcn_readlane(g, 63);
        s.all_grown = __builtin_amdgcn_readlane(t, 63);
        s.all_add = __builtin_amdgcn_readlane(n, 63);
        s.bad = bad;
    } else {
        __syncthreads();  // wave_sums may still be read from the call before
        if (lane == 63) wave_sums[wave] = make_uint4(g, t, n, (uint32_t)bad);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            const uint4 x = wave_sums[w];
            if (w == wave) {
                s.given = s.all_given;
                s.grown = s.all_grown;
                s.add = s.all_add;
            }
            s.all_given = __builtin_elementwise_add_sat(s.all_given, x.x);
            s.all_grown = __builtin_elementwise_add_sat(s.all_grown, x.y);
            s.all_add = __builtin_elementwise_add_sat(s.all_add, x.z);
            s.bad |= (int32_t)x.w;
        }
    }
    s.given += g - q.given;
    s.grown += t - q.grown;
    s.add += n - q.add;
    return s;
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

// What the sums of all requests allow: LORA_KV_* bits.
__device__ inline int32_t plan_check(const PlanArgs &a, const PlanSums &s, int32_t top0)
{
    int32_t bad = s.bad;
    if (top0 < 0 || top0 > a.pg.num_pages || top0 + (int64_t)s.all_given > a.pg.num_pages) bad |= LORA_KV_INVALID;
    if (s.all_grown > top0 + (int64_t)s.all_given) bad |= LORA_KV_NO_PAGES;
    if ((int64_t)s.all_add > a.out.max_tokens) bad |= LORA_KV_TOO_MANY;
    return bad;
}

__device__ inline void plan_status(const PlanArgs &a, const PlanSums &s, int32_t top0, int32_t bad)
{
    a.out.status[0] = bad;
    a.out.status[1] = (int32_t)min(s.all_add, (uint32_t)INT32_MAX);
    a.out.status[2] = (int32_t)min(s.all_grown, (uint32_t)INT32_MAX);
    a.out.status[3] = (int32_t)min(s.all_given, (uint32_t)INT32_MAX);
    a.out.free_top[0] = bad ? top0 : (int32_t)(top0 + (int64_t)s.all_given - s.all_grown);
    a.out.q_ptr[a.pg.n_req] = bad ? 0 : (int32_t)s.all_add;
}

// The plan of up to THREADS requests.  Every workgroup makes the prefix sums and checks for
// itself (all or nothing), then takes its share of the pages given back, the pages taken
// and the token rows, each found by a binary search in the sums.  Nothing that one thread
// reads is written by another: the table entries read were there before, and free_pages is
// read below its old end only -- a page that an ended request gives back in this step is
// taken from that request's table row.  Lengths and free top are written by workgroup 0,
// or, where they are updated in place and there are more workgroups, by a second launch.
// Bound by the latency of its chain of loads (lengths, then ids), so small batches run in
// few wavefronts, whose barriers are cheap: 32 decoding requests 3.7 us (in a graph 3.9, with
// 1024 threads 5.2), 509 requests with 9,400 token rows 6.4 us.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void lora_kv_plan_kernel(PlanArgs a)
{
    __shared__ uint4 wave_sums[THREADS / 64];
    __shared__ int32_t off[THREADS], off_given[THREADS], off_tok[THREADS], had_s[THREADS], len_s[THREADS];
    const int tid = threadIdx.x;
    const int32_t n = a.pg.n_req;
    const int32_t top0 = *a.pg.free_top;
    const PlanReq q = plan_req(a, tid);
    const PlanSums s = plan_scan<THREADS>(q, wave_sums);
    const int32_t bad = plan_check(a, s, top0);
    off[tid] = (int32_t)s.grown;
    off_given[tid] = (int32_t)s.given;
    off_tok[tid] = (int32_t)s.add;
    had_s[tid] = q.had;
    len_s[tid] = q.len;
    __syncthreads();  // also: every thread has read its lengths and the free top
    if (a.finish && blockIdx.x == 0) {
        if (tid == 0) plan_status(a, s, top0, bad);
        if (tid < n) {
            a.out.kv_end[tid] = bad ? q.len : (int32_t)q.end;
            a.out.q_ptr[tid] = bad ? 0 : (int32_t)s.add;
        }
    }
    if (!a.move) return;
    const int32_t first = blockIdx.x * THREADS + tid, step = gridDim.x * THREADS;
    const int32_t given = bad ? 0 : (int32_t)s.all_given, taken = bad ? 0 : (int32_t)s.all_grown;
    const int32_t rows = bad ? 0 : (int32_t)s.all_add, top = top0 + given;
    auto page_given = [&](int32_t k) {  // k-th page of the ended requests
        const int r = last_at_most(off_given, THREADS, k);
        return a.pg.block_table[(int64_t)r * a.pg.ld_table + (k - off_given[r])];
    };
    auto page_taken = [&](int32_t k) {  // k-th page from the list's end
        const int32_t at = top - 1 - k;
        return at < top0 ? a.pg.free_pages[at] : page_given(at - top0);
    };
    // one line of items: token rows, pages taken, pages given back
    const int64_t n_tok = a.out.max_tokens, n_all = n_tok + taken + given;
    for (int64_t i = first; i < n_all; i += step) {
        if (i < n_tok) {
            const int32_t t = (int32_t)i;
            if (t >= rows) {
                plan_map_row(a, t, -1, -1, 0);
                continue;
            }
            const int r = last_at_most(off_tok, THREADS, t);
            const int32_t pos = len_s[r] + (t - off_tok[r]), b = pos >> a.shift;
            plan_map_row(a, t, r, pos, b < had_s[r] ? a.pg.block_table[(int64_t)r * a.pg.ld_table + b]
                                                    : page_taken(off[r] + b - had_s[r]));
        } else if (i < n_tok + taken) {
            const int32_t k = (int32_t)(i - n_tok);
            const int r = last_at_most(off, THREADS, k);
            a.pg.block_table[(int64_t)r * a.pg.ld_table + had_s[r] + (k - off[r])] = page_taken(k);
        } else {
            const int32_t k = (int32_t)(i - n_tok - taken);
            a.pg.free_pages[top0 + k] = page_given(k);
        }
    }
}

// The plan of more requests than one chunk holds, by one workgroup: totals and checks first,
// then, a chunk at a time, the pages of ended requests onto the free list, and after all
// of those the pages of growing ones off it.  4096 requests, 13,400 pages and 6,850 token rows:
// 33 us, and 5.6 for the maps.
__global__ __launch_bounds__(kPlanThreads) void lora_kv_plan_chunks_kernel(PlanArgs a)
{
    constexpr int THREADS = kPlanThreads;
    __shared__ uint4 wave_sums[THREADS / 64];
    __shared__ int32_t off[THREADS], had_s[THREADS];
    const int tid = threadIdx.x;
    const int32_t n = a.pg.n_req;
    const int32_t top0 = *a.pg.free_top;
    PlanReq sum = plan_req(a, tid);
    for (int32_t r = tid + THREADS; r < n; r += THREADS) {
        const PlanReq x = plan_req(a, r);
        sum.bad |= x.bad;
        sum.given = __builtin_elementwise_add_sat(sum.given, x.given);
        sum.grown = __builtin_elementwise_add_sat(sum.grown, x.grown);
        sum.add = __builtin_elementwise_add_sat(sum.add, x.add);
    }
    const PlanSums all = plan_scan<THREADS>(sum, wave_sums);
    const int32_t bad = plan_check(a, all, top0);
    __syncthreads();  // every thread has read the free top
    if (tid == 0) plan_status(a, all, top0, bad);
    if (bad) {
        for (int32_t r = tid; r < n; r += THREADS) {
            a.out.kv_end[r] = a.kv_len[r];
            a.out.q_ptr[r] = 0;
        }
        return;
    }
    int32_t at = top0;
    for (int32_t c = 0; c < n && all.all_given > 0; c += THREADS) {
        const PlanSums s = plan_scan<THREADS>(plan_req(a, c + tid), wave_sums);
        off[tid] = (int32_t)s.given;
        __syncthreads();
        const int32_t here = (int32_t)s.all_given;
        for (int32_t k = tid; k < here; k += THREADS) {
            const int i = last_at_most(off, THREADS, k);
            a.pg.free_pages[at + k] = a.pg.block_table[(int64_t)(c + i) * a.pg.ld_table + (k - off[i])];
        }
        at += here;
        __syncthreads();  // off, and below the list, are read by other threads
    }
    at -= 1;
    int32_t row0 = 0;
    for (int32_t c = 0; c < n; c += THREADS) {
        const PlanReq q = plan_req(a, c + tid);
        const PlanSums s = plan_scan<THREADS>(q, wave_sums);
        off[tid] = (int32_t)s.grown;
        had_s[tid] = q.had;
        if (c + tid < n) {
            a.out.q_ptr[c + tid] = row0 + (int32_t)s.add;
            a.out.kv_end[c + tid] = (int32_t)q.end;
        }
        __syncthreads();
        const int32_t here = (int32_t)s.all_grown;
        for (int32_t k = tid; k < here; k += THREADS) {
            const int i = last_at_most(off, THREADS, k);
            a.pg.block_table[(int64_t)(c + i) * a.pg.ld_table + had_s[i] + (k - off[i])] = a.pg.free_pages[at - k];
        }
        at -= here;
        row0 += (int32_t)s.all_add;
        __syncthreads();
    }
}

// Token maps of a step planned in chunks, one row per thread, from what the plan left: q_ptr
// (searched), kv_end and the table.
__global__ __launch_bounds__(256) void lora_kv_maps_kernel(PlanArgs a)
{
    const int32_t t = blockIdx.x * 256 + threadIdx.x;
    if (t >= a.out.max_tokens) return;
    const int32_t n = a.pg.n_req;
    if (t >= a.out.q_ptr[n]) {
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

constexpr int32_t kAppendFill = 1024;  // rows that fill the CUs with one workgroup each

// cos and sin of position * inv_freq.  The product (31 + 24 bits) is kept as p + e, exactly,
// and 1 / (2 pi) to twice 53 bits, so the fraction of a turn is right to 2^-50 at any 32-bit
// position; it is rounded to fp32 only then.
__device__ inline float2 turn_of(int32_t pos, float inv_freq)
{
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double p = (double)pos * (double)inv_freq, e = __builtin_fma((double)pos, (double)inv_freq, -p);
    const double whole = rint(p * kHi);
    const double part = __builtin_fma(p, kHi, -whole) + __builtin_fma(p, kLo, e * kHi);
    const float half_turns = (float)(2.0 * part);
    float2 cs;
    sincospif(half_turns, &cs.y, &cs.x);
    return cs;
}

// Workgroups of up to 256 threads: blockIdx.x is the token row, and the row's units go round over
// the threads of its gridDim.y workgroups.  A unit moves one 16-byte chunk, or the two
// chunks x[i..], x[i + rot/2..] whose elements turn together (interleaved, one chunk holds
// whole pairs).  A thread asks for its first chunks first; while they are on their way, the
// row's cos and sin are worked out, once, into LDS.  Bound by reading q, k, v and writing
// q_out and the cells: 12,907 rows of the 7B layout 114 us (5.55 TB/s), 4001 rows of the
// 70B layout on three axes 25.7 us (6.4 TB/s: 82 MB in and 82 out, part of which stays in the
// 256 MB cache beside the memory), 12,000 rows of 8/1 heads 14.4 us (4.3 TB/s, a
// workgroup of two wavefronts a row), 32 decode rows 3.5 us.  Four chunks a thread
// in flight from the start were slower on the large ones (125.5 and 37 us against 122 and
// 36, before streaming stores).
template <typename T, bool INTER, bool STREAM>
__global__ __launch_bounds__(256) void lora_rope_append_kernel(AppendArgs a)
{
    __shared__ float2 cs[LORA_KV_MAX_HEAD_DIM / 2];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int32_t slot = a.slots[t];  // waited for only where something is stored
    const int half = a.rot / 2;
    const int n_qk = (a.q_heads + a.kv_heads) * a.units_rot;
    const int n_all = n_qk + a.kv_heads * a.units_v;
    enum { kQ, kK, kV };
    struct Unit {
        int what, head, col;  // its (first) chunk
        int turn;             // first of its frequencies, -1: its chunk passes through
    };
    auto unit_of = [&](int u) {
        if (u >= n_qk) {
            const int h = (u - n_qk) / a.units_v;
            return Unit{kV, h, 8 * (u - n_qk - h * a.units_v), -1};
        }
        const int h = u / a.units_rot;
        int d = 8 * (u - h * a.units_rot), turn = -1;
        if (INTER) turn = d < a.rot ? d / 2 : -1;
        else if (d < half) turn = d;
        else d += half;  // the chunks behind the pairs
        return h < a.q_heads ? Unit{kQ, h, d, turn} : Unit{kK, h - a.q_heads, d, turn};
    };
    const int step = blockDim.x * gridDim.y;
    int u = blockIdx.y * blockDim.x + tid;
    Unit un{};
    uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
    auto fetch = [&]() {
        un = unit_of(u);
        const void *src = un.what == kQ ? a.q : un.what == kK ? a.k : a.v;
        const int64_t ld = un.what == kQ ? a.ldq : un.what == kK ? a.ldk : a.ldv;
        const int64_t from = t * ld + (int64_t)un.head * a.head_dim + un.col;
        ra = load16(src, from);
        if (!INTER && un.turn >= 0) rb = load16(src, from + half);
    };
    if (u < n_all) fetch();
    for (int i = tid; i < half; i += blockDim.x) {
        const int ax = a.axis ? a.axis[i] : 0;
        cs[i] = ax >= 0 && ax < a.n_axes ? turn_of(a.pos[ax * a.ld_pos + t], a.inv_freq[i]) : make_float2(1.f, 0.f);
    }
    if (slot < 0 || slot >= (int64_t)a.c.num_pages << a.shift) return;
    const int64_t cell = (int64_t)(slot >> a.shift) * a.c.page_stride +
                         (int64_t)(slot & ((1 << a.shift) - 1)) * a.c.token_stride;
    __syncthreads();
    while (u < n_all) {
        void *const dst = un.what == kQ ? a.q_out : un.what == kK ? a.c.k : a.c.v;
        const int64_t to = (un.what == kQ ? t * a.ldqo + (int64_t)un.head * a.head_dim : cell + un.head * a.c.head_stride) + un.col;
        if (un.turn < 0) {
            store16<STREAM>(dst, to, ra);
        } else {
            float x[8], y[8];
            unpack8<T>(ra, x);
            if (INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 w = cs[un.turn + e];
                    y[2 * e] = __builtin_fmaf(x[2 * e], w.x, -(x[2 * e + 1] * w.y));
                    y[2 * e + 1] = __builtin_fmaf(x[2 * e], w.y, x[2 * e + 1] * w.x);
                }
                store16<STREAM>(dst, to, pack8<T>(y));
            } else {
                float b[8], z[8];
                unpack8<T>(rb, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 w = cs[un.turn + e];
                    y[e] = __builtin_fmaf(x[e], w.x, -(b[e] * w.y));
                    z[e] = __builtin_fmaf(x[e], w.y, b[e] * w.x);
                }
                store16<STREAM>(dst, to, pack8<T>(y));
                store16<STREAM>(dst, to + half, pack8<T>(z));
            }
        }
        u += step;
        if (u < n_all) fetch();
    }
}

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
    lora_kv_cache c;
};

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kAttnWaves = 4;        // wavefronts of an attention workgroup
constexpr int kAttnTile = 32;        // tokens a wavefront takes at a time
constexpr int kAttnMinShare = 4;     // tiles a workgroup takes at least: one per wavefront
constexpr int kAttnRowTiles = 4;     // what starting and finishing a row costs, in tiles
constexpr int kAttnJoin = 16;        // parts joined at a time
constexpr int kAttnMaxTiles = 4096;  // key/value heads x 16-head tiles of one launch
constexpr int kAttnCUs = 256;
constexpr int32_t kAttnMaxSpan = 1 << 30;  // tokens of a table row: positions and steps past them fit 32 bits
// Wavefronts per SIMD, and so workgroups per CU, that the registers are kept to.
constexpr int attn_occupancy(int dp) { return dp <= 64 ? 2 : 1; }
// Arrival counters: two part slots per workgroup, and at most 4 workgroups per CU or one
// per head tile.  They lie first in a workspace, at one size for every shape, so calls of
// different shapes sharing a workspace never put sums where another finds its counters.
constexpr size_t kAttnCounters = 2 * (4 * kAttnCUs + kAttnMaxTiles);

// Visible tokens [first, first + span) of row i; span -1: the row is not active, or none.
struct RowSpan {
    int32_t req, first, span;
};

__device__ inline RowSpan row_span(const AttnArgs &a, int32_t i)
{
    const int32_t at = min(i, a.n_rows - 1);  // loads without a branch, so many can be in flight
    const int32_t n = a.kv_len[at], r = a.req ? a.req[at] : at;
    const bool on = i < a.n_rows && n >= 0 && n <= a.max_blocks << a.shift && r >= 0 && r < a.n_req;
    const int32_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    return RowSpan{r, first, on ? n - first : -1};
}

// The schedule of a launch, found by every workgroup from the lengths on the device.  Each
// active row costs its visible tokens in 32-token tiles (at least one) and kAttnRowTiles
// more; the rows' costs are laid end to end, and workgroup w takes [w share, (w + 1) share)
// of them: parts of one or more rows, the same amount of work in every workgroup whatever
// the lengths.  Row i's tiles lie at [tile0, tile0 + tiles) of that line.
struct RowWork {
    int32_t row, tile0, tiles;
    RowSpan rs;
};

__device__ inline int32_t row_tiles(const RowSpan &rs)
{
    return rs.span < 0 ? 0 : rs.span <= kAttnTile ? 1 : (rs.span - 1) / kAttnTile + 1;
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
struct RowWalk {
    int32_t base;   // the lanes hold rows base .. base + 63
    RowSpan rs;     // lane's row
    int32_t tiles;

    __device__ inline void load(const AttnArgs &a, int32_t b)
    {
        base = b;
        rs = row_span(a, b + (int32_t)(threadIdx.x & 63));
        tiles = row_tiles(rs);
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
__device__ inline RowWork first_row(const AttnArgs &a, int32_t w, RowWalk &walk, int32_t &share, int32_t &total)
{
    const int lane = threadIdx.x & 63;
    walk.load(a, 0);
    int32_t sum = walk.tiles > 0 ? walk.tiles + kAttnRowTiles : 0;
#pragma unroll 8
    for (int32_t c = 64; c < a.n_rows; c += 64) {
        const int32_t t = row_tiles(row_span(a, c + lane));
        sum += t > 0 ? t + kAttnRowTiles : 0;
    }
    total = __builtin_amdgcn_readlane(wave_scan(sum), 63);
    share = max((total + a.shares - 1) / a.shares, kAttnMinShare);
    const int64_t begin = (int64_t)w * share;
    int32_t at0 = 0;
    while (begin < total) {
        const int32_t cost = walk.tiles > 0 ? walk.tiles + kAttnRowTiles : 0, end = at0 + wave_scan(cost);
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

// True in the workgroup that is the n-th to come here with this counter, which is then 0
// again.  Every wavefront waits for its own stores to complete before the workgroup
// counts itself, so the last one's loads find all parts.
__device__ inline bool last_arrival(uint32_t *count, int n)
{
    __shared__ bool last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
        if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return last;
}

// Slot of part p of a row whose first part is in workgroup w0: a workgroup has one slot for
// the row it found begun and one for the row it leaves unfinished.
__device__ inline int32_t part_slot(int32_t w0, int32_t p) { return p == 0 ? 2 * w0 + 1 : 2 * (w0 + p); }

// Adds n parts (part0, part0 + step, ...) of a split row's heads, in that order, into part0's
// slot, or with `finish` into the row.
template <typename T, int DP>
__device__ inline void join_parts(const AttnArgs &a, int32_t row, int32_t w0, int64_t head0, int heads, int part0,
                                  int step, int n, bool finish)
{
    __shared__ float2 joined[16];
    constexpr int kBatch = 8;
    const int cols = a.head_dim / 4, tid = threadIdx.x;
    for (int i0 = 0; i0 < heads * cols; i0 += 64 * kAttnWaves) {
        const int i = i0 + tid;
        const bool on = i < heads * cols;
        const int h = on ? i / cols : 0, d = on ? 4 * (i - h * cols) : 0;
        // eight parts at a time, all their loads in flight together
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
    __syncthreads();  // every lane has read its heads' (m, l) of part0
    if (tid < heads)
        put_part(&a.part_ml[2 * ((int64_t)part_slot(w0, part0) * a.q_heads + head0 + tid)], joined[tid].x, joined[tid].y);
}

// The part `part` of a split row is stored: of every kAttnJoin parts, the workgroup that
// arrives last adds them up in order into the first one's slot; of those sums, the last
// arrival adds all and writes the row.  Who that is does not change what is added in which
// order.
template <typename T, int DP>
__device__ inline void join_row(const AttnArgs &a, int32_t row, int32_t w0, int32_t parts, int32_t part, int per_share,
                                int rest, int64_t head0, int heads)
{
    const int group0 = part / kAttnJoin * kAttnJoin, n_groups = (parts + kAttnJoin - 1) / kAttnJoin;
    const int in_group = min(kAttnJoin, parts - group0);
    if (!last_arrival(a.count + (int64_t)part_slot(w0, group0) * per_share + rest, in_group)) return;
    join_parts<T, DP>(a, row, w0, head0, heads, group0, 1, in_group, n_groups == 1);
    // (part 1 leads no group, so its counter is free for the groups)
    if (n_groups == 1 || !last_arrival(a.count + (int64_t)part_slot(w0, 1) * per_share + rest, n_groups)) return;
    join_parts<T, DP>(a, row, w0, head0, heads, 0, kAttnJoin, n_groups, true);
}

// One workgroup per (share of the rows, key/value head, 16 of its query heads), all of them
// resident at once; it takes the rows of its share one after another.
//
// Each wavefront walks its 32-token tiles of a row's part with its own running maximum and
// sums; nothing is shared until the end, so the loop has no barrier.  Scores are
// S^T = K Q^T on v_mfma_f32_16x16x32: the K rows go from memory straight into the A
// operand (lane: token l % 16, 16 bytes of it), Q^T stays in registers.  A lane then
// holds 4 + 4 tokens of one head, which is just the B operand of O^T += V^T P^T with
// the tokens in that order, so the weights never leave their lane.  V^T comes from a
// wave-private LDS tile by transposing reads (ds_read_tr, 4 tokens x 16 columns per
// sixteen lanes); its row pitch of 2 DP + 32 bytes keeps writes and reads free of bank
// conflicts.  The next tile's K is requested when this tile's scores are done, its V when
// this tile's V is in LDS, its page ids a tile ahead of both.
//
// Bound by reading K and V once; every head of a group shares the read, and 16 columns of
// heads cost the same matrix instructions as one.  Measured (fp16, 128 columns): 32 rows of
// 8192 tokens x 32 heads 724 us, 5.93 TB/s (a plain read of the bytes reaches 6.05); 32 rows
// of 64 to 4096 tokens 97 us, 5.2 TB/s; one row of 131,071 tokens, one key/value head 23.7 us
// (12.6 us beyond the read: the launch and lengths, table and first K one after another, which
// are all of the 6.5 us that one row of 17 tokens takes, and two joins; other joins than of
// kAttnJoin parts are not measured).  In a graph, slower than 98 / 24 / 6.2 us on the last
// three: two workgroups per CU 104 / 24.4 / 6.4, three 145 / 37 / 9.2 (what is in flight queues up, and every row's first loads
// wait behind it); eight wavefronts 105 / 27 / 9; 64-token tiles 104 / 26 / 8.2; one part
// per row and workgroup, a dynamic grid and a second launch to join 122 / 104 / 13.9;
// streaming loads 125 / 25 / 5.8 on that grid's successor (64-byte pieces of a row miss
// the L1 line their other half brought in).
template <typename T, int DP, bool FULL>
__global__ __launch_bounds__(64 * kAttnWaves) __attribute__((amdgpu_waves_per_eu(attn_occupancy(DP)))) void
lora_paged_attention_kernel(AttnArgs a)
{
    typedef typename T::elem E;
    typedef short s4 __attribute__((ext_vector_type(4)));
    constexpr int KC = DP / 32;              // 32-column steps of a score
    constexpr int DB = DP / 16;              // 16-column blocks of the output
    constexpr int kPitch = DP + 16;          // LDS row pitch, elements
    constexpr int kRegion = kAttnTile * kPitch;
    __shared__ __align__(16) uint16_t vt[kAttnWaves][kRegion];
    __shared__ float jm[kAttnWaves][16], jl[kAttnWaves][16];
    static_assert(sizeof(uint16_t) * kRegion >= sizeof(float) * 16 * DP, "the join fits the V tiles");

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int per_share = a.kv_heads * a.head_tiles;
    // The head tiles of one share and key/value head follow each other on one XCD (workgroups
    // go to the 8 XCDs in turn), so that its L2 serves K and V to all but the first.
    // (32 rows of 4000 tokens, 64/1 heads: 49 us without, 42 so.)
    int32_t pair = blockIdx.x, ht = 0;
    if (a.head_tiles > 1) {
        const int32_t eight = blockIdx.x / (8 * a.head_tiles);
        ht = blockIdx.x / 8 - eight * a.head_tiles;
        pair = 8 * eight + blockIdx.x % 8;
    }
    const int32_t wg = pair / a.kv_heads, kvh = pair - wg * a.kv_heads, rest = kvh * a.head_tiles + ht;
    if (wg >= a.shares) return;
    const int heads = min(16, a.group - 16 * ht);    // query heads of this tile
    const int64_t head0 = (int64_t)kvh * a.group + 16 * ht;
    const int32_t in_page = (1 << a.shift) - 1;
    int32_t share, total;
    RowWalk walk;
    RowWork rw = first_row(a, wg, walk, share, total);
    if (rw.row >= a.n_rows) return;
    const int32_t line0 = wg * share, line1 = (int32_t)min((int64_t)line0 + share, (int64_t)total);

    // A row's part in this share: tokens [begin, end); the row has `parts` parts from workgroup w0 on.
    struct Part {
        int32_t row, begin, end, w0, parts;
        const int32_t *table;
    };
    auto next_part = [&]() {
        while (rw.row < a.n_rows) {
            const int32_t row_end = rw.tile0 + rw.tiles;
            const int32_t from = max(rw.tile0, line0), to = min(row_end, line1), tile0 = rw.tile0;
            const Part p{rw.row, rw.rs.first + (from - tile0) * kAttnTile,
                         rw.rs.first + (int32_t)min((int64_t)(to - tile0) * kAttnTile, (int64_t)rw.rs.span),
                         tile0 < line0 ? tile0 / share : wg, 1, a.table + (int64_t)rw.rs.req * a.ld_table};
            int32_t last = wg;
            if (row_end > line1) last = (row_end - 1) / share;
            if (row_end < line1) rw = walk.after(a, rw.row, row_end + kAttnRowTiles);
            else rw.row = a.n_rows;
            if (from < to) return Part{p.row, p.begin, p.end, p.w0, last - p.w0 + 1, p.table};
            // else the row's tiles lie in the next workgroup's share
        }
        return Part{-1, 0, 0, 0, 0, nullptr};
    };
    // Tokens t0 + li and t0 + 16 + li of a tile: table entries, then cell offsets; a token
    // past the end or without a page reads cell 0 and is masked.
    auto ids_of = [&](const Part &p, int32_t t0, int32_t (&id)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) id[u] = t0 < p.end ? p.table[min(t0 + 16 * u + li, p.end - 1) >> a.shift] : -1;
    };
    auto cells_of = [&](const Part &p, int32_t t0, const int32_t (&id)[2], int64_t (&cell)[2]) {
        uint32_t seen = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t t = t0 + 16 * u + li;
            const bool ok = t < p.end && id[u] >= 0 && id[u] < a.c.num_pages;
            cell[u] = ok ? (int64_t)id[u] * a.c.page_stride + (int64_t)(t & in_page) * a.c.token_stride +
                               kvh * a.c.head_stride : 0;
            seen |= ((uint32_t)__ballot(ok) & 0xffffu) << (16 * u);
        }
        return seen;
    };
    auto load_rows = [&](const void *base, const int64_t (&cell)[2], uint4 (&r)[2][KC]) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int d = 32 * c + 8 * lg;
                r[u][c] = load16(base, cell[u] + (FULL || d < a.head_dim ? d : 0));
            }
    };
    auto load_q = [&](int32_t row, uint4 (&r)[KC]) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d = 32 * c + 8 * lg;
            r[c] = make_uint4(0, 0, 0, 0);
            if (li < heads && (FULL || d < a.head_dim)) r[c] = load16(a.q, row * a.ldq + (head0 + li) * a.head_dim + d);
        }
    };

    constexpr int kStep = kAttnWaves * kAttnTile;
    const uint4 zero4 = make_uint4(0, 0, 0, 0);
    const float scale = a.scale * kLog2e;
    uint16_t *const tile = vt[wave];
    const int tr_row = 4 * lg + (li >> 2), tr_col = 4 * (li & 3);
    typedef __attribute__((address_space(3))) s4 *lds4;

    // What is in flight: the K and V rows of this wavefront's next tile (cell, seen), which
    // may be the first of the next part, and the page ids of the tile after it (id).
    Part part = next_part();
    if (part.row < 0) return;
    int32_t id[2];
    int64_t cell[2];
    uint4 kr[2][KC], vr[2][KC], q[KC];
    int32_t t0 = part.begin + wave * kAttnTile;
    ids_of(part, t0, id);
    load_q(part.row, q);
    uint32_t seen = cells_of(part, t0, id, cell);
    load_rows(a.c.k, cell, kr);
    load_rows(a.c.v, cell, vr);
    ids_of(part, t0 + kStep, id);

    for (;;) {
        const Part next = next_part();
        const int32_t next_t0 = next.begin + wave * kAttnTile;
        int32_t next_id[2];
        ids_of(next, next_t0, next_id);
        float m = -INFINITY, l = 0.f;
        f4_t o[DB];
#pragma unroll
        for (int b = 0; b < DB; ++b) o[b] = f4_t{0.f, 0.f, 0.f, 0.f};

        // A wavefront without a tile in this part runs the loop once on masked tokens.
        for (;;) {
            const bool more = t0 + kStep < part.end;
            f4_t s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 r = FULL || 32 * c + 8 * lg < a.head_dim ? kr[u][c] : zero4;
                    s[u] = mfma(__builtin_bit_cast(vec8<T>, r), __builtin_bit_cast(vec8<T>, q[c]), s[u]);
                }
            }
            const uint32_t seen_now = seen;
            const bool mine[2] = {(seen_now >> li & 1) != 0, (seen_now >> (16 + li) & 1) != 0};
            if (more) {
                seen = cells_of(part, t0 + kStep, id, cell);
                ids_of(part, t0 + 2 * kStep, id);
            } else {
                seen = cells_of(next, next_t0, next_id, cell);
                ids_of(next, next_t0 + kStep, id);
                load_q(next.row < 0 ? part.row : next.row, q);
            }
            load_rows(a.c.k, cell, kr);
            // scores in base 2, the running maximum of this lane's head
            float x[8], mx = m;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool ok = seen_now >> (16 * u + 4 * lg + e) & 1;
                    x[4 * u + e] = ok ? s[u][e] * scale : -INFINITY;
                    mx = __builtin_fmaxf(mx, x[4 * u + e]);
                }
            mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
            mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
            if (__any(mx != m)) {
                const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.f : mx));
                l *= f;
#pragma unroll
                for (int b = 0; b < DB; ++b) o[b] *= f;
                m = mx;
            }
            const float base = (m == -INFINITY ? 0.f : m) - Weight<T>::kBias;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __builtin_amdgcn_exp2f(x[e] - base);
                l += x[e];
            }
            uint4 hi, lo;
            Weight<T>::split(x[0], x[1], hi.x, lo.x);
            Weight<T>::split(x[2], x[3], hi.y, lo.y);
            Weight<T>::split(x[4], x[5], hi.z, lo.z);
            Weight<T>::split(x[6], x[7], hi.w, lo.w);
            const vec8<T> ph = __builtin_bit_cast(vec8<T>, hi), pl = __builtin_bit_cast(vec8<T>, lo);
            // V rows to LDS; what is masked is 0 there
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int d = 32 * c + 8 * lg;
                    const uint4 r = mine[u] && (FULL || d < a.head_dim) ? vr[u][c] : zero4;
                    *reinterpret_cast<uint4 *>(&tile[(16 * u + li) * kPitch + d]) = r;
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            load_rows(a.c.v, cell, vr);
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                const s4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(&tile[tr_row * kPitch + 16 * b + tr_col]));
                const s4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(&tile[(16 + tr_row) * kPitch + 16 * b + tr_col]));
                const vec8<T> vv = __builtin_bit_cast(vec8<T>, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
                o[b] = mfma(vv, ph, o[b]);
                o[b] = mfma(vv, pl, o[b]);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (!more) break;
            t0 += kStep;
        }
        // Join the wavefronts: every one's sums in LDS, scaled to the common maximum.
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (lg == 0) {
            jm[wave][li] = m;
            jl[wave][li] = l;
        }
        __syncthreads();
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) mx = __builtin_fmaxf(mx, jm[w][li]);
        const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.f : mx));
        float *const mine_o = reinterpret_cast<float *>(vt[wave]);
        if (li < heads)
#pragma unroll
            for (int b = 0; b < DB; ++b) *reinterpret_cast<f4_t *>(&mine_o[li * DP + 16 * b + 4 * lg]) = o[b] * f;
        __syncthreads();
        for (int i = tid; i < heads * (DP / 4); i += 64 * kAttnWaves) {
            const int h = i / (DP / 4), d = 4 * (i - h * (DP / 4));
            if (!FULL && d >= a.head_dim) continue;
            float hm = -INFINITY, hl = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) hm = __builtin_fmaxf(hm, jm[w][h]);
            f4_t sum = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) {
                hl = __builtin_fmaf(jl[w][h], __builtin_amdgcn_exp2f(jm[w][h] - (hm == -INFINITY ? 0.f : hm)), hl);
                sum += *reinterpret_cast<const f4_t *>(&reinterpret_cast<const float *>(vt[w])[h * DP + d]);
            }
            const int64_t head = head0 + h;
            if (part.parts > 1) {
                const int64_t slot = (int64_t)part_slot(part.w0, wg - part.w0) * a.q_heads + head;
                put_part(&a.part_o[slot * a.head_dim + d], sum[0], sum[1]);
                put_part(&a.part_o[slot * a.head_dim + d + 2], sum[2], sum[3]);
                if (d == 0) put_part(&a.part_ml[2 * slot], hm, hl);
            } else {
                write_row<T>(a, part.row, head, d, sum, hm, hl);
            }
        }
        if (part.parts > 1)
            join_row<T, DP>(a, part.row, part.w0, part.parts, wg - part.w0, per_share, rest, head0, heads);
        if (next.row < 0) break;
        __syncthreads();  // the join is done with the LDS tiles
        part = next;
        t0 = next_t0;
    }
}

int32_t attn_tiles(int32_t q_heads, int32_t kv_heads)
{
    return (int32_t)std::min<int64_t>((int64_t)kv_heads * ((q_heads / kv_heads + 15) / 16), INT32_MAX);
}

// Workgroups per head tile: what the CUs hold at once.
int32_t attn_shares(int32_t tiles, int32_t head_dim)
{
    return std::max(1, kAttnCUs * attn_occupancy(head_dim) / tiles);
}

template <typename T>
void attention_launch(const AttnArgs &a, dim3 grid, hipStream_t s)
{
    const int D = a.head_dim;
#define LORA_ATTN(DP)                                                                                         \
    (D == DP ? launch(lora_paged_attention_kernel<T, DP, true>, grid, 64 * kAttnWaves, 0, s, a)          \
             : launch(lora_paged_attention_kernel<T, DP, false>, grid, 64 * kAttnWaves, 0, s, a))
    if (D <= 64) LORA_ATTN(64);
    else if (D <= 96) LORA_ATTN(96);
    else if (D <= 128) LORA_ATTN(128);
    else LORA_ATTN(256);
#undef LORA_ATTN
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
// Bound by those: 12,907 rows of 4096 70 us (6.0 TB/s); 4001 rows of 8192 with both norms
// and gates 50 us (5.3 TB/s, two sums over the row one after the other); 500 rows of
// 65,536 with both 57 us (4.6 TB/s; in a graph 53, and 283 with the weights asked for early
// too, which spill); 32 rows of 4096 3.1 us, a launch and one trip to memory.  A row of fewer
// than 512 columns leaves lanes of its wavefront idle (seven in eight at 64).
template <typename T, int NC, bool STREAM>
__global__ __launch_bounds__(1024) void
lora_residual_norm_kernel(lora_norm_args a)
{
    __shared__ float wave_sums[16];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int64_t row = blockIdx.x;
    const int chunks = a.hidden / 8;
    // Everything is asked for before anything waits; of the longest rows, which fill the
    // registers, x and res only.
    constexpr bool kEarly = NC <= 4;
    constexpr int NE = kEarly ? NC : 1;
    const int32_t gi = a.gate ? a.gate_idx ? a.gate_idx[row] : 0 : -1;
    const uint4 zero4 = make_uint4(0, 0, 0, 0);
    uint4 res[NC], x[NC], pw[NE], gate[NE], w[NE];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + i * nt;
        const bool in = c < chunks;
        res[i] = in ? load16(a.res, row * a.ldr + 8 * c) : zero4;
        x[i] = a.x && in ? load16(a.x, row * a.ldx + 8 * c) : zero4;
        if (kEarly) {
            pw[i] = a.post_w && in ? load16(a.post_w, 8 * c) : zero4;
            w[i] = a.y && in ? load16(a.w, 8 * c) : zero4;
        }
    }
    if (gi < -1 || gi >= max(a.n_gates, 1)) return;
    if (kEarly) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int c = tid + i * nt;
            gate[i] = gi >= 0 && c < chunks ? load16(a.gate, gi * a.ldg + 8 * c) : zero4;
        }
    }
    float h[NC][8], p[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        unpack8<T>(res[i], h[i]);
        unpack8<T>(x[i], p[i]);
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
            float f[8];
            unpack8<T>(kEarly ? pw[i % NE] : load16(a.post_w, 8 * c), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] = p[i][e] * inv * (f[e] + a.w_offset);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + i * nt;
        if (c >= chunks) continue;
        if (gi >= 0) {
            float g[8];
            unpack8<T>(kEarly ? gate[i % NE] : load16(a.gate, gi * a.ldg + 8 * c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] *= g[e];
        }
        if (a.x)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = __builtin_fmaf(a.alpha, p[i][e], h[i][e]);
        if (a.res_out) store16<STREAM>(a.res_out, row * a.ldro + 8 * c, pack8<T>(h[i]));
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
    }
    if (!a.y) return;
    const float inv = 1.f / __builtin_sqrtf(block_sum(ss, wave_sums) / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + i * nt;
        if (c >= chunks) continue;
        float f[8], y[8];
        unpack8<T>(kEarly ? w[i % NE] : load16(a.w, 8 * c), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[i][e] * inv * (f[e] + a.w_offset);
        store16<STREAM>(a.y, row * a.ldy + 8 * c, pack8<T>(y));
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
        if (s < c->head_dim) return fail(LORA_E_SHAPE, "cache stride %lld < head_dim = %d", (long long)s, c->head_dim);
        if (s % 8) return fail(LORA_E_ALIGN, "cache stride %lld is not a multiple of 8", (long long)s);
    }
    const __int128 reach = (__int128)(c->num_pages - 1) * c->page_stride + (__int128)(c->page_size - 1) * c->token_stride +
                           (__int128)(c->kv_heads - 1) * c->head_stride + c->head_dim;
    if (reach > (__int128)1 << 48) return fail(LORA_E_SHAPE, "the cache's last element is beyond 2^48");
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

// A launch of one workgroup per row has at most 2^32 - 1 threads along its rows.
int check_rows(int32_t n_rows, int threads)
{
    if ((int64_t)n_rows * threads > UINT32_MAX)
        return fail(LORA_E_UNSUPPORTED, "%d rows of %d threads are too many for one launch", n_rows, threads);
    return LORA_OK;
}

// The arrays that a plan writes share no entry with each other or with those it reads, but
// that kv_end may be kv_len and free_top the pages' own: its workgroups each read all the
// lengths, at times of their own.
int check_plan_arrays(const lora_kv_pages &pg, const int32_t *kv_len, const int32_t *new_len, const int32_t *req_slot,
                      const lora_kv_plan_out &o)
{
    struct Range {
        const int32_t *p;
        int64_t n;
        const char *name;
    };
    const int64_t n = pg.n_req, t = o.max_tokens;
    const Range all[] = {{o.kv_end, n, "kv_end"}, {o.free_top, 1, "out free_top"}, {o.status, 4, "status"},
                         {o.q_ptr, n + 1, "q_ptr"}, {o.tok_req, t, "tok_req"}, {o.tok_pos, t, "tok_pos"},
                         {o.slots, t, "slots"}, {o.idx, t, "idx"}, {pg.free_pages, pg.num_pages, "free_pages"},
                         {kv_len, n, "kv_len"}, {new_len, n, "new_len"}, {req_slot, n, "req_slot"},
                         {pg.free_top, 1, "free_top"}};
    constexpr int kKvEnd = 0, kTop = 1, kWritten = 9, kLen = 9, kOldTop = 12, kAll = 13;
    // The table: n rows of max_blocks entries, ld_table apart; what lies between them is none.
    const __int128 ld = 4 * (__int128)pg.ld_table, row = 4 * (__int128)pg.max_blocks;
    for (const Range &x : all) {
        if (!x.p || !x.n || !n) continue;
        const __int128 from = (__int128)reinterpret_cast<uintptr_t>(x.p) - reinterpret_cast<uintptr_t>(pg.block_table);
        const __int128 to = from + 4 * x.n, r = from > 0 ? from / ld : 0;  // in bytes; the row that `from` is in or behind
        const bool here = r < n && from < r * ld + row && to > r * ld, next = r + 1 < n && to > (r + 1) * ld;
        if (here || next) return fail(LORA_E_SHAPE, "block_table and %s overlap", x.name);
    }
    for (int i = 0; i < kWritten; ++i)
        for (int j = i + 1; j < kAll; ++j) {
            const Range &w = all[i], &x = all[j];
            const auto a = reinterpret_cast<uintptr_t>(w.p), b = reinterpret_cast<uintptr_t>(x.p);
            if (!a || !b || a >= b + 4 * x.n || b >= a + 4 * w.n || !w.n || !x.n) continue;
            if (a == b && ((i == kKvEnd && j == kLen) || (i == kTop && j == kOldTop))) continue;
            return fail(LORA_E_SHAPE, "%s and %s overlap", w.name, x.name);
        }
    return LORA_OK;
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
    PlanArgs a{*pages, *out, kv_len, new_len, req_slot, 0, 1, 1};
    a.shift = page_shift(pages->page_size);
    if (a.shift < 0)
        return fail(LORA_E_SHAPE, "page_size = %d is not a power of two in 1..%d", pages->page_size, LORA_KV_MAX_PAGE);
    if (pages->n_req < 0 || pages->n_req > kPlanMaxReq || pages->num_pages < 1 ||
        (int64_t)pages->num_pages * pages->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "n_req = %d, num_pages = %d of %d tokens", pages->n_req, pages->num_pages,
                    pages->page_size);
    // no request that fits its row then ends beyond a 32-bit position
    if (pages->max_blocks < 1 || (int64_t)pages->max_blocks * pages->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "max_blocks = %d of %d tokens (1 page to 2^31 - 1 tokens)", pages->max_blocks,
                    pages->page_size);
    if (pages->ld_table < pages->max_blocks)
        return fail(LORA_E_SHAPE, "max_blocks = %d, ld_table = %lld", pages->max_blocks, (long long)pages->ld_table);
    if (out->max_tokens < 0 || out->reserved != 0)
        return fail(LORA_E_SHAPE, "max_tokens = %d, reserved = %d", out->max_tokens, out->reserved);
    if (!pages->free_pages || !pages->free_top || !out->status || !out->free_top || !out->q_ptr)
        return fail(LORA_E_NULL, "free_pages, free_top, status and q_ptr are required");
    if (pages->n_req > 0 && (!pages->block_table || !kv_len || !new_len || !out->kv_end))
        return fail(LORA_E_NULL, "block_table, kv_len, new_len and kv_end are required");
    if (out->max_tokens > 0 && (!out->tok_req || !out->tok_pos || !out->slots))
        return fail(LORA_E_NULL, "tok_req, tok_pos and slots are required");
    if (const int st = check_plan_arrays(*pages, kv_len, new_len, req_slot, *out)) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int32_t n = pages->n_req;
    if (n > kPlanThreads) {
        launch(lora_kv_plan_chunks_kernel, dim3(1), kPlanThreads, 0, s, a);
        if (out->max_tokens > 0)
            launch(lora_kv_maps_kernel, dim3((unsigned)((out->max_tokens + 255ll) / 256)), 256, 0, s, a);
        return launch_status("step plan");
    }
    // The work there may be: every token row, and every page that the tables can hold.  Up to
    // two of these a thread, since every workgroup makes its sums at the same time.  A plan
    // in place would need the second launch then (2.9 us); while its token rows are few, so
    // most likely are its pages, and one workgroup is faster.  Where they are not it is far
    // slower: 1000 requests giving back 240,000 one-token pages, 504 token rows, 260 us in
    // place against 7.2 with arrays of their own.
    const int64_t moves = out->max_tokens + std::min<int64_t>(pages->num_pages, (int64_t)n * pages->max_blocks);
    const bool in_place = out->kv_end == kv_len || out->free_top == pages->free_top;
    const bool small = n <= 64 && moves <= 1024, medium = n <= 256;
    const int threads = small ? 64 : medium ? 256 : kPlanThreads;
    int64_t groups = std::min<int64_t>((moves + 2 * threads - 1) / (2 * threads), kPlanGroups);
    if (small || (in_place && out->max_tokens <= kPlanThreads)) groups = 1;
    a.move = 1;
    a.finish = groups == 1 || !in_place;
    auto go = [&](unsigned g) {
        if (small) launch(lora_kv_plan_kernel<64>, dim3(g), 64, 0, s, a);
        else if (medium) launch(lora_kv_plan_kernel<256>, dim3(g), 256, 0, s, a);
        else launch(lora_kv_plan_kernel<kPlanThreads>, dim3(g), kPlanThreads, 0, s, a);
    };
    go((unsigned)std::max<int64_t>(groups, 1));
    if (!a.finish) {
        a.finish = 1;
        a.move = 0;
        go(1);
    }
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
    const bool stream_out = 2 * (int64_t)n_rows * ((int64_t)q_heads + 2 * (int64_t)cache->kv_heads) * cache->head_dim > kStreamBytes;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf = cache->type == LORA_TYPE_BF16;
    const int64_t units = ((int64_t)q_heads + cache->kv_heads) * a.units_rot + (int64_t)cache->kv_heads * a.units_v;
    // One workgroup per row, unless there are too few rows to fill the CUs: then one per 256
    // units (32 rows of the 7B shape: 4.4 us against 3.0).
    const int64_t blocks = n_rows < kAppendFill ? std::min<int64_t>((units + 255) / 256, 64) : 1;
    const dim3 grid((unsigned)n_rows, (unsigned)blocks);
    // a row of few units (one GPU's shard of 64/8 heads has 88) in as few wavefronts
    const int threads = (int)std::min<int64_t>((units + 63) / 64 * 64, 256);
    if ((st = check_rows(n_rows, threads))) return st;
#define LORA_APPEND(T, INTER)                                                                      \
    (stream_out ? launch(lora_rope_append_kernel<T, INTER, true>, grid, threads, 0, s, a)         \
                : launch(lora_rope_append_kernel<T, INTER, false>, grid, threads, 0, s, a))
    if (rope->interleaved) {
        if (bf) LORA_APPEND(BF16, true);
        else LORA_APPEND(F16, true);
    } else {
        if (bf) LORA_APPEND(BF16, false);
        else LORA_APPEND(F16, false);
    }
#undef LORA_APPEND
    return launch_status("rotary append");
}

size_t lora_paged_attention_bytes(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim)
{
    if (n_rows < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 8 ||
        head_dim > LORA_KV_MAX_HEAD_DIM || head_dim % 8)
        return 0;
    const int32_t tiles = attn_tiles(q_heads, kv_heads);
    if (tiles > kAttnMaxTiles) return 0;
    const size_t slots = 2 * (size_t)attn_shares(tiles, head_dim) * q_heads;
    return (kAttnCounters * sizeof(uint32_t) + slots * (head_dim + 2) * sizeof(float) + 255) & ~size_t(255);
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
    if (max_blocks < 1 || ld_table < max_blocks || (int64_t)max_blocks * cache->page_size > kAttnMaxSpan)
        return fail(LORA_E_SHAPE, "max_blocks = %d of %d tokens, ld_table = %lld", max_blocks, cache->page_size,
                    (long long)ld_table);
    if (window < 0) return fail(LORA_E_SHAPE, "window = %d", window);
    if (!std::isfinite(scale)) return fail(LORA_E_SHAPE, "scale is not finite");
    if ((int64_t)n_rows * q_heads > (int64_t)1 << 30)
        return fail(LORA_E_SHAPE, "%d rows of %d heads are too many for one launch", n_rows, q_heads);
    if (attn_tiles(q_heads, cache->kv_heads) > kAttnMaxTiles)
        return fail(LORA_E_UNSUPPORTED, "%d key/value heads of %d query heads", cache->kv_heads, q_heads);
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
    a.n_rows = n_rows;
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.n_req = n_req;
    a.max_blocks = max_blocks;
    a.window = window;
    a.shift = page_shift(cache->page_size);
    a.group = q_heads / cache->kv_heads;
    a.head_tiles = (a.group + 15) / 16;
    const int32_t tiles = attn_tiles(q_heads, cache->kv_heads), most = attn_shares(tiles, cache->head_dim);
    // no row is longer than its table or the window, and no share shorter than kAttnMinShare
    const int64_t span = std::min<int64_t>((int64_t)max_blocks * cache->page_size, window > 0 ? window : INT32_MAX);
    const int64_t line = n_rows * ((span + kAttnTile - 1) / kAttnTile + kAttnRowTiles);
    if (line > INT32_MAX - most)  // (rounded up to whole shares)
        return fail(LORA_E_UNSUPPORTED, "%d rows of up to %lld tokens", n_rows, (long long)span);
    a.shares = (int32_t)std::min<int64_t>(most, (line + kAttnMinShare - 1) / kAttnMinShare);
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
    const size_t slots = 2 * (size_t)most * q_heads;
    a.count = static_cast<uint32_t *>(work);
    a.part_o = reinterpret_cast<float *>(a.count + kAttnCounters);
    a.part_ml = a.part_o + slots * cache->head_dim;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int32_t pairs = a.shares * a.kv_heads;
    const dim3 grid((unsigned)(a.head_tiles > 1 ? (pairs + 7) / 8 * 8 * a.head_tiles : pairs));
    if (cache->type == LORA_TYPE_BF16) attention_launch<BF16>(a, grid, s);
    else attention_launch<F16>(a, grid, s);
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
    if (a.n_rows == 0) return LORA_OK;  // whatever the pointers: an empty tensor's is NULL
    if (!a.y && !a.res_out) return fail(LORA_E_NULL, "y and res_out are both NULL");
    if (!a.x && (a.post_w || a.gate)) return fail(LORA_E_NULL, "post_w and gate need x");
    if (!a.gate && a.gate_idx) return fail(LORA_E_NULL, "gate_idx without gate");
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
    // One chunk per thread up to 512 threads, then two: a row of 8192 in 1024 threads of one
    // chunk waits longer at its barriers than it gains (4001 rows with both norms and a
    // gate: 64 us against 54).
    int threads = 64;
    while (threads < 1024 && (threads < 512 ? threads : 2 * threads) < chunks) threads *= 2;
    if ((st = check_rows(a.n_rows, threads))) return st;
    const int nc = (chunks + threads - 1) / threads;
    const bool stream_out = 2 * (int64_t)a.n_rows * a.hidden * ((a.y ? 1 : 0) + (a.res_out ? 1 : 0)) > kStreamBytes;
    const dim3 grid((unsigned)a.n_rows);
    const bool bf = a.type == LORA_TYPE_BF16;
#define LORA_NORM_T(T, NC)                                                                        \
    (stream_out ? launch(lora_residual_norm_kernel<T, NC, true>, grid, threads, 0, s, a)      \
                : launch(lora_residual_norm_kernel<T, NC, false>, grid, threads, 0, s, a))
#define LORA_NORM(NC) (bf ? LORA_NORM_T(BF16, NC) : LORA_NORM_T(F16, NC))
    if (nc <= 1) LORA_NORM(1);
    else if (nc <= 2) LORA_NORM(2);
    else if (nc <= 4) LORA_NORM(4);
    else LORA_NORM(8);
#undef LORA_NORM
#undef LORA_NORM_T
    return launch_status("residual norm");
}

}  // extern "C"
