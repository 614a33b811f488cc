// HIP kernels (gfx950 / CDNA4) and launchers of sampling (lora_sample.h).
#include "lora_sample.h"

#include <cstddef>
#include <type_traits>

#include "step_device.hpp"

namespace lora {
namespace {

constexpr int kSampleThreads = 1024;
constexpr int kWaves = kSampleThreads / 64;
constexpr int kBins = 2 * kSampleThreads;  // of a histogram: two a thread
constexpr int kAhead = 4;                  // segments of 512 logits that a wavefront asks for at a time
constexpr int kUnitBits = 40;              // the largest weight is 2^kUnitBits

// ------------------------------------------------------------------------ logits
struct F32 {
    typedef float elem;
};

// How a logit's bits are read.
template <typename T>
struct Bits;
template <>
struct Bits<F16> {
    static constexpr uint32_t kInf = 0x7c00, kSign = 0x8000;
    static constexpr int kDrop = 13;  // low bits of its values in 32 bits that are never set
};
template <>
struct Bits<BF16> {
    static constexpr uint32_t kInf = 0x7f80, kSign = 0x8000;
    static constexpr int kDrop = 16;
};
template <>
struct Bits<F32> {
    static constexpr uint32_t kInf = 0x7f800000, kSign = 0x80000000;
    static constexpr int kDrop = 0;
};

// Whole numbers in the order of the values (0 and -0 equal): the magnitude's bits, negated where the sign is set; without
// the bits that the type never sets, so that neighbours differ by 1.
template <typename T>
__device__ inline int32_t key_of(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const int32_t mag = (int32_t)((b & 0x7fffffffu) >> Bits<T>::kDrop);
    return (int32_t)b < 0 ? -mag : mag;
}
template <typename T>
__device__ inline float value_of(int32_t key)
{
    const float v = __builtin_bit_cast(float, (uint32_t)(key < 0 ? -key : key) << Bits<T>::kDrop);
    return key < 0 ? -v : v;
}

// Eight neighbouring logits, what one lane loads at a time; 16-bit ones two in a word.
template <typename T>
struct alignas(16) Chunk {
    static constexpr bool kHalf = sizeof(typename T::elem) == 2;
    static constexpr int kWords = kHalf ? 4 : 8;
    static constexpr uint32_t kNone = Bits<T>::kSign | Bits<T>::kInf;
    typedef short s2_t __attribute__((ext_vector_type(2)));
    typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
    uint32_t w[kWords];

    // Logit e of the first four.
    __device__ inline float value(int e) const
    {
        if constexpr (std::is_same_v<T, F16>) return (float)__builtin_bit_cast(h2_t, w[e / 2])[e % 2];
        else if constexpr (kHalf) return __builtin_bit_cast(float, e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else return __builtin_bit_cast(float, w[e]);
    }
    // Logit e of the eight, in LDS.
    __device__ inline float one(int e) const
    {
        if constexpr (std::is_same_v<T, F16>) return (float)reinterpret_cast<const _Float16 *>(w)[e];
        else if constexpr (kHalf) return __builtin_bit_cast(float, (uint32_t)reinterpret_cast<const uint16_t *>(w)[e] << 16);
        else return __builtin_bit_cast(float, w[e]);
    }
    // The last four in the place of the first: loops over the logits take two rounds of four, for little code.
    __device__ inline void swap()
    {
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
            const uint32_t x = w[i];
            w[i] = w[i + kWords / 2];
            w[i + kWords / 2] = x;
        }
    }
    // The second logit in the place of the first, and one behind the last.
    __device__ inline void put(uint32_t bits)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t after = i + 1 < kWords ? w[i + 1] : bits;
            w[i] = kHalf ? w[i] >> 16 | after << 16 : after;
        }
    }
    __device__ inline float largest() const
    {
        if constexpr (std::is_same_v<T, F16>) {
            h2_t m = __builtin_bit_cast(h2_t, w[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(h2_t, w[i]));
            return __builtin_fmaxf((float)m[0], (float)m[1]);
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (kHalf)
                    m = __builtin_fmaxf(m, __builtin_fmaxf(__builtin_bit_cast(float, w[i] << 16),
                                                           __builtin_bit_cast(float, w[i] & 0xffff0000u)));
                else m = __builtin_fmaxf(m, __builtin_bit_cast(float, w[i]));
            }
            return m;
        }
    }
    __device__ inline void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = kHalf ? 0x10001u * kNone : kNone;
    }
    // NaN counts as -inf.
    __device__ inline void clean()
    {
        if constexpr (kHalf) {
            const s2_t inf = {(short)Bits<T>::kInf, (short)Bits<T>::kInf};
            s2_t most = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(s2_t, w[i] & 0x7fff7fffu));
            if (max((int32_t)most[0], (int32_t)most[1]) > (int32_t)Bits<T>::kInf) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const s2_t bad = __builtin_bit_cast(s2_t, w[i] & 0x7fff7fffu) > inf;
                    const uint32_t mask = __builtin_bit_cast(uint32_t, bad);
                    w[i] = (w[i] & ~mask) | (0x10001u * kNone & mask);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = (w[i] & 0x7fffffffu) > Bits<T>::kInf ? kNone : w[i];
        }
    }
    // +inf as 0, all others as -inf.
    __device__ inline void only_infinite()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (kHalf)
                w[i] = ((w[i] & 0xffffu) == Bits<T>::kInf ? 0 : kNone) | (w[i] >> 16 == Bits<T>::kInf ? 0 : kNone) << 16;
            else w[i] = w[i] == Bits<T>::kInf ? 0 : kNone;
        }
    }
};

// A row in chunks, the first of which begins at a 16-byte boundary at or before the row.
template <typename T>
struct Row {
    const uint8_t *base;  // of chunk 0
    int32_t before;       // elements of it that lie before the row
    int32_t vocab, chunks, segments;

    // Logit e, counted from the first chunk's beginning; NaN as -inf.
    __device__ inline float one(int32_t e) const
    {
        const float v = (float)reinterpret_cast<const typename T::elem *>(base)[e];
        return v >= -INFINITY ? v : -INFINITY;
    }
    // The bits of chunk c; what is no logit of the row is -inf.
    __device__ inline Chunk<T> bits(int32_t c) const
    {
        typedef typename T::elem E;
        const int32_t first = 8 * c - before;
        Chunk<T> r;
        r.clear();
        if (first >= 0 && first + 8 <= vocab) {
#pragma unroll
            for (int i = 0; i < Chunk<T>::kWords; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(base + (int64_t)c * (8 * sizeof(E)) + 4 * i);
                r.w[i] = v.x;
                r.w[i + 1] = v.y;
                r.w[i + 2] = v.z;
                r.w[i + 3] = v.w;
            }
        } else if (c < chunks) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const bool in = first + e >= 0 && first + e < vocab;
                if constexpr (Chunk<T>::kHalf) r.put(in ? reinterpret_cast<const uint16_t *>(base)[8 * c + e] : Chunk<T>::kNone);
                else r.put(in ? reinterpret_cast<const uint32_t *>(base)[8 * c + e] : Chunk<T>::kNone);
            }
        }
        return r;
    }
};

// ------------------------------------------------------------------------ weights
// a b + c with c in scalar registers (the compiler copies it into vector registers before every use).
__device__ inline double fma_c(double a, double b, double c)
{
    double r;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "s"(c));
    return r;
}

// floor(2^40 2^y) for y <= 0, to 2^-40 of it before the floor, as a whole number in 64-bit floating point: y = k + f with
// |f| <= 1/2, 2^f = e^(f ln 2) by nine terms of its series, 2^k by the exponent.  2^0 is exact.  The tenth term (2^-36.6 of
// 2^f at f = -1/2) lies on the eighth: f^10 is within 2^-14 of 15/64 f^8, so it costs nothing, and 2^-40.5 of 2^f is left.
// Two y that lie closer than that on both sides of some k + 1/2 may get weights one apart in the wrong order.
__device__ inline double weight_of(double y)
{
    constexpr double kRound = 6755399441055744.0 + kUnitBits;  // 1.5 2^52: a sum's low bits are a whole number, the nearest to y + 40
    constexpr double l = 0.693147180559945309417;
    constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5, c6 = c5 * l / 6, c7 = c6 * l / 7,
                     c8_of_series = c7 * l / 8, c9 = c8_of_series * l / 9, c8 = c8_of_series + c9 * l / 10 * (15.0 / 64);
    y = __builtin_fmax(y, -64.0);
    const double big = y + kRound, f = y - (big - kRound);
    double s = fma_c(f, c9, c8);
    s = fma_c(f, s, c7);
    s = fma_c(f, s, c6);
    s = fma_c(f, s, c5);
    s = fma_c(f, s, c4);
    s = fma_c(f, s, c3);
    s = fma_c(f, s, c2);
    s = fma_c(f, s, l);
    s = __builtin_fma(f, s, 1.0);
    return __builtin_floor(__builtin_ldexp(s, (int)__builtin_bit_cast(uint64_t, big)));
}

// A whole number below 2^52 as an integer.
__device__ inline uint64_t whole(double x)
{
    return __builtin_bit_cast(uint64_t, x + 4503599627370496.0) & 0xfffffffffffffull;
}

// ------------------------------------------------------------------------ sums over the workgroup
#define LORA_SCAN_STEP(ctrl, rows)                                                                             \
    v += (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), ctrl, rows, 0xf, false) << 32 |    \
         (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false)
// Inclusive sums over each row of sixteen lanes, and over the wavefront.
__device__ inline uint64_t row_scan64(uint64_t v)
{
    LORA_SCAN_STEP(0x111, 0xf);  // row_shr:1, 2, 4, 8
    LORA_SCAN_STEP(0x112, 0xf);
    LORA_SCAN_STEP(0x114, 0xf);
    LORA_SCAN_STEP(0x118, 0xf);
    return v;
}
__device__ inline uint64_t wave_scan64(uint64_t v)
{
    v = row_scan64(v);
    LORA_SCAN_STEP(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
    LORA_SCAN_STEP(0x143, 0xc);  // row_bcast:31 into rows 2 and 3
    return v;
}
#undef LORA_SCAN_STEP
__device__ inline uint64_t lane_of(uint64_t v, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ inline float wave_max(float v)
{
#define LORA_MAX_STEP(ctrl, rows) \
    v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, v), __builtin_bit_cast(int, v), ctrl, rows, 0xf, false)))
    LORA_MAX_STEP(0x111, 0xf);
    LORA_MAX_STEP(0x112, 0xf);
    LORA_MAX_STEP(0x114, 0xf);
    LORA_MAX_STEP(0x118, 0xf);
    LORA_MAX_STEP(0x142, 0xa);
    LORA_MAX_STEP(0x143, 0xc);
#undef LORA_MAX_STEP
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

struct Pair {
    uint64_t count, mass;
};

// Sums of the threads before this one, and of all.
__device__ inline Pair group_before(Pair v, Pair *wave_sums, Pair &all)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Pair s{wave_scan64(v.count), wave_scan64(v.mass)};
    __syncthreads();
    if (lane == 63) wave_sums[wave] = s;
    __syncthreads();
    Pair w = wave_sums[lane & (kWaves - 1)];  // sixteen lanes, a wavefront each: sums up to theirs
    w.count = row_scan64(w.count);
    w.mass = row_scan64(w.mass);
    all = Pair{lane_of(w.count, kWaves - 1), lane_of(w.mass, kWaves - 1)};
    Pair before{0, 0};
    if (wave > 0) before = Pair{lane_of(w.count, wave - 1), lane_of(w.mass, wave - 1)};
    return Pair{before.count + s.count - v.count, before.mass + s.mass - v.mass};
}

// ------------------------------------------------------------------------ the draw
// What stays of a row by order: values above `value`, and of those equal to it the first `ties` by index.
struct Border {
    float value;
    int32_t ties;
};

constexpr int kList = 256;                // candidates on a list
constexpr int kListTopK = 128;            // top-k of this many or fewer looks for one
constexpr size_t kSampleLds = 120 << 10;  // for a row's logits, of a workgroup's 160 KB

struct alignas(16) Shared {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    Pair wave_sums[kWaves];
    float wave_best[kWaves], wave_bound[kWaves];
    int32_t wave_at[kWaves];
    // the list: value and index as one number, larger where it comes first; weight; the candidates in order, and their
    // places by index
    uint64_t order[kList], weight[kList], line[kList];
    uint8_t place[kList], place_by_index[kList];
    int32_t chunk[kList];
    int32_t listed;
    uint64_t found_mass;
    int64_t found_count;
    int32_t found, found_ties;
    float found_value;
};

// One workgroup per row.  Its logits are kept in LDS (KEPT), or the row is read again in every pass.
//   - The largest.
//   - For top-k of few, a bound that at least k logits reach: every wavefront gives the value that k / 16 of its lanes' largest
//     reach, and the lowest of these is taken.  What reaches it (for k = 50 of normal logits some 135) is put on a
//     list.  (A row of fewer than 16 segments leaves wavefronts without logits, and a bound that all reach: beyond kList
//     logits such a row takes a histogram.  32 rows of 4,000 with top-k 50 and top-p 19 us, of 9,000 11.5.)
//   - Otherwise, for top-k and top-p, a histogram of how many and what mass lie how far below the largest, and the
//     bin in which the border lies.  If few lie above it, they are put on the list.
//   - On a list of at most 256, a candidate's place in order and by index is the number of those before it, counted by
//     ballots; one wavefront then goes along the list.
//   - Without one: the list of what lies in the border's bin gives the border and how many of its equals stay (or, where
//     that is too much, histograms of the values between two bounds, narrower until a bin is one value); then the
//     mass that stays of each segment of 512 logits, the segment that the draw falls into, and the token in it.
// Counts and masses are whole numbers, so the order of their atomics does not matter.
//
// Where every logit's weight is needed (no filter, top-p), a pass that weighs is some 30 instructions a logit, most of them
// in 64 bits, which run at the rate of 32-bit ones here: 251 rows of 128,257 without a filter take 53 us with the vector
// units busy 68% of it.  A row is one CU's, so a call of few rows leaves the others idle and lasts as long as its slowest
// row: one row of 32,000 with top-k and top-p (a list) 10.5 us, without a filter 15, with a top-p that keeps too many for a
// list 33; 32 rows of all kinds 36.6; 251 rows of 128,257 of all kinds 121.5, where a row is at work for 46 on average and
// the vector units are busy 27%.
// Masses in whole numbers cost 64-bit atomics in LDS and buy draws that are the same every time and exact sums.
template <typename T, bool KEPT>
__global__ __launch_bounds__(kSampleThreads) void lora_sample_kernel(lora_sample_args a)
{
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint64_t seg_mass[];  // [segments], then their ties, then the logits
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t r = blockIdx.x, src = a.rows ? a.rows[r] : r;
    if (src < 0 || src >= a.n_logits) return;
    Row<T> row;
    const uint8_t *const first = static_cast<const uint8_t *>(a.logits) + (int64_t)src * a.ld * (int64_t)sizeof(typename T::elem);
    row.base = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(first) & ~uintptr_t(15));
    row.before = (int32_t)((first - row.base) / sizeof(typename T::elem));
    row.vocab = a.vocab;
    row.chunks = (a.vocab + row.before + 7) / 8;
    row.segments = (row.chunks + 63) / 64;
    uint32_t *const seg_ties = reinterpret_cast<uint32_t *>(seg_mass + (row.segments + 1) / 2 * 2);
    Chunk<T> *const held = reinterpret_cast<Chunk<T> *>(seg_ties + (row.segments + 3) / 4 * 4);
    const float temperature = a.temperature ? a.temperature[r] : 1.f, top_p = a.top_p ? a.top_p[r] : 1.f;
    const float min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u[r];
    const int32_t top_k = a.top_k ? a.top_k[r] : 0;
    if (!(temperature >= 0.f) || temperature == INFINITY || top_k < 0 || !(top_p >= 0.f && top_p <= 1.f) ||
        !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f))
        return;
    // fn(segment, chunk) for the row's segments of 64 chunks, a wavefront each
    auto stream = [&](auto &&fn) __attribute__((always_inline)) {
        Chunk<T> next = row.bits(64 * wave + lane);
        for (int32_t s = wave; s < row.segments; s += kWaves) {
            Chunk<T> c = next;
            next = row.bits(64 * (s + kWaves) + lane);
            c.clean();
            fn(s, c);
        }
    };
    bool infinite = false;  // the largest is +inf: it counts as 0, all others as -inf
    auto each = [&](auto &&fn) __attribute__((always_inline)) {
        auto as_they_count = [&](int32_t s, Chunk<T> &c) __attribute__((always_inline)) {
            if (infinite) c.only_infinite();
            fn(s, c);
        };
        if constexpr (KEPT) {
            for (int32_t s = wave; s < row.segments; s += kWaves) {
                Chunk<T> c = held[64 * s + lane];
                as_they_count(s, c);
            }
        } else {
            stream(as_they_count);
        }
    };
    // fn(value) for every logit
    auto all = [&](auto &&fn) __attribute__((always_inline)) {
        each([&](int32_t, Chunk<T> &c) __attribute__((always_inline)) {
#pragma unroll 1
            for (int i = 0; i < 8; i += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) fn(c.value(e));
                c.swap();
            }
        });
    };

    float best = -INFINITY;  // this thread's largest
    if constexpr (KEPT) {
        // (a short row in one trip to memory: 0.3 us less than one segment ahead, which long ones are as fast with)
        for (int32_t s0 = wave; s0 < row.segments; s0 += kAhead * kWaves) {
            Chunk<T> c[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) c[j] = row.bits(64 * (s0 + j * kWaves) + lane);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int32_t s = s0 + j * kWaves;
                c[j].clean();
                best = __builtin_fmaxf(best, c[j].largest());
                if (s < row.segments) held[64 * s + lane] = c[j];
            }
        }
    } else {
        stream([&](int32_t, Chunk<T> &c) __attribute__((always_inline)) { best = __builtin_fmaxf(best, c.largest()); });
    }
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f;
    const float wave_top = wave_max(best);
    if (by_k && top_k <= kListTopK && temperature > 0.f) {
        float left = best, bound = wave_top;
        for (int32_t need = (top_k + kWaves - 1) / kWaves;;) {
            const uint64_t on = __ballot(left == bound);
            need -= __builtin_popcountll(on);
            if (need <= 0 || bound == -INFINITY) break;
            left = left == bound ? -INFINITY : left;
            bound = wave_max(left);
        }
        if (lane == 0) sh.wave_bound[wave] = bound;
    }
    if (lane == 0) sh.wave_best[wave] = wave_top;
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    float top = sh.wave_best[lane & (kWaves - 1)];
    top = wave_max(top);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    if (temperature == 0.f) {
        int32_t at = INT32_MAX;
        each([&](int32_t s, Chunk<T> &c) __attribute__((always_inline)) {
            if (!__any(c.largest() == top)) return;
#pragma unroll 1
            for (int i = 0; i < 8; i += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c.value(e) == top) at = min(at, 8 * (64 * s + lane) + i + e - row.before);
                c.swap();
            }
        });
#pragma unroll
        for (int d = 1; d < 64; d *= 2) at = min(at, __shfl_xor(at, d));
        if (lane == 0) sh.wave_at[wave] = at;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWaves; ++w) at = min(at, sh.wave_at[w]);
            a.token[r] = at;
            if (a.logprob) a.logprob[r] = 0.f;
        }
        return;
    }
    infinite = top == INFINITY;
    if (infinite) top = 0.f;
    const double rate = 1.44269504088896340736 / (double)temperature;
    auto weight = [&](float v) { return weight_of(((double)v - (double)top) * rate); };
    const double least = (double)min_p * (double)(1ull << kUnitBits);
    auto finish = [&](int32_t token, float v, uint64_t total) {
        a.token[r] = token;
        if (a.logprob)
            a.logprob[r] = (float)(((double)v - (double)top) / (double)temperature -
                                   log((double)total / (double)(1ull << kUnitBits)));
    };
    // Bins by the distance from the largest: 1/64 of a power of two each, the last one takes all beyond.
    const float per = (float)__builtin_fmin(rate * 64.0, 1e30);
    auto bin_of = [&](float v) { return (int32_t)__builtin_fminf((top - v) * per, (float)(kBins - 1)); };

    auto clear = [&]() {
        static_assert(alignof(Shared) % alignof(uint4) == 0 && offsetof(Shared, mass) % alignof(uint4) == 0, "16-byte stores");
        __syncthreads();
        *reinterpret_cast<uint4 *>(&sh.mass[2 * tid]) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint2 *>(&sh.count[2 * tid]) = make_uint2(0, 0);
        __syncthreads();
    };
    auto add = [&](int32_t bin, double w) {
        __hip_atomic_fetch_add(&sh.count[bin], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (by_p) __hip_atomic_fetch_add(&sh.mass[bin], whole(w), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    // This thread's two bins of a histogram, and what lies before them.
    struct Bins {
        uint32_t c0, c1;
        uint64_t m0, m1;
        Pair before;
    };
    auto scan = [&](Pair from, Pair &every) {
        __syncthreads();
        Bins b{sh.count[2 * tid], sh.count[2 * tid + 1], sh.mass[2 * tid], sh.mass[2 * tid + 1], {0, 0}};
        b.before = group_before(Pair{(uint64_t)b.c0 + b.c1, b.m0 + b.m1}, sh.wave_sums, every);
        b.before.count += from.count;
        b.before.mass += from.mass;
        if (tid == 0) sh.found = 0;
        __syncthreads();
        return b;
    };
    // Where a border lies: the bin, what lies before it, and its count.  By count: the bin of the k-th token.  By
    // mass: the first bin at whose end `target` is reached.
    struct Found {
        int32_t bin, ties;
        Pair before;
    };
    auto locate = [&](const Bins &b, bool by_count, double target) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t cb = (int64_t)b.before.count + (i ? b.c0 : 0), ce = cb + (i ? b.c1 : b.c0);
            const uint64_t mb = b.before.mass + (i ? b.m0 : 0), me = mb + (i ? b.m1 : b.m0);
            if (by_count ? cb < top_k && top_k <= ce : (double)mb < target && !((double)me < target)) {
                sh.found = 2 * tid + i;
                sh.found_count = cb;
                sh.found_mass = mb;
                sh.found_ties = (int32_t)(i ? b.c1 : b.c0);
            }
        }
        __syncthreads();
        const Found f{sh.found, sh.found_ties, Pair{(uint64_t)sh.found_count, sh.found_mass}};
        __syncthreads();
        return f;
    };
    // The lowest key for whose value fits() holds; it holds for the largest, and above any for which it does.
    auto first_key = [&](auto &&fits) {
        int32_t lo = key_of<T>(-INFINITY), hi = key_of<T>(top);
        while (lo < hi) {
            const uint32_t step = ((uint32_t)hi - (uint32_t)lo) / 64 + 1;
            const int32_t probe = (int32_t)min((int64_t)lo + (int64_t)lane * step, (int64_t)hi);
            const uint64_t on = __ballot(fits(value_of<T>(probe)));
            const int j = on ? __builtin_ctzll(on) : 64;
            const int32_t to = j < 64 ? __builtin_amdgcn_readlane(probe, j & 63) : hi;
            if (j > 0) lo = __builtin_amdgcn_readlane(probe, (j - 1) & 63) + 1;
            hi = to;
        }
        return lo;
    };

    // One logit onto the list, whose length is counted beyond its end.
    auto put = [&](float v, uint32_t at) {
        const int32_t n = __hip_atomic_fetch_add(&sh.listed, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);  // -0 as 0
        if (n < kList) sh.order[n] = (uint64_t)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32 | ~at;
    };
    // Puts all logits from `bound` up on the list: the chunks that have one, and then a thread for each of their logits.
    auto gather_from = [&](float from) __attribute__((always_inline)) {
        if (tid == 0) sh.found = 0;
        __syncthreads();
        each([&](int32_t s, Chunk<T> &c) __attribute__((always_inline)) {
            if (c.largest() >= from) {
                const int32_t n = __hip_atomic_fetch_add(&sh.found, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                if (n < kList) sh.chunk[n] = 64 * s + lane;
            }
        });
        __syncthreads();
        const int32_t n = sh.found;
        if (n > kList) return n;
        for (int32_t i = tid; i < 8 * n; i += kSampleThreads) {
            const int32_t c = sh.chunk[i / 8];
            const uint32_t at = (uint32_t)(8 * c + i % 8 - row.before);
            if (at >= (uint32_t)row.vocab) continue;
            float v;
            if constexpr (KEPT) v = held[c].one(i % 8);
            else v = row.one(8 * c + i % 8);
            if (infinite) v = v == INFINITY ? 0.f : -INFINITY;
            if (v >= from) put(v, at);
        }
        __syncthreads();
        return sh.listed;
    };
    // Puts all logits of a bin on the list.
    auto gather_bin = [&](int32_t bin) __attribute__((always_inline)) {
        each([&](int32_t s, Chunk<T> &c) __attribute__((always_inline)) {
#pragma unroll 1
            for (int i = 0; i < 8; i += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = c.value(e);
                    const uint32_t at = (uint32_t)(8 * (64 * s + lane) + i + e - row.before);
                    if (bin_of(v) == bin && at < (uint32_t)row.vocab) put(v, at);
                }
                c.swap();
            }
        });
        __syncthreads();
        return sh.listed;
    };
    auto value_on_list = [](uint64_t order) {
        const uint32_t b = (uint32_t)(order >> 32);
        return __builtin_bit_cast(float, b & 0x80000000u ? b & 0x7fffffffu : ~b);
    };
    // The places of the list's n candidates and their weights; each wavefront counts for every sixteenth.
    auto arrange = [&](int32_t n) {
        uint64_t o[kList / 64];
#pragma unroll
        for (int q = 0; q < kList / 64; ++q) o[q] = 64 * q + lane < n ? sh.order[64 * q + lane] : 0;
        if (tid < n) sh.weight[tid] = whole(weight(value_on_list(sh.order[tid])));
#pragma unroll
        for (int q = 0; q < kList / 64; ++q) {
#pragma unroll 1
            for (int l = wave; l < 64 && 64 * q + l < n; l += kWaves) {
                const uint64_t mine = lane_of(o[q], l);
                int sooner = 0, lower = 0;
#pragma unroll
                for (int j = 0; j < kList / 64; ++j) {
                    if (64 * j >= n) break;
                    sooner += __builtin_popcountll(__ballot(o[j] > mine));
                    lower += __builtin_popcountll(__ballot((uint32_t)o[j] > (uint32_t)mine));
                }
                if (lane == 0) {
                    sh.place[sooner] = (uint8_t)(64 * q + l);
                    sh.place_by_index[64 * q + l] = (uint8_t)lower;
                }
            }
        }
        __syncthreads();
    };

    // ---- a list, or where it would begin
    float bound = -INFINITY;
    bool list = by_k && top_k <= kListTopK;
    if (list) {
        const float b = sh.wave_bound[lane & (kWaves - 1)];
        bound = -wave_max(-b);
        if (infinite) bound = bound == INFINITY ? 0.f : -INFINITY;
    }
    Bins bins{};
    uint64_t sum = 0;  // mass of what top-k leaves
    bool counted = false;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        // A histogram: for top-p alone at first, for all that is filtered where a list has come to nothing.
        if ((by_k || by_p) && !counted && (round == 1 || !list) && (round == 1 || !by_k)) {
            counted = true;
            clear();
            uint64_t masses = 0;
            each([&](int32_t, Chunk<T> &c) __attribute__((always_inline)) {
                double mass = 0.0;
#pragma unroll 1
                for (int i = 0; i < 8; i += 4) {
                    double w[4] = {0.0, 0.0, 0.0, 0.0};
                    if (by_p)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = weight(c.value(e));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t b = bin_of(c.value(e));
                        mass += w[e];
                        if (b < kBins - 1) add(b, w[e]);
                    }
                    c.swap();
                }
                masses += whole(mass);
            });
            // the last bin: what the others have not
            __syncthreads();
            Pair others{0, masses}, every;
            for (int i = 2 * tid; i < 2 * tid + 2 && i < kBins - 1; ++i) {
                others.count += sh.count[i];
                others.mass -= sh.mass[i];
            }
            group_before(others, sh.wave_sums, every);
            if (tid == 0) {
                sh.count[kBins - 1] = (uint32_t)(a.vocab - (int64_t)every.count);
                sh.mass[kBins - 1] = every.mass;
            }
            bins = scan(Pair{0, 0}, every);
            if (!by_k) sum = every.mass;
        }
        if (round == 1) break;
        if (counted) {  // top-p alone: a list of all that lies above the end of the border's bin
            const double target = (double)top_p * (double)sum;
            if (target > 0.0) {
                const Found f = locate(bins, false, target);
                list = (int64_t)f.before.count + f.ties <= kList && f.bin < kBins - 1;
                if (list) bound = value_of<T>(first_key([&](float v) { return bin_of(v) <= f.bin; }));
            } else {
                list = true;
                bound = top;
            }
        }
        if (!list) continue;
        const int32_t n = gather_from(bound);
        if (n > kList) continue;
        arrange(n);
        if (wave != 0) return;
        // Four candidates a lane, in order.
        uint64_t w[4], before[4], mass = 0;
        int32_t who[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int32_t rank = 4 * lane + q;
            who[q] = rank < n ? sh.place[rank] : 0;
            w[q] = rank < n ? sh.weight[who[q]] : 0;
            before[q] = mass;
            mass += w[q];
        }
        const uint64_t ahead = wave_scan64(mass) - mass;
        if (by_k) {  // the mass of the first k
            uint64_t k_mass = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) k_mass += 4 * lane + q < top_k ? w[q] : 0;
            sum = lane_of(wave_scan64(k_mass), 63);
        }
        const double target = (double)top_p * (double)sum;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int32_t rank = 4 * lane + q;
            const bool stays = rank < n && (!by_k || rank < top_k) &&
                               (!by_p || rank == 0 || (double)(ahead + before[q]) < target) && (double)w[q] >= least;
            if (rank < n) sh.line[sh.place_by_index[who[q]]] = stays ? w[q] : 0;
        }
        // and by index
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        mass = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = 4 * lane + q < n ? sh.line[4 * lane + q] : 0;
            before[q] = mass;
            mass += w[q];
        }
        const uint64_t upto = wave_scan64(mass), total = lane_of(upto, 63);
        const uint64_t at = min((uint64_t)((double)u * (double)total), total - 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint64_t from = upto - mass + before[q];
            if (from <= at && at < from + w[q]) sh.found = 4 * lane + q;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int32_t chosen = sh.found;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (64 * q + lane < n && sh.place_by_index[64 * q + lane] == chosen) {
                const uint64_t order = sh.order[64 * q + lane];
                finish((int32_t)~(uint32_t)order, value_on_list(order), total);
            }
        return;
    }

    // ---- without one: the border
    Border border{-INFINITY, a.vocab + 8};  // all stay (what is no logit, too: it weighs 0)
#pragma unroll 1
    for (int what = by_k ? 0 : 1; what < (by_p ? 2 : 1); ++what) {
        const bool by_count = what == 0;
        const double target = by_count ? 0.0 : (double)top_p * (double)sum;
        Border b{top, 1};
        if (by_count || target > 0.0) {
            Found f = locate(bins, by_count, target);
            const int32_t bin = f.bin;
            if (f.ties <= kList) {  // (`ties` counts the bin)
                if (tid == 0) sh.listed = 0;
                __syncthreads();
                const int32_t n = gather_bin(bin);  // (f.ties)
                arrange(n);
                if (wave == 0) {
                    uint64_t w[4], before[4], mass = 0;
                    int32_t who[4], left = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int32_t rank = 4 * lane + q;
                        who[q] = rank < n ? sh.place[rank] : 0;
                        w[q] = rank < n ? sh.weight[who[q]] : 0;
                        before[q] = mass;
                        mass += w[q];
                    }
                    const uint64_t ahead = f.before.mass + wave_scan64(mass) - mass;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int32_t rank = 4 * lane + q;
                        const bool stays = rank < n && (by_count ? (int64_t)f.before.count + rank < top_k : (double)(ahead + before[q]) < target);
                        left += __builtin_popcountll(__ballot(stays));
                    }
                    // the last that stays, and its equals before it
                    const float value = value_on_list(sh.order[sh.place[max(left - 1, 0)]]);
                    int32_t ties = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int32_t rank = 4 * lane + q;
                        ties += __builtin_popcountll(__ballot(rank < left && value_on_list(sh.order[who[q]]) == value));
                        if (rank == left - 1) sh.found_mass = ahead + before[q] + w[q];
                    }
                    if (lane == 0) {
                        sh.found_value = value;
                        sh.found_ties = ties;
                    }
                }
                __syncthreads();
                b = Border{sh.found_value, sh.found_ties};
                if (by_count) sum = sh.found_mass;
                __syncthreads();
            } else {
                // what lies in it, from the least to the largest
                float least_in = INFINITY, most_in = -INFINITY;
                all([&](float v) __attribute__((always_inline)) {
                    const bool in = bin_of(v) == bin;
                    least_in = in ? __builtin_fminf(least_in, v) : least_in;
                    most_in = in ? __builtin_fmaxf(most_in, v) : most_in;
                });
                least_in = -wave_max(-least_in);
                most_in = wave_max(most_in);
                if (lane == 0) {
                    sh.wave_best[wave] = most_in;
                    sh.wave_bound[wave] = -least_in;
                }
                __syncthreads();
                most_in = wave_max(sh.wave_best[lane & (kWaves - 1)]);
                least_in = -wave_max(sh.wave_bound[lane & (kWaves - 1)]);
                int32_t lo = key_of<T>(least_in), hi = key_of<T>(most_in);
                while (lo < hi) {
                    const int shift = max(0, 32 - __builtin_clz((uint32_t)hi - (uint32_t)lo) - 11);
                    const float from = value_of<T>(lo), to = value_of<T>(hi);
                    clear();
                    all([&](float v) __attribute__((always_inline)) {
                        if (v >= from && v <= to)
                            add((int32_t)(((uint32_t)hi - (uint32_t)key_of<T>(v)) >> shift), by_p ? weight(v) : 0.0);
                    });
                    Pair every;
                    f = locate(scan(f.before, every), by_count, target);
                    hi = (int32_t)((uint32_t)hi - ((uint32_t)f.bin << shift));
                    if (shift == 0) break;
                    const uint32_t rest = (uint32_t)hi - (uint32_t)lo;
                    if (rest > (1u << shift) - 1) lo = (int32_t)((uint32_t)hi - ((1u << shift) - 1));
                }
                b.value = value_of<T>(hi);
                const uint64_t w = whole(weight(b.value));
                if (by_count) {
                    b.ties = (int32_t)(top_k - (int64_t)f.before.count);
                    sum = f.before.mass + (uint64_t)b.ties * w;
                } else {  // equals stay while the mass before them is below the target
                    int32_t less = 0, more = f.ties;
                    while (less < more) {
                        const int32_t mid = less + (more - less) / 2;
                        if ((double)(f.before.mass + (uint64_t)mid * w) < target) less = mid + 1;
                        else more = mid;
                    }
                    b.ties = less;
                }
            }
        }
        if (what == 1 && by_k && b.value == border.value) b.ties = min(b.ties, border.ties);
        if (what == 0 || !by_k || b.value >= border.value) border = b;
    }
    if (min_p > 0.f) {
        const float v = value_of<T>(first_key([&](float x) { return weight(x) >= least; }));
        if (v > border.value) border = Border{v, a.vocab + 8};
    }

    // ---- what stays, by segments
    each([&](int32_t s, Chunk<T> &c) __attribute__((always_inline)) {
        double mass = 0.0;
        uint32_t ties = 0;
        if (__any(c.largest() >= border.value)) {
#pragma unroll 1
            for (int i = 0; i < 8; i += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = c.value(e);
                    mass += weight(v > border.value ? v : -INFINITY);
                    ties += v == border.value ? 1 : 0;
                }
                c.swap();
            }
        }
        const uint64_t m = lane_of(wave_scan64(whole(mass)), 63), n = lane_of(wave_scan64(ties), 63);
        if (lane == 0) {
            seg_mass[s] = m;
            seg_ties[s] = (uint32_t)n;
        }
    });
    __syncthreads();
    const uint64_t tie = whole(weight(border.value));
    const int32_t per_thread = (row.segments + kSampleThreads - 1) / kSampleThreads;
    const int32_t s0 = min(tid * per_thread, row.segments), s1 = min(s0 + per_thread, row.segments);
    auto stays = [&](int32_t s, int64_t left) {  // mass of a segment whose first `left` equals stay
        return seg_mass[s] + (uint64_t)max((int64_t)0, min(left, (int64_t)seg_ties[s])) * tie;
    };
    Pair own{0, 0}, every;
    for (int32_t s = s0; s < s1; ++s) own.count += seg_ties[s];
    int64_t left0 = border.ties;  // (all equals stay where there are more than logits)
    if (border.ties <= a.vocab) left0 -= (int64_t)group_before(own, sh.wave_sums, every).count;
    int64_t left = left0;
    for (int32_t s = s0; s < s1; ++s) {
        own.mass += stays(s, left);
        left -= seg_ties[s];
    }
    uint64_t before = group_before(own, sh.wave_sums, every).mass;
    const uint64_t total = every.mass, at = min((uint64_t)((double)u * (double)total), total - 1);
    if (before <= at && at < before + own.mass) {
        left = left0;
        for (int32_t s = s0; s < s1; ++s) {
            const uint64_t m = stays(s, left);
            if (before <= at && at < before + m) {
                sh.found = s;
                sh.found_mass = before;
                sh.found_count = left;
            }
            before += m;
            left -= seg_ties[s];
        }
    }
    __syncthreads();
    // The token in its segment, by one wavefront.
    if (wave != 0) return;
    const int32_t c = 64 * sh.found + lane;
    Chunk<T> chunk = row.bits(c);
    chunk.clean();
    if (infinite) chunk.only_infinite();
    float v[8];
    int32_t equals = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = chunk.value(e % 4);
        if (e == 3) chunk.swap();
        equals += v[e] == border.value ? 1 : 0;
    }
    int64_t room = sh.found_count - (int64_t)(wave_scan64(equals) - equals);
    uint64_t w[8], mass = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool equal = v[e] == border.value;
        w[e] = whole(weight(v[e] > border.value || (equal && room > 0) ? v[e] : -INFINITY));
        room -= equal ? 1 : 0;
        mass += w[e];
    }
    uint64_t from = sh.found_mass + wave_scan64(mass) - mass;
    if (from <= at && at < from + mass) {
        float value = 0.f;
        int32_t token = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (from <= at && at < from + w[e]) {
                token = 8 * c + e - row.before;
                value = v[e];
            }
            from += w[e];
        }
        finish(token, value, total);
    }
}

int32_t sample_segments(int32_t vocab) { return (vocab + 7 + 7) / 8 / 64 + 1; }

// LDS beside the histograms: segments' masses and ties, and the keys where they are kept.
size_t sample_lds(int32_t vocab, int elem, bool kept)
{
    const size_t segments = sample_segments(vocab);
    return (segments + 1) / 2 * 16 + (segments + 3) / 4 * 16 + (kept ? segments * 512 * elem : 0);
}

template <typename T>
void sample_launch(const lora_sample_args &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.n_rows);
    const size_t lds = sample_lds(a.vocab, sizeof(typename T::elem), true);
    if (lds <= kSampleLds) launch(lora_sample_kernel<T, true>, grid, kSampleThreads, lds, s, a);
    else launch(lora_sample_kernel<T, false>, grid, kSampleThreads, sample_lds(a.vocab, 0, false), s, a);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_sample_bytes(int32_t n_rows, int32_t vocab)
{
    if (n_rows < 0 || vocab < 1 || vocab > LORA_SAMPLE_MAX_VOCAB) return 0;
    return 256;
}

int lora_sample(void *stream, const lora_sample_args *args)
{
    clear_error();
    if (!args) return fail(LORA_E_NULL, "args is NULL");
    const lora_sample_args &a = *args;
    if (a.type != LORA_TYPE_F16 && a.type != LORA_TYPE_BF16 && a.type != LORA_TYPE_F32)
        return fail(LORA_E_UNSUPPORTED, "unknown type %d", a.type);
    if (a.n_rows < 0 || a.n_logits < 0 || (!a.rows && a.n_logits < a.n_rows))
        return fail(LORA_E_SHAPE, "n_rows = %d, n_logits = %d", a.n_rows, a.n_logits);
    if (a.vocab < 1 || a.vocab > LORA_SAMPLE_MAX_VOCAB)
        return fail(LORA_E_SHAPE, "vocab = %d outside 1..%d", a.vocab, LORA_SAMPLE_MAX_VOCAB);
    if (a.n_rows == 0) return LORA_OK;
    if (a.ld < a.vocab || a.ld > (int64_t)1 << 40) return fail(LORA_E_SHAPE, "leading dimension of logits = %lld", (long long)a.ld);
    if ((!a.logits && a.n_logits > 0) || !a.u || !a.token) return fail(LORA_E_NULL, "logits, u and token are required");
    const uintptr_t mask = a.type == LORA_TYPE_F32 ? 3 : 1;
    if (reinterpret_cast<uintptr_t>(a.logits) & mask) return fail(LORA_E_ALIGN, "logits must be aligned to their elements");
    for (const void *p : {(const void *)a.rows, (const void *)a.temperature, (const void *)a.top_k, (const void *)a.top_p,
                          (const void *)a.min_p, (const void *)a.u, (const void *)a.token, (const void *)a.logprob})
        if (reinterpret_cast<uintptr_t>(p) & 3) return fail(LORA_E_ALIGN, "settings and outputs must be 4-byte aligned");
    if (!a.work) return fail(LORA_E_NULL, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(a.work) & 255) return fail(LORA_E_ALIGN, "workspace must be 256-byte aligned");
    const size_t need = lora_sample_bytes(a.n_rows, a.vocab);
    if (a.work_bytes < need) return fail(LORA_E_SHAPE, "workspace of %zu bytes < %zu", a.work_bytes, need);
    int st = check_rows(a.n_rows, kSampleThreads);
    if (st) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.type == LORA_TYPE_F16) sample_launch<F16>(a, s);
    else if (a.type == LORA_TYPE_BF16) sample_launch<BF16>(a, s);
    else sample_launch<F32>(a, s);
    return launch_status("sample");
}

}  // extern "C"
