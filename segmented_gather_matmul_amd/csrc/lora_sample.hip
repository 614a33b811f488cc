// HIP kernels (gfx950 / CDNA4) and launchers of sampling (lora_sample.h).
#include "lora_sample.h"

#include "step_device.hpp"

namespace lora {
namespace {

constexpr int kSampleThreads = 1024;
constexpr int kWaves = kSampleThreads / 64;
constexpr int kBins = 2 * kSampleThreads;  // of a histogram: two a thread
constexpr int kUnitBits = 40;              // the largest weight is 2^kUnitBits

// ------------------------------------------------------------------------ logits
struct F32 {
    typedef float elem;
};

// Logits as whole numbers in the same order (equal ones equal, -0 taken as 0 before): the sign folded into the bits of
// the 32-bit value, without the bits that the type never sets.  0 is below all of them: no token.
template <typename T>
struct Key;
template <>
struct Key<F16> {
    static constexpr int kDrop = 13;
};
template <>
struct Key<BF16> {
    static constexpr int kDrop = 16;
};
template <>
struct Key<F32> {
    static constexpr int kDrop = 0;
};
template <typename T>
__device__ inline uint32_t key_of(float f)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, f);
    return (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) >> Key<T>::kDrop;
}
template <typename T>
__device__ inline float value_of(uint32_t key)
{
    constexpr uint32_t low = (1u << Key<T>::kDrop) - 1;
    const uint32_t s = key << Key<T>::kDrop;
    return __builtin_bit_cast(float, s & 0x80000000u ? s & 0x7fffffffu : ~(s | low));
}

// A row in chunks of eight logits, one lane's load, whose first begins at a 16-byte boundary at or before the row.
template <typename T>
struct Row {
    const uint8_t *base;  // of chunk 0
    int32_t before;       // elements of it that lie before the row
    int32_t vocab, chunks, segments;
    bool infinite;        // its largest is +inf: others count as -inf, that as 0

    // Logits [8 c - before, ...): what is no logit is the number whose key is 0.
    __device__ inline void load(int32_t c, float (&f)[8]) const
    {
        typedef typename T::elem E;
        const int32_t first = 8 * c - before;
        if (first >= 0 && first + 8 <= vocab) {
            E v[8];
#pragma unroll
            for (int i = 0; i < (int)(8 * sizeof(E) / 16); ++i)
                reinterpret_cast<uint4 *>(v)[i] = reinterpret_cast<const uint4 *>(base)[(8 * sizeof(E) / 16) * (int64_t)c + i];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = clean((float)v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t at = first + e;
                f[e] = at >= 0 && at < vocab ? clean((float)reinterpret_cast<const E *>(base)[at + before])
                                             : __builtin_bit_cast(float, 0xffffffffu);
            }
        }
    }
    __device__ inline float clean(float f) const
    {
        f = f > -INFINITY ? f + 0.f : -INFINITY;  // NaN; -0
        return infinite ? (f == INFINITY ? 0.f : -INFINITY) : f;
    }
};

// ------------------------------------------------------------------------ weights
// 2^(j / 128)
struct PowerTable {
    double v[128];
    constexpr PowerTable() : v{}
    {
        for (int j = 0; j < 128; ++j) {
            const double x = j * (0.693147180559945309417 / 128.0);
            double term = 1.0, sum = 1.0;
            for (int n = 1; n < 24; ++n) {
                term *= x / n;
                sum += term;
            }
            v[j] = sum;
        }
    }
};
__constant__ const PowerTable kPowers{};

// floor(2^40 2^y) for y <= 0, to 2^-50 of it before the floor: y = k / 128 + f, 2^y = 2^(k / 128) e^(f ln 2), the
// second factor by four terms of its series (the fifth is below 2^-49), the first from the table and a shift.
__device__ inline uint64_t weight_of(double y, const double *powers)
{
    y = __builtin_fmax(y, -64.0);  // NaN: no logit
    const double big = y * 128.0 + 6755399441055744.0;  // rounded to a whole number in the low bits
    const int32_t k = (int32_t)__builtin_bit_cast(uint64_t, big);
    const double f = __builtin_fma(big - 6755399441055744.0, -1.0 / 128.0, y);
    const double g = f * 0.693147180559945309417;
    double s = __builtin_fma(g, 1.0 / 24.0, 1.0 / 6.0);
    s = __builtin_fma(g, s, 0.5);
    s = __builtin_fma(g, s, 1.0) * g;
    const double t = powers[k & 127], m = __builtin_fma(t, s, t);
    const uint64_t bits = __builtin_bit_cast(uint64_t, m);
    const int shift = 52 - kUnitBits - (k >> 7) + 1023 - (int)(bits >> 52);
    return ((bits & 0xfffffffffffffull) | 0x10000000000000ull) >> (shift < 63 ? shift : 63);
}

// ------------------------------------------------------------------------ sums over the workgroup
__device__ inline uint64_t wave_sum(uint64_t v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}
__device__ inline uint64_t wave_before(uint64_t v)  // sum of the lanes before
{
    const int lane = threadIdx.x & 63;
    uint64_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t x = __shfl_up(s, d);
        if (lane >= d) s += x;
    }
    return s - v;
}

// Sums of the threads before this one, and of all.
__device__ inline uint64_t group_before(uint64_t v, uint64_t *wave_sums, uint64_t &all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t b = wave_before(v);
    __syncthreads();
    if (lane == 63) wave_sums[wave] = b + v;
    __syncthreads();
    uint64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = all;
        all += wave_sums[w];
    }
    return before + b;
}

// ------------------------------------------------------------------------ the draw
// What stays of a row by order: keys above `key`, and of those equal to it the first `ties` by index.
struct Border {
    uint32_t key;
    int32_t ties;
};

struct Shared {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    double powers[128];
    uint64_t wave_sums[kWaves];
    uint64_t found_mass;
    int64_t found_count;
    int32_t found, found_ties;
    float wave_max[kWaves];
    int32_t wave_min[kWaves];
};

// One workgroup per row, several passes over its logits, which stay in the caches:
//   - their largest;
//   - for top-k and top-p, a histogram of how many and what mass lie how far below it; the bin in which the
//     border lies; and a histogram of the keys of that bin (again, while a bin holds several keys), which gives the
//     border's key and how many of its equals stay;
//   - the mass that stays of each segment of 512 logits; the segment that the draw falls into, and the
//     token in it.
// Histograms and masses are whole numbers, so the order of their atomics does not matter.
template <typename T>
__global__ __launch_bounds__(kSampleThreads) void lora_sample_kernel(lora_sample_args a)
{
    __shared__ Shared sh;
    extern __shared__ uint64_t seg_mass[];  // [segments], then their ties
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t r = blockIdx.x, src = a.rows ? a.rows[r] : r;
    const float temperature = a.temperature ? a.temperature[r] : 1.f, top_p = a.top_p ? a.top_p[r] : 1.f;
    const float min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u[r];
    const int32_t top_k = a.top_k ? a.top_k[r] : 0;
    if (src < 0 || src >= a.n_logits || !(temperature >= 0.f) || temperature == INFINITY || top_k < 0 ||
        !(top_p >= 0.f && top_p <= 1.f) || !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f))
        return;
    Row<T> row;
    const uint8_t *const first = static_cast<const uint8_t *>(a.logits) + (int64_t)src * a.ld * (int64_t)sizeof(typename T::elem);
    row.base = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(first) & ~uintptr_t(15));
    row.before = (int32_t)((first - row.base) / sizeof(typename T::elem));
    row.vocab = a.vocab;
    row.chunks = (a.vocab + row.before + 7) / 8;
    row.segments = (row.chunks + 63) / 64;
    row.infinite = false;
    uint32_t *const seg_ties = reinterpret_cast<uint32_t *>(seg_mass + row.segments);
    // Calls fn(segment, logits) for the segments in turn, a wavefront each.
    auto each = [&](auto &&fn) {
        for (int32_t s = wave; s < row.segments; s += kWaves) {
            float f[8];
            if (64 * s + lane < row.chunks) row.load(64 * s + lane, f);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(float, 0xffffffffu);
            fn(s, f);
        }
    };

    float top = -INFINITY;
    each([&](int32_t, const float (&f)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = __builtin_fmaxf(top, f[e]);
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) sh.wave_max[wave] = top;
    if (tid < 128) sh.powers[tid] = kPowers.v[tid];
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, sh.wave_max[w]);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    if (temperature == 0.f) {
        int32_t at = INT32_MAX;
        each([&](int32_t s, const float (&f)[8]) {
#pragma unroll
            for (int e = 7; e >= 0; --e)
                if (f[e] == top) at = min(at, 8 * (64 * s + lane) + e - row.before);
        });
#pragma unroll
        for (int d = 1; d < 64; d *= 2) at = min(at, __shfl_xor(at, d));
        if (lane == 0) sh.wave_min[wave] = at;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWaves; ++w) at = min(at, sh.wave_min[w]);
            a.token[r] = at;
            if (a.logprob) a.logprob[r] = 0.f;
        }
        return;
    }
    if (top == INFINITY) {
        row.infinite = true;
        top = 0.f;
    }
    const double rate = 1.44269504088896340736 / (double)temperature;
    auto weight = [&](float f) { return weight_of(((double)f - (double)top) * rate, sh.powers); };
    // Bins by the distance from the largest: 1/64 of a power of two each, the last one takes all beyond.
    const float per = (float)__builtin_fmin(rate * 64.0, 1e30);
    auto bin_of = [&](float f) { return (int32_t)__builtin_fminf((top - f) * per, (float)(kBins - 1)); };
    const uint32_t top_key = key_of<T>(top), no_key = key_of<T>(-INFINITY);
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f;

    auto clear = [&]() {
        __syncthreads();
        for (int i = tid; i < kBins; i += kSampleThreads) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
    };
    auto add = [&](int32_t bin, uint64_t w) {
        __hip_atomic_fetch_add(&sh.count[bin], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (by_p) __hip_atomic_fetch_add(&sh.mass[bin], w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    // Where a border lies: the bin, and what lies before it (counts and masses beyond `count0`, `mass0`).
    // By count: the bin of the k-th token.  By mass: the first bin at whose end `target` is reached.
    struct Found {
        int32_t bin;
        int64_t count;
        uint64_t mass;
        int32_t ties;
    };
    auto find = [&](bool by_count, double target, int64_t count0, uint64_t mass0) {
        __syncthreads();
        if (tid == 0) sh.found = 0;
        const uint32_t c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
        const uint64_t m0 = sh.mass[2 * tid], m1 = sh.mass[2 * tid + 1];
        uint64_t all;
        const int64_t c = count0 + (int64_t)group_before((uint64_t)c0 + c1, sh.wave_sums, all);
        const uint64_t m = mass0 + group_before(m0 + m1, sh.wave_sums, all);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t cb = c + (i ? c0 : 0), ce = cb + (i ? c1 : c0);
            const uint64_t mb = m + (i ? m0 : 0), me = mb + (i ? m1 : m0);
            const bool here = by_count ? cb < top_k && top_k <= ce : (double)mb < target && !((double)me < target);
            if (here) {
                sh.found = 2 * tid + i;
                sh.found_count = cb;
                sh.found_mass = mb;
                sh.found_ties = (int32_t)(i ? c1 : c0);
            }
        }
        __syncthreads();
        return Found{sh.found, sh.found_count, sh.found_mass, sh.found_ties};
    };
    // The lowest key whose bin is at most b.
    auto first_key = [&](int32_t b) {
        uint32_t lo = no_key, hi = top_key;
        while (lo < hi) {
            const uint32_t step = (hi - lo) / 64 + 1, probe = min(lo + lane * step, hi);
            const uint64_t on = __ballot(bin_of(value_of<T>(probe)) <= b);
            const int j = on ? __builtin_ctzll(on) : 64;
            const uint32_t to = j < 64 ? __builtin_amdgcn_readlane(probe, j & 63) : hi;
            if (j > 0) lo = __builtin_amdgcn_readlane(probe, (j - 1) & 63) + 1;
            hi = to;
        }
        return lo;
    };
    // From a bin of the distances to the border's key: histograms of the keys in it, from the largest down.
    auto refine = [&](Found f, bool by_count, double target) {
        uint32_t hi = f.bin == 0 ? top_key : first_key(f.bin - 1) - 1, lo = first_key(f.bin);
        for (;;) {
            const uint32_t range = hi - lo;
            const int shift = max(0, 32 - (range ? __builtin_clz(range) : 32) - 11);
            clear();
            each([&](int32_t, const float (&x)[8]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t k = key_of<T>(x[e]);
                    if (k >= lo && k <= hi) add((hi - k) >> shift, by_p ? weight(x[e]) : 0);
                }
            });
            f = find(by_count, target, f.count, f.mass);
            hi -= (uint32_t)f.bin << shift;
            if (shift == 0) break;
            lo = max(lo, hi - ((1u << shift) - 1));
        }
        f.bin = (int32_t)hi;
        return f;
    };

    Border border{0, 0};
    if (by_k || by_p) {
        clear();
        uint64_t total = 0;
        uint32_t count = 0;
        each([&](int32_t, const float (&f)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t b = bin_of(f[e]);
                const uint64_t w = by_p ? weight(f[e]) : 0;
                total += w;
                if (b < kBins - 1) add(b, w);
            }
        });
        // the last bin: what the others have not
        __syncthreads();
        for (int i = tid; i < kBins - 1; i += kSampleThreads) {
            count += sh.count[i];
            total -= sh.mass[i];
        }
        uint64_t all, rest;
        group_before(count, sh.wave_sums, all);
        group_before(total, sh.wave_sums, rest);
        if (tid == 0) {
            sh.count[kBins - 1] = (uint32_t)(a.vocab - (int64_t)all);
            sh.mass[kBins - 1] = rest;
        }
        uint64_t sum = 0;  // mass of the first k
        if (by_p && !by_k) {
            __syncthreads();
            group_before(sh.mass[2 * tid] + sh.mass[2 * tid + 1], sh.wave_sums, sum);
        }
        Found by_count{};
        if (by_k) {
            // the histogram of distances is looked at once more for top-p
            const Found f = find(true, 0.0, 0, 0);
            uint64_t keep_m0 = sh.mass[2 * tid], keep_m1 = sh.mass[2 * tid + 1];
            uint32_t keep_c0 = sh.count[2 * tid], keep_c1 = sh.count[2 * tid + 1];
            by_count = refine(f, true, 0.0);
            border = Border{(uint32_t)by_count.bin, (int32_t)(top_k - by_count.count)};
            if (by_p) {
                sum = by_count.mass + (uint64_t)border.ties * weight(value_of<T>(border.key));
                __syncthreads();
                sh.mass[2 * tid] = keep_m0;
                sh.mass[2 * tid + 1] = keep_m1;
                sh.count[2 * tid] = keep_c0;
                sh.count[2 * tid + 1] = keep_c1;
            }
        }
        if (by_p) {
            const double target = (double)top_p * (double)sum;
            Border p{top_key, 1};
            if (target > 0.0) {
                const Found f = refine(find(false, target, 0, 0), false, target);
                p.key = (uint32_t)f.bin;
                // equals stay while the mass before them is below the target
                const uint64_t w = weight(value_of<T>(p.key));
                int32_t lo = 0, hi = f.ties;  // the first that does not
                while (lo < hi) {
                    const int32_t mid = lo + (hi - lo) / 2;
                    if ((double)(f.mass + (uint64_t)mid * w) < target) lo = mid + 1;
                    else hi = mid;
                }
                p.ties = lo;
            }
            if (!by_k || p.key > border.key) border = p;
            else if (p.key == border.key) border.ties = min(border.ties, p.ties);
        }
    }

    // What stays, by segments.
    const uint64_t least = (uint64_t)__builtin_ceil((double)min_p * (double)(1ull << kUnitBits));
    auto kept = [&](float f) {
        const uint64_t w = weight(f);
        return w >= least ? w : 0;
    };
    each([&](int32_t s, const float (&f)[8]) {
        uint64_t mass = 0;
        uint32_t ties = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t k = key_of<T>(f[e]);
            if (k > border.key) mass += kept(f[e]);
            ties += k == border.key ? 1 : 0;
        }
        mass = wave_sum(mass);
        ties = (uint32_t)wave_sum(ties);
        if (lane == 0) {
            seg_mass[s] = mass;
            seg_ties[s] = ties;
        }
    });
    __syncthreads();
    const uint64_t tie = border.key ? kept(value_of<T>(border.key)) : 0;
    const int32_t per_thread = (row.segments + kSampleThreads - 1) / kSampleThreads;
    const int32_t s0 = min(tid * per_thread, row.segments), s1 = min(s0 + per_thread, row.segments);
    uint64_t ties = 0, all, mass = 0, total;
    for (int32_t s = s0; s < s1; ++s) ties += seg_ties[s];
    const int64_t ties_before = (int64_t)group_before(ties, sh.wave_sums, all);
    int64_t left = border.ties - ties_before;
    for (int32_t s = s0; s < s1; ++s) {
        mass += seg_mass[s] + (uint64_t)max((int64_t)0, min(left, (int64_t)seg_ties[s])) * tie;
        left -= seg_ties[s];
    }
    uint64_t before = group_before(mass, sh.wave_sums, total);
    const uint64_t at = min((uint64_t)((double)u * (double)total), total - 1);
    left = border.ties - ties_before;
    for (int32_t s = s0; s < s1; ++s) {
        const uint64_t m = seg_mass[s] + (uint64_t)max((int64_t)0, min(left, (int64_t)seg_ties[s])) * tie;
        if (before <= at && at < before + m) {
            sh.found = s;
            sh.found_mass = before;
            sh.found_count = left;
        }
        before += m;
        left -= seg_ties[s];
    }
    __syncthreads();
    // The token in its segment, by one wavefront.
    if (wave != 0) return;
    const int32_t c = 64 * sh.found + lane;
    float f[8];
    if (c < row.chunks) row.load(c, f);
    else
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(float, 0xffffffffu);
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mine += key_of<T>(f[e]) == border.key ? 1 : 0;
    int64_t room = sh.found_count - (int64_t)wave_before(mine);
    uint64_t w[8], sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t k = key_of<T>(f[e]);
        const bool equal = k == border.key;
        w[e] = k > border.key || (equal && room > 0) ? kept(f[e]) : 0;
        if (equal) --room;
        sum += w[e];
    }
    uint64_t from = sh.found_mass + wave_before(sum);
    if (from <= at && at < from + sum) {
        for (int e = 0; e < 8; ++e) {
            if (at < from + w[e]) {
                a.token[r] = 8 * c + e - row.before;
                if (a.logprob)
                    a.logprob[r] = (float)(((double)f[e] - (double)top) / (double)temperature -
                                           log((double)total / (double)(1ull << kUnitBits)));
                break;
            }
            from += w[e];
        }
    }
}

int32_t sample_segments(int32_t vocab) { return (vocab + 7 + 7) / 8 / 64 + 1; }

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
    const size_t lds = (size_t)sample_segments(a.vocab) * 12;
    const dim3 grid((unsigned)a.n_rows);
    if (a.type == LORA_TYPE_F16) launch(lora_sample_kernel<F16>, grid, kSampleThreads, lds, s, a);
    else if (a.type == LORA_TYPE_BF16) launch(lora_sample_kernel<BF16>, grid, kSampleThreads, lds, s, a);
    else launch(lora_sample_kernel<F32>, grid, kSampleThreads, lds, s, a);
    return launch_status("sample");
}

}  // extern "C"
