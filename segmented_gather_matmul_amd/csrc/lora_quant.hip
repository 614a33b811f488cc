// HIP kernels (gfx950 / CDNA4) and launchers of the quantised key/value cache (lora_quant.h): the append
// that quantises what it writes, reading back, and attention over the cache.
#include "lora_quant.h"

#include "step_device.hpp"

namespace lora {
namespace {

// ------------------------------------------------------------------------ the format
constexpr int kBlock = LORA_QUANT_BLOCK;

// Exponent bytes written for a type: its least and largest (lora_quant.h).
template <typename T, int BITS>
struct Exponents;
template <>
struct Exponents<F16, 4> {
    static constexpr int kLeast = 127 - 23, kMost = 127 + 13;
};
template <>
struct Exponents<F16, 8> {
    static constexpr int kLeast = 127 - 15, kMost = 127 + 7;
};
template <>
struct Exponents<BF16, 4> {
    static constexpr int kLeast = 127 - 125, kMost = 127 + 125;
};
template <>
struct Exponents<BF16, 8> {
    static constexpr int kLeast = 127 - 117, kMost = 127 + 119;
};
constexpr int kNanExponent = 255;

// The exponent byte of a block from the bits of its largest magnitude: adding the mantissa's distance
// from 2 to 1.75 (of 7) or 1.8125 (of 464) carries into the exponent for what does not fit.
template <typename T, int BITS>
__device__ inline int exponent_of(uint32_t most)
{
    if (most >= 0x7f800000u) return kNanExponent;
    const int e = (int)((most + (BITS == 4 ? 0x200000u : 0x180000u)) >> 23) - (BITS == 4 ? 2 : 8);
    return min(max(e, Exponents<T, BITS>::kLeast), Exponents<T, BITS>::kMost);
}

__device__ inline float power_of(uint32_t exponent) { return __builtin_bit_cast(float, exponent << 23); }

// Eight columns' codes: one word of 4-bit codes, two of 8-bit ones.
template <int BITS>
struct Codes {
    uint32_t w[BITS / 4];
};

// x / scale, rounded to nearest even, as codes.  (The 4-bit conversion takes what is too large to the
// largest code by itself; the 8-bit one would make it NaN.)
template <int BITS>
__device__ inline Codes<BITS> codes_of(const float (&x)[8], float scale)
{
    Codes<BITS> r;
    if constexpr (BITS == 4) {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
        r.w[0] = w;
    } else {
        typedef short s2 __attribute__((ext_vector_type(2)));
        const float most = 448.f * scale;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_amdgcn_fmed3f(x[e], -most, most);
        s2 a = {0, 0}, b = {0, 0};
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, y[0], y[1], scale, false);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, y[2], y[3], scale, true);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, y[4], y[5], scale, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, y[6], y[7], scale, true);
        r.w[0] = __builtin_bit_cast(uint32_t, a);
        r.w[1] = __builtin_bit_cast(uint32_t, b);
    }
    return r;
}

// Two values an instruction, exactly; a scale of exponent 255 makes every one NaN.
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
#define LORA_PAIRS(T2, name4, name8)                                                      \
    __device__ inline uint4 values_of(T2, const uint32_t (&w)[1], float s)                \
    {                                                                                     \
        return make_uint4(__builtin_bit_cast(uint32_t, name4(w[0], s, 0)),                \
                          __builtin_bit_cast(uint32_t, name4(w[0], s, 1)),                \
                          __builtin_bit_cast(uint32_t, name4(w[0], s, 2)),                \
                          __builtin_bit_cast(uint32_t, name4(w[0], s, 3)));               \
    }                                                                                     \
    __device__ inline uint4 values_of(T2, const uint32_t (&w)[2], float s)                \
    {                                                                                     \
        return make_uint4(__builtin_bit_cast(uint32_t, name8(w[0], s, false)),            \
                          __builtin_bit_cast(uint32_t, name8(w[0], s, true)),             \
                          __builtin_bit_cast(uint32_t, name8(w[1], s, false)),            \
                          __builtin_bit_cast(uint32_t, name8(w[1], s, true)));            \
    }
LORA_PAIRS(F16, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8)
LORA_PAIRS(BF16, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8)
#undef LORA_PAIRS

template <int BITS>
__device__ inline Codes<BITS> load_codes(const uint8_t *p)
{
    Codes<BITS> r;
    if constexpr (BITS == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    }
    return r;
}
template <int BITS>
__device__ inline void store_codes(uint8_t *p, const Codes<BITS> &c)
{
    if constexpr (BITS == 4) *reinterpret_cast<uint32_t *>(p) = c.w[0];
    else *reinterpret_cast<uint2 *>(p) = make_uint2(c.w[0], c.w[1]);
}

// Where the cells of a slot begin: codes and exponents, in bytes.
struct Cell {
    int64_t code, exp;
};
__device__ inline Cell cell_of(const lora_quant_cache &c, int shift, int32_t slot)
{
    const int64_t page = slot >> shift, off = slot & ((1 << shift) - 1);
    return Cell{page * c.page_stride + off * c.token_stride, page * c.exp_page_stride + off * c.exp_token_stride};
}

// ------------------------------------------------------------------------ rotary positions and append
struct QuantAppendArgs {
    int32_t n_rows, q_heads, kv_heads, head_dim, rot, n_axes, shift;
    int32_t units_q;   // chunks of a head of q, or pairs of chunks that turn together
    int32_t units_kv;  // chunks of a padded head of k or v
    int32_t n_q;       // units of all heads of q, rounded up to a multiple of 4
    void *q_out;
    const void *q, *k, *v;
    int64_t ldqo, ldq, ldk, ldv;
    const float *inv_freq;
    const int32_t *axis, *pos, *slots;
    int64_t ld_pos;
    lora_quant_cache c;
};

// cos and sin of position * inv_freq in 64 bits: the product (31 + 24 bits) is kept as p + e, exactly, and
// 1 / (2 pi) to twice 53 bits, so the fraction of a turn is right to 2^-50 at any 32-bit position.
__device__ inline double2 turn_of_64(int32_t pos, float inv_freq)
{
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double p = (double)pos * (double)inv_freq, e = __builtin_fma((double)pos, (double)inv_freq, -p);
    const double whole = rint(p * kHi);
    const double part = __builtin_fma(p, kHi, -whole) + __builtin_fma(p, kLo, e * kHi);
    double2 cs;
    sincospi(2.0 * part, &cs.y, &cs.x);
    return cs;
}

// Largest of four lanes' values, in each of them.
__device__ inline uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
}

// Rows of a launch with one workgroup each: the rows of a page lie 16 to a group, and groups go to the 8 XCDs in turn
// (workgroups do), so that what neighbouring tokens write of a line meets in one L2.
constexpr int kRowGroup = 16;
constexpr int32_t kFillRows = 1024;  // rows that fill the CUs with one workgroup each
__device__ inline int64_t row_of_group(uint32_t b)
{
    return ((int64_t)(b / (8 * kRowGroup)) * 8 + b % 8) * kRowGroup + b / 8 % kRowGroup;
}
unsigned groups_of_rows(int32_t n)
{
    return (unsigned)(((int64_t)n + 8 * kRowGroup - 1) / (8 * kRowGroup) * (8 * kRowGroup));
}

// A workgroup works on one token row (GROUPED: see above; else blockIdx.x, and its units go round over the threads of
// gridDim.y workgroups).  A unit is eight columns of the cells of k or v, four neighbouring lanes a block, or what turns
// together of a head of q.  k is turned in 64 bits: where a value rounds to one code or the next must not hang on the last
// bits of a sine, and 64-bit multiply-adds run at the rate of 32-bit ones here.
//
// What it reads and writes bounds a long call (4096 rows of 64 and 8 heads of 128, 4 bits: 30.3 us, 5.1 TB/s), and the
// sines and turns in 64 bits one with as many heads of k (12,907 rows of 32 heads, 4 bits: 111 us, 4.3 TB/s); a short one
// (32 rows of 32 heads) is 3.6 us of one row's latency.  Rows in groups are 3% faster there, and marking q_out as not
// read again makes 35.7 us into 30.3.  Two units at a time, asked for before the turns, cost more in registers and so in
// wavefronts than they hid: 121 us.
template <typename T, bool INTER, int BITS, bool GROUPED, bool STREAM>
__global__ __launch_bounds__(256) void lora_quant_append_kernel(QuantAppendArgs a)
{
    __shared__ double2 cs[LORA_KV_MAX_HEAD_DIM / 2];
    const int tid = threadIdx.x;
    const int64_t t = GROUPED ? row_of_group(blockIdx.x) : blockIdx.x;
    if (t >= a.n_rows) return;
    const int32_t slot = a.slots[t];
    const int half = a.rot / 2;
    for (int i = tid; i < half; i += blockDim.x) {
        const int ax = a.axis ? a.axis[i] : 0;
        cs[i] = ax >= 0 && ax < a.n_axes ? turn_of_64(a.pos[ax * a.ld_pos + t], a.inv_freq[i]) : make_double2(1.0, 0.0);
    }
    if (slot < 0 || slot >= (int64_t)a.c.num_pages << a.shift) return;
    const Cell cell = cell_of(a.c, a.shift, slot);
    __syncthreads();
    const int n_kv = a.kv_heads * a.units_kv, n_all = a.n_q + 2 * n_kv;
    for (int u = blockIdx.y * blockDim.x + tid; u < n_all; u += blockDim.x * gridDim.y) {
        if (u < a.n_q) {
            const int h = u / a.units_q;
            if (h >= a.q_heads) continue;
            int d = 8 * (u - h * a.units_q), turn = -1;
            if (INTER) turn = d < a.rot ? d / 2 : -1;
            else if (d < half) turn = d;
            else d += half;  // the chunks behind the pairs
            const int64_t from = t * a.ldq + (int64_t)h * a.head_dim + d, to = t * a.ldqo + (int64_t)h * a.head_dim + d;
            const uint4 ra = load16(a.q, from);
            if (turn < 0) {
                store16<STREAM>(a.q_out, to, ra);
                continue;
            }
            float x[8], y[8];
            unpack8<T>(ra, x);
            if (INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float c = (float)cs[turn + e].x, s = (float)cs[turn + e].y;
                    y[2 * e] = __builtin_fmaf(x[2 * e], c, -(x[2 * e + 1] * s));
                    y[2 * e + 1] = __builtin_fmaf(x[2 * e], s, x[2 * e + 1] * c);
                }
                store16<STREAM>(a.q_out, to, pack8<T>(y));
            } else {
                float b[8], z[8];
                unpack8<T>(load16(a.q, from + half), b);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float c = (float)cs[turn + e].x, s = (float)cs[turn + e].y;
                    y[e] = __builtin_fmaf(x[e], c, -(b[e] * s));
                    z[e] = __builtin_fmaf(x[e], s, b[e] * c);
                }
                store16<STREAM>(a.q_out, to, pack8<T>(y));
                store16<STREAM>(a.q_out, to + half, pack8<T>(z));
            }
            continue;
        }
        const bool is_k = u < a.n_q + n_kv;
        const int i = u - a.n_q - (is_k ? 0 : n_kv);
        const int h = i / a.units_kv, d = 8 * (i - h * a.units_kv);
        const void *const src = is_k ? a.k : a.v;
        const int64_t from = t * (is_k ? a.ldk : a.ldv) + (int64_t)h * a.head_dim;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (d < a.head_dim) unpack8<T>(load16(src, from + d), x);
        if (is_k && d < a.rot) {
            if (INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double2 w = cs[d / 2 + e];
                    const double p = x[2 * e], q = x[2 * e + 1];
                    x[2 * e] = (float)__builtin_fma(p, w.x, -(q * w.y));
                    x[2 * e + 1] = (float)__builtin_fma(p, w.y, q * w.x);
                }
            } else {
                const bool first = d < half;
                float b[8];
                unpack8<T>(load16(src, from + (first ? d + half : d - half)), b);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double2 w = cs[(first ? d : d - half) + e];
                    x[e] = (float)__builtin_fma((double)x[e], w.x, (double)b[e] * (first ? -w.y : w.y));
                }
            }
        }
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max(most, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
        most = quad_max(most);
        const int exp = exponent_of<T, BITS>(most);
        uint8_t *const codes = static_cast<uint8_t *>(is_k ? a.c.k : a.c.v) + cell.code + h * a.c.head_stride + d * BITS / 8;
        store_codes<BITS>(codes, codes_of<BITS>(x, power_of(exp == kNanExponent ? 127 : exp)));
        if ((tid & 3) == 0) {
            uint8_t *const exps = is_k ? a.c.k_exp : a.c.v_exp;
            exps[cell.exp + h * a.c.exp_head_stride + d / kBlock] = (uint8_t)exp;
        }
    }
}

// ------------------------------------------------------------------------ reading back
struct QuantReadArgs {
    int32_t n_rows, kv_heads, head_dim, shift;
    int32_t rows, units;  // rows of a workgroup; units of a row
    uint32_t magic;       // 2^32 / units, rounded up: its product with fewer than 2^16 has the quotient in its upper
                          // half; 0 where there is one unit, which 32 bits do not hold
    void *k_out, *v_out;
    int64_t ldko, ldvo;
    const int32_t *slots;
    lora_quant_cache c;
};

// A unit is eight columns of k or v of one row.  A workgroup has a.rows rows (then gridDim.y is 1) or a part of one; a
// thread asks for AHEAD units before it stores the first.  Bound by what it writes, 16 bits a value: 12,907 rows of 32
// heads of 128, of 4 bits, in 45 us (6.0 TB/s); 32,749 rows of 8 heads, of 8 bits, in 35 us (5.8 TB/s).  One row a
// workgroup and one unit a thread at a time took 68 and 52 us; marking the outputs as not read again makes the former 51.
template <typename T, int BITS, bool STREAM, int AHEAD>
__global__ __launch_bounds__(256) void lora_quant_read_kernel(QuantReadArgs a)
{
    const int chunks = a.head_dim / 8, n = a.kv_heads * chunks, first = a.k_out ? 0 : n;
    const int64_t t0 = (int64_t)blockIdx.x * a.rows;
    const int all = a.rows * a.units, step = blockDim.x * gridDim.y;
    for (int f0 = blockIdx.y * blockDim.x + threadIdx.x; f0 < all; f0 += AHEAD * step) {
        Codes<BITS> c[AHEAD];
        uint32_t exp[AHEAD];
        void *to[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int f = f0 + j * step, r = a.rows == 1 ? 0 : a.magic ? (int)__umulhi((uint32_t)f, a.magic) : f;
            const int64_t t = t0 + r;
            const int32_t slot = f < all && t < a.n_rows ? a.slots[t] : -1;
            to[j] = nullptr;
            if (slot < 0 || slot >= (int64_t)a.c.num_pages << a.shift) continue;
            const Cell cell = cell_of(a.c, a.shift, slot);
            const int u = first + f - r * a.units;
            const bool is_k = u < n;
            const int i = is_k ? u : u - n, h = i / chunks, d = 8 * (i - h * chunks);
            const uint8_t *const codes = static_cast<const uint8_t *>(is_k ? a.c.k : a.c.v);
            const uint8_t *const exps = is_k ? a.c.k_exp : a.c.v_exp;
            c[j] = load_codes<BITS>(codes + cell.code + h * a.c.head_stride + d * BITS / 8);
            exp[j] = exps[cell.exp + h * a.c.exp_head_stride + d / kBlock];
            to[j] = static_cast<uint16_t *>(is_k ? a.k_out : a.v_out) + t * (is_k ? a.ldko : a.ldvo) + 8 * (int64_t)i;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (to[j]) store16<STREAM>(to[j], 0, values_of(T{}, c[j].w, power_of(exp[j])));
    }
}

// ------------------------------------------------------------------------ attention
struct QuantArgs : AttnArgs {
    lora_quant_cache c;
};

constexpr int kQWaves = 4, kQTile = 64;
// The two ways to split the rows' tiles (quant_solo): a workgroup's wavefronts take those of a part in turn and join
// at its end, or each wavefront has parts of its own and waits for no other.  A tile of 64 tokens is what the registers
// hold of K and V in flight while the one before is worked on; two workgroups fit a CU up to 128 columns, one beyond.
// (Of 8-bit cells in pages below 16 tokens, whose cells every lane finds for itself, not quite: the 128-column instances
// keep 9 to 14 registers a lane in scratch.  32 rows of 64 to 4096 tokens of 32 heads: 59 us in pages of 16, 65 of 8.)
typedef AttnLine<kQWaves, kQTile, 8, 8, 16, false, 8, 32> GangLine;
typedef AttnLine<kQWaves, kQTile, 4, 2, 16, true, 8, 32> SoloLine;
constexpr int kQSub = kQTile / 16;  // 16-token subtiles of a tile
// Wavefronts per SIMD, and so workgroups per CU, that the registers are kept to.
constexpr int quant_occupancy(int dp) { return dp <= 128 ? 2 : 1; }

// A weight in [0, 2^kBias] as two 16-bit parts, hi + lo, both cut off: fp16 keeps 22 bits of it (and
// none below 2^-38 of the row's largest), bf16 16 bits.
template <typename T>
__device__ inline void split_weight(float p0, float p1, uint32_t &hi, uint32_t &lo);
template <>
__device__ inline void split_weight<F16>(float p0, float p1, uint32_t &hi, uint32_t &lo)
{
    const h2_t h = __builtin_bit_cast(h2_t, __builtin_amdgcn_cvt_pkrtz(p0, p1));
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(p0 - (float)h[0], p1 - (float)h[1]));
}
template <>
__device__ inline void split_weight<BF16>(float p0, float p1, uint32_t &hi, uint32_t &lo)
{
    const uint32_t a = __builtin_bit_cast(uint32_t, p0), b = __builtin_bit_cast(uint32_t, p1);
    const float r0 = p0 - __builtin_bit_cast(float, a & 0xffff0000u), r1 = p1 - __builtin_bit_cast(float, b & 0xffff0000u);
    hi = (a >> 16) | (b & 0xffff0000u);
    lo = (__builtin_bit_cast(uint32_t, r0) >> 16) | (__builtin_bit_cast(uint32_t, r1) & 0xffff0000u);
}

// Largest over the four lanes that hold a column.  (The exchanges are written out, with the two wait states that they
// need behind a vector write: given one value twice, the compiler takes both results for the same.)
__device__ inline float column_max(float x)
{
    float y = x;
    asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    x = y = __builtin_fmaxf(x, y);
    asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    return __builtin_fmaxf(x, y);
}

// One workgroup per (share of the rows, key/value head, 16 of its query heads), as in the 16-bit
// attention, whose split of the rows and join of their parts it takes.
//
// A wavefront walks 64-token tiles, four subtiles of 16.  Scores are S^T = K Q^T on
// v_mfma_f32_16x16x32, on the codes turned into 16-bit values in registers (two an instruction, exactly).  The order of
// the columns within a score does not matter as long as K and Q have the same one, so a lane
// takes whole blocks: its 16 (or 32) bytes of a token are one block of codes with one
// exponent.  V goes the same way from registers to LDS as 16-bit rows, and from there by transposing
// reads to the A operand of O^T += V^T P^T.
//
// The 16 columns of a product are the query heads of a key/value head.  Where a group has 8
// or 4 heads or fewer, the columns hold them R = 2 or 4 times, once for each of R subtiles: every lane
// keeps the scores of its own column's subtile and lays the others aside, so the softmax
// of R subtiles costs what one does, and each copy has its own maximum and sums, which are joined
// at the row's end.
//
// What is rounded: nothing on the way from codes to products, which are summed in 32 bits; the weights, cut to two 16-bit
// parts (split_weight); the output, once.  Maxima, sums and joins are in 32 bits.
//
// Long rows are bound by the cells' bytes: 32 rows of 8192 tokens, 32/32 heads of 128, in 200 us with 4 bits (5.7 TB/s),
// 8 bits at 5.3 TB/s.  32 rows of 64 to 4096 tokens (135 MB) take 34.7 us, of which the read is 22.4 and the rest
// starting, the rows' ends and joins (8 bits: 262 MB, 59 us, the read 43); one row of 131,071 tokens of 1 head 18.4 (a
// read of 3), 256 parts of 8 tiles on half of the places that the CUs have; one of 17 tokens 7.6, loads
// one after another.  All of V converted at the top of a round, in twice the LDS, was slower; joins that load 16 parts
// at a time, and not 8, cost every call registers.  Rows know nothing of each other: a prompt's tokens as rows read the
// cells before them once each (12,907 rows of 16 prompts, 32 heads: 5.0 ms with 4 bits, 8.3 with 8).
template <typename T, int BITS, int DP, int R, typename LINE, bool PAGES>
__global__ __launch_bounds__(64 * kQWaves) __attribute__((amdgpu_waves_per_eu(quant_occupancy(DP)))) void
lora_quant_attention_kernel(QuantArgs a)
{
    typedef short s4 __attribute__((ext_vector_type(4)));
    constexpr int KC = DP / 32;                // 32-column steps of a score
    constexpr int DB = DP / 16;                // 16-column blocks of the output
    constexpr int NB = DP < 128 ? 1 : DP / 128;  // blocks (or, of 64 columns, half a block) a lane takes of a token
    constexpr int W = KC / NB * BITS / 4;      // words of one
    constexpr int PASSES = kQSub / R, G = 16 / R;
    constexpr int kPitch = DP + 16;            // LDS row pitch, elements
    constexpr int kRegion = 32 * kPitch;
    static_assert(kQSub == 4 && (R == 1 || R == 2 || R == 4), "the weights' operand");
    __shared__ __align__(16) uint16_t vt[kQWaves][kRegion];
    __shared__ float jm[kQWaves][16], jl[kQWaves][16];
    static_assert(sizeof(uint16_t) * kRegion >= sizeof(float) * 16 * DP, "the join fits the V tiles");

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int copy = li / G, hcol = li % G;  // the column's subtile of R, and its head
    const int per_share = a.kv_heads * a.head_tiles;
    // the head tiles of one share and key/value head follow each other on one XCD
    int32_t pair = blockIdx.x, ht = 0;
    if (a.head_tiles > 1) {
        const int32_t eight = blockIdx.x / (8 * a.head_tiles);
        ht = blockIdx.x / 8 - eight * a.head_tiles;
        pair = 8 * eight + blockIdx.x % 8;
    }
    if (LINE::kSolo) pair = pair * kQWaves + wave;
    const int32_t wg = pair / a.kv_heads, kvh = pair - wg * a.kv_heads, rest = kvh * a.head_tiles + ht;
    if (wg >= a.shares) return;
    const int heads = min(G, a.group - 16 * ht);  // query heads of this tile
    const int64_t head0 = (int64_t)kvh * a.group + 16 * ht;
    const int32_t in_page = (1 << a.shift) - 1;
    int32_t share, total;
    RowWalk<LINE> walk;
    RowWork rw = first_row(a, wg, walk, share, total);
    if (rw.row >= a.n_rows) return;
    const int32_t line0 = wg * share, line1 = (int32_t)min((int64_t)line0 + share, (int64_t)total);

    // A row's part in this share: tokens [begin, end), of which those before `first` lie before the window; the row has
    // `parts` parts from share w0 on.
    struct Part {
        int32_t row, begin, end, first, w0, parts;
        const int32_t *table;
    };
    auto next_part = [&]() {
        while (rw.row < a.n_rows) {
            const int32_t row_end = rw.tile0 + rw.tiles;
            const int32_t from = max(rw.tile0, line0), to = min(row_end, line1), tile0 = rw.tile0;
            const int32_t n = rw.rs.first + rw.rs.span;
            const Part p{rw.row, rw.rs.first + (from - tile0) * kQTile,
                         rw.rs.first + (int32_t)min((int64_t)(to - tile0) * kQTile, (int64_t)rw.rs.span),
                         a.window > 0 ? max(n - a.window, 0) : 0, tile0 < line0 ? tile0 / share : wg, 1,
                         a.table + (int64_t)rw.rs.req * a.ld_table};
            int32_t last = wg;
            if (row_end > line1) last = (row_end - 1) / share;
            if (row_end < line1) rw = walk.after(a, rw.row, row_end + LINE::kRowTiles);
            else rw.row = a.n_rows;
            if (from < to) return Part{p.row, p.begin, p.end, p.first, p.w0, last - p.w0 + 1, p.table};
            // else the row's tiles lie in the next workgroup's share
        }
        return Part{-1, 0, 0, 0, 0, 0, a.table};
    };
    // This lane's columns: unit c (of KC) is the eight columns from col_of(c) on.
    auto col_of = [&](int c) { return DP < 128 ? 16 * lg + 8 * c : 128 * (c / 4) + 32 * lg + 8 * (c % 4); };
    // Its block j: where its codes and its exponent lie in a cell.  Columns that a head of fewer has not read the last block.
    const int blocks = (a.head_dim + kBlock - 1) / kBlock;
    int code_at[NB], exp_at[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        exp_at[j] = min(DP < 128 ? lg / 2 : 4 * j + lg, blocks - 1);
        code_at[j] = exp_at[j] * (4 * BITS) + (DP < 128 ? (lg & 1) * (2 * BITS) : 0);
    }
    // Tokens t0 + 16 u + li of a tile: table entries, then where their cells begin; a token past the end or
    // without a page reads page 0 and is masked.  Where pages hold whole subtiles (PAGES), a subtile's page and place in
    // it are scalars.
    struct Tile {
        uint32_t code[kQSub][NB][W], exp[kQSub][NB];
    };
    constexpr int kIds = PAGES ? 1 : kQSub;
    const int64_t head_code = kvh * a.c.head_stride, head_exp = kvh * a.c.exp_head_stride;
    const uint32_t lane_code = li * (uint32_t)a.c.token_stride, lane_exp = li * (uint32_t)a.c.exp_token_stride;
    auto ids_of = [&](const Part &p, int32_t t0, int32_t (&id)[kIds]) {
#pragma unroll
        for (int u = 0; u < kIds; ++u)
            id[u] = p.table[max(min(t0 + (PAGES ? 16 * (lane % kQSub) : 16 * u + li), p.end - 1), 0) >> a.shift];
    };
    auto cells_of = [&](const Part &p, int32_t t0, const int32_t (&id)[kIds], Cell (&cell)[kQSub]) {
        uint64_t seen = 0;
#pragma unroll
        for (int u = 0; u < kQSub; ++u) {
            if constexpr (PAGES) {
                const int32_t page = __builtin_amdgcn_readlane(id[0], u), s0 = t0 + 16 * u;
                const bool ok = (uint32_t)page < (uint32_t)a.c.num_pages;
                const uint32_t off = s0 & in_page;
                const uint64_t at = ok ? page : 0;
                cell[u] = Cell{(int64_t)(at * (uint64_t)a.c.page_stride + off * (uint32_t)a.c.token_stride) + head_code,
                               (int64_t)(at * (uint64_t)a.c.exp_page_stride + off * (uint32_t)a.c.exp_token_stride) + head_exp};
                const int before = min(max(p.first - s0, 0), 16), behind = min(max(p.end - s0, 0), 16);
                const uint64_t in = ok ? (1u << behind) - 1 & ~((1u << before) - 1) : 0;
                seen |= in << (16 * u);
            } else {
                const int32_t t = t0 + 16 * u + li;
                const bool ok = t < p.end && t >= p.first && (uint32_t)id[u] < (uint32_t)a.c.num_pages;
                const uint32_t page = ok ? id[u] : 0, off = t & in_page;
                cell[u] = Cell{(int64_t)((uint64_t)page * (uint64_t)a.c.page_stride + off * (uint32_t)a.c.token_stride) + head_code,
                               (int64_t)((uint64_t)page * (uint64_t)a.c.exp_page_stride + off * (uint32_t)a.c.exp_token_stride) + head_exp};
                seen |= (__ballot(ok) & 0xffffu) << (16 * u);
            }
        }
        return seen;
    };
    auto load_tile = [&](const void *codes, const uint8_t *exps, const Cell (&cell)[kQSub], Tile &r) {
#pragma unroll
        for (int u = 0; u < kQSub; ++u) {
            const uint8_t *const code_base = static_cast<const uint8_t *>(codes) + cell[u].code;
            const uint8_t *const exp_base = exps + cell[u].exp;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint8_t *const p = code_base + ((PAGES ? lane_code : 0u) + (uint32_t)code_at[j]);
                if constexpr (W == 2) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(p);
                    r.code[u][j][0] = v.x;
                    r.code[u][j][1] = v.y;
                } else {
#pragma unroll
                    for (int w = 0; w < W; w += 4) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * w);
                        r.code[u][j][w] = v.x;
                        r.code[u][j][w + 1] = v.y;
                        r.code[u][j][w + 2] = v.z;
                        r.code[u][j][w + 3] = v.w;
                    }
                }
                r.exp[u][j] = exp_base[(PAGES ? lane_exp : 0u) + (uint32_t)exp_at[j]];
            }
        }
    };
    // Two subtiles of it.
    auto load_half = [&](const void *codes, const uint8_t *exps, const Cell (&cell)[kQSub], Tile &r, int half) {
        Tile all;  // (what of it is not used is not loaded)
        load_tile(codes, exps, cell, all);
#pragma unroll
        for (int u = 2 * half; u < 2 * half + 2; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
#pragma unroll
                for (int w = 0; w < W; ++w) r.code[u][j][w] = all.code[u][j][w];
                r.exp[u][j] = all.exp[u][j];
            }
    };
    // Unit c of subtile u as 16-bit values.
    auto unit_of = [&](const Tile &r, int u, int c) {
        constexpr int per = KC / NB;  // units of a block
        const int j = c / per, i = c % per;
        uint32_t w[BITS / 4];
#pragma unroll
        for (int k = 0; k < BITS / 4; ++k) w[k] = r.code[u][j][i * (BITS / 4) + k];
        return values_of(T{}, w, power_of(r.exp[u][j]));
    };
    auto load_q = [&](int32_t row, uint4 (&r)[KC]) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d = col_of(c);
            r[c] = make_uint4(0, 0, 0, 0);
            if (hcol < heads && d < a.head_dim) r[c] = load16(a.q, row * a.ldq + (head0 + hcol) * a.head_dim + d);
        }
    };

    constexpr int kStep = LINE::kWaves * kQTile;
    const int turn = LINE::kSolo ? 0 : wave;  // which of a part's tiles it begins with
    const float scale = a.scale * kLog2e;
    uint16_t *const tile = vt[wave];
    const int tr_row = 4 * lg + (li >> 2), tr_col = 4 * (li & 3);
    typedef __attribute__((address_space(3))) s4 *lds4;

    // What is in flight: the K and V cells of this wavefront's next tile (cell, seen), which may be the
    // first of the next part, and the page ids of the tile after it (id).
    Part part = next_part();
    if (part.row < 0) return;
    int32_t id[kIds];
    Cell cell[kQSub];
    Tile kr, vr;
    uint4 q[KC];
    int32_t t0 = part.begin + turn * kQTile;
    ids_of(part, t0, id);
    load_q(part.row, q);
    uint64_t seen = cells_of(part, t0, id, cell);
    load_tile(a.c.k, a.c.k_exp, cell, kr);
    load_tile(a.c.v, a.c.v_exp, cell, vr);
    ids_of(part, t0 + kStep, id);

    for (;;) {
        const Part next = next_part();
        const int32_t next_t0 = next.begin + turn * kQTile;
        int32_t next_id[kIds];
        ids_of(next, next_t0, next_id);
        float m = -INFINITY, l = 0.f;
        f4_t o[DB];
#pragma unroll
        for (int b = 0; b < DB; ++b) o[b] = f4_t{0.f, 0.f, 0.f, 0.f};

        // A wavefront without a tile in this part runs the loop once on masked tokens.
        for (;;) {
            const bool more = t0 + kStep < part.end;
            f4_t s[kQSub];
#pragma unroll
            for (int u = 0; u < kQSub; ++u) {
                s[u] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    s[u] = mfma(__builtin_bit_cast(vec8<T>, unit_of(kr, u, c)), __builtin_bit_cast(vec8<T>, q[c]), s[u]);
            }
            const uint64_t seen_now = seen;
            const bool whole = seen_now == ~(uint64_t)0;
            if (more) {
                seen = cells_of(part, t0 + kStep, id, cell);
                ids_of(part, t0 + 2 * kStep, id);
            } else {
                seen = cells_of(next, next_t0, next_id, cell);
                ids_of(next, next_t0 + kStep, id);
                load_q(next.row < 0 ? part.row : next.row, q);
            }
            load_tile(a.c.k, a.c.k_exp, cell, kr);
            // scores in base 2 of this lane's column and subtiles
            float x[PASSES][4], mx = m;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                f4_t v = s[p * R];
#pragma unroll
                for (int r = 1; r < R; ++r) v = copy == r ? s[p * R + r] : v;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[p][e] = v[e] * scale;
            }
            if (!whole) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    const uint32_t ok = (uint32_t)(seen_now >> (16 * (p * R + copy) + 4 * lg));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[p][e] = ok >> e & 1 ? x[p][e] : -INFINITY;
                }
                // what is masked of V is 0
#pragma unroll
                for (int u = 0; u < kQSub; ++u) {
                    const bool mine = (seen_now >> (16 * u + li) & 1) != 0;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        vr.exp[u][j] = mine ? vr.exp[u][j] : 127;
#pragma unroll
                        for (int w = 0; w < W; ++w) vr.code[u][j][w] = mine ? vr.code[u][j][w] : 0;
                    }
                }
            }
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = __builtin_fmaxf(mx, x[p][e]);
            mx = column_max(mx);
            if (__any(mx != m)) {
                const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.f : mx));
                l *= f;
#pragma unroll
                for (int b = 0; b < DB; ++b) o[b] *= f;
                m = mx;
            }
            const float base = (m == -INFINITY ? 0.f : m) - Weight<T>::kBias;
            uint32_t hi[PASSES][2], lo[PASSES][2];
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[p][e] = __builtin_amdgcn_exp2f(x[p][e] - base);
                    l += x[p][e];
                }
                split_weight<T>(x[p][0], x[p][1], hi[p][0], lo[p][0]);
                split_weight<T>(x[p][2], x[p][3], hi[p][1], lo[p][1]);
            }
#pragma unroll
            for (int half = 0; half < kQSub / 2; ++half) {
                // V rows of two subtiles to LDS
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        *reinterpret_cast<uint4 *>(&tile[(16 * u + li) * kPitch + col_of(c)]) = unit_of(vr, 2 * half + u, c);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                load_half(a.c.v, a.c.v_exp, cell, vr, half);
                // the weights of the two subtiles, each in its own columns
                uint4 wh, wl;
                if constexpr (R == 1) {
                    wh = make_uint4(hi[2 * half][0], hi[2 * half][1], hi[2 * half + 1][0], hi[2 * half + 1][1]);
                    wl = make_uint4(lo[2 * half][0], lo[2 * half][1], lo[2 * half + 1][0], lo[2 * half + 1][1]);
                } else {
                    const int p = 2 * half / R, first = 2 * half % R;
                    const bool on0 = copy == first, on1 = copy == first + 1;
                    wh = make_uint4(on0 ? hi[p][0] : 0, on0 ? hi[p][1] : 0, on1 ? hi[p][0] : 0, on1 ? hi[p][1] : 0);
                    wl = make_uint4(on0 ? lo[p][0] : 0, on0 ? lo[p][1] : 0, on1 ? lo[p][0] : 0, on1 ? lo[p][1] : 0);
                }
                const vec8<T> ph = __builtin_bit_cast(vec8<T>, wh), pl = __builtin_bit_cast(vec8<T>, wl);
#pragma unroll
                for (int b = 0; b < DB; ++b) {
                    const s4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(&tile[tr_row * kPitch + 16 * b + tr_col]));
                    const s4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(&tile[(16 + tr_row) * kPitch + 16 * b + tr_col]));
                    const vec8<T> vv = __builtin_bit_cast(vec8<T>, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
                    o[b] = mfma(vv, ph, o[b]);
                    o[b] = mfma(vv, pl, o[b]);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            if (!more) break;
            t0 += kStep;
        }
        // Join the wavefronts and the copies: every one's sums in LDS, scaled to the common maximum.
        const int w0 = LINE::kSolo ? wave : 0;
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (lg == 0) {
            jm[wave][li] = m;
            jl[wave][li] = l;
        }
        line_sync<LINE>();
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < LINE::kWaves; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) mx = __builtin_fmaxf(mx, jm[w0 + w][r * G + hcol]);
        const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.f : mx));
        float *const mine_o = reinterpret_cast<float *>(vt[wave]);
        if (hcol < heads)
#pragma unroll
            for (int b = 0; b < DB; ++b) *reinterpret_cast<f4_t *>(&mine_o[li * DP + 16 * b + 4 * lg]) = o[b] * f;
        line_sync<LINE>();
        for (int i = LINE::kSolo ? lane : tid; i < heads * (DP / 4); i += 64 * LINE::kWaves) {
            const int h = i / (DP / 4), d = 4 * (i - h * (DP / 4));
            if (d >= a.head_dim) continue;
            float hm = -INFINITY, hl = 0.f;
#pragma unroll
            for (int w = 0; w < LINE::kWaves; ++w)
#pragma unroll
                for (int r = 0; r < R; ++r) hm = __builtin_fmaxf(hm, jm[w0 + w][r * G + h]);
            f4_t sum = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < LINE::kWaves; ++w)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    hl = __builtin_fmaf(jl[w0 + w][r * G + h], __builtin_amdgcn_exp2f(jm[w0 + w][r * G + h] - (hm == -INFINITY ? 0.f : hm)), hl);
                    sum += *reinterpret_cast<const f4_t *>(&reinterpret_cast<const float *>(vt[w0 + w])[(r * G + h) * DP + d]);
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
            join_row<T, LINE>(a, part.row, part.w0, part.parts, wg - part.w0, per_share, rest, head0, heads);
        if (next.row < 0) break;
        line_sync<LINE>();  // the join is done with the LDS tiles
        part = next;
        t0 = next_t0;
    }
}

// Shares per head tile: what the CUs hold at once.
int32_t quant_shares(int32_t tiles, int32_t head_dim, bool solo)
{
    return std::max(1, kAttnCUs * quant_occupancy(head_dim) * (solo ? kQWaves : 1) / tiles);
}

// Whether wavefronts take parts of their own: where each has half a row and key/value head or more, so that few rows are
// split.  Measured (4 bits, 128 columns, gang / solo): 32 rows of 64-4096 tokens, 32/32 heads 44.8 / 37.0 us, 256 rows of
// 100-900 144 / 107; 61 rows of 1-16,381 tokens, 64/8 heads 41 / 49, one row of 131,071, 8/1 heads 24 / 43.  That is at
// 1024 and 8192 rows x tiles for it and at 512 and 1 against it; between 512 and 1024 both sides have not been measured, and
// the border lies at the upper end (31 rows of 32 heads, a gang's: 37.8 us, 32 of them: 32).  Rows that are not active count.
bool quant_solo(int32_t n_rows, int32_t tiles, int32_t head_dim)
{
    return 2 * (int64_t)n_rows * tiles >= kAttnCUs * kQWaves * quant_occupancy(head_dim);
}

template <typename T, int BITS, int DP, int R, typename LINE>
void quant_attention_launch(const QuantArgs &a, dim3 grid, hipStream_t s)
{
    if (a.c.page_size >= 16) launch(lora_quant_attention_kernel<T, BITS, DP, R, LINE, true>, grid, 64 * kQWaves, 0, s, a);
    else launch(lora_quant_attention_kernel<T, BITS, DP, R, LINE, false>, grid, 64 * kQWaves, 0, s, a);
}

template <typename T, int BITS, int DP, typename LINE>
void quant_attention_launch(const QuantArgs &a, dim3 grid, hipStream_t s)
{
    if (a.group <= 4) quant_attention_launch<T, BITS, DP, 4, LINE>(a, grid, s);
    else if (a.group <= 8) quant_attention_launch<T, BITS, DP, 2, LINE>(a, grid, s);
    else quant_attention_launch<T, BITS, DP, 1, LINE>(a, grid, s);
}

template <typename T, int BITS, typename LINE>
void quant_attention_launch(const QuantArgs &a, dim3 grid, hipStream_t s)
{
    if (a.head_dim <= 64) quant_attention_launch<T, BITS, 64, LINE>(a, grid, s);
    else if (a.head_dim <= 128) quant_attention_launch<T, BITS, 128, LINE>(a, grid, s);
    else quant_attention_launch<T, BITS, 256, LINE>(a, grid, s);
}

template <typename LINE>
void quant_attention_launch(const QuantArgs &a, dim3 grid, hipStream_t s)
{
    const bool bf = a.c.type == LORA_TYPE_BF16;
    if (a.c.bits == 4) bf ? quant_attention_launch<BF16, 4, LINE>(a, grid, s) : quant_attention_launch<F16, 4, LINE>(a, grid, s);
    else bf ? quant_attention_launch<BF16, 8, LINE>(a, grid, s) : quant_attention_launch<F16, 8, LINE>(a, grid, s);
}

// ------------------------------------------------------------------------ host checks
int quant_blocks(int32_t head_dim) { return (head_dim + kBlock - 1) / kBlock; }

int check_quant_cache(const lora_quant_cache *c)
{
    if (!c) return fail(LORA_E_NULL, "cache descriptor is NULL");
    int st = check_type(c->type);
    if (st) return st;
    if (c->bits != 4 && c->bits != 8) return fail(LORA_E_UNSUPPORTED, "bits = %d is not 4 or 8", c->bits);
    if (page_shift(c->page_size) < 0)
        return fail(LORA_E_SHAPE, "page_size = %d is not a power of two in 1..%d", c->page_size, LORA_KV_MAX_PAGE);
    if (c->num_pages < 1 || (int64_t)c->num_pages * c->page_size > INT32_MAX)
        return fail(LORA_E_SHAPE, "num_pages = %d of %d tokens (1 page to 2^31 - 1 tokens)", c->num_pages, c->page_size);
    if (c->kv_heads < 1) return fail(LORA_E_SHAPE, "kv_heads = %d", c->kv_heads);
    if (c->head_dim < 8 || c->head_dim > LORA_KV_MAX_HEAD_DIM || c->head_dim % 8)
        return fail(LORA_E_SHAPE, "head_dim = %d is not a multiple of 8 in 8..%d", c->head_dim, LORA_KV_MAX_HEAD_DIM);
    if (!c->k || !c->v || !c->k_exp || !c->v_exp) return fail(LORA_E_NULL, "cache needs k, v, k_exp and v_exp");
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(LORA_E_ALIGN, "cache k and v must be 16-byte aligned");
    const int64_t blocks = quant_blocks(c->head_dim), bytes = 4 * c->bits * blocks;
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride}) {
        if (s < bytes) return fail(LORA_E_SHAPE, "cache stride %lld < %lld bytes", (long long)s, (long long)bytes);
        if (s % 16) return fail(LORA_E_ALIGN, "cache stride %lld is not a multiple of 16 bytes", (long long)s);
    }
    if ((c->page_size - 1) * (__int128)c->token_stride + bytes > INT32_MAX ||
        (c->page_size - 1) * (__int128)c->exp_token_stride + blocks > INT32_MAX)
        return fail(LORA_E_SHAPE, "a page's tokens span more than 2^31 bytes");
    for (int64_t s : {c->exp_page_stride, c->exp_token_stride, c->exp_head_stride})
        if (s < blocks) return fail(LORA_E_SHAPE, "cache exponent stride %lld < %lld blocks", (long long)s, (long long)blocks);
    auto reach = [&](int64_t page, int64_t token, int64_t head, int64_t cell) {
        return (__int128)(c->num_pages - 1) * page + (__int128)(c->page_size - 1) * token + (__int128)(c->kv_heads - 1) * head + cell;
    };
    if (reach(c->page_stride, c->token_stride, c->head_stride, bytes) > (__int128)1 << 48 ||
        reach(c->exp_page_stride, c->exp_token_stride, c->exp_head_stride, blocks) > (__int128)1 << 48)
        return fail(LORA_E_SHAPE, "the cache's last byte is beyond 2^48");
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

int lora_quant_append(void *stream, int32_t n_rows, int32_t q_heads, void *q_out, int64_t ldqo, const void *q,
                      int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const lora_rope *rope,
                      const int32_t *positions, int64_t ld_pos, const int32_t *slots, const lora_quant_cache *cache)
{
    clear_error();
    int st = check_quant_cache(cache);
    if (st) return st;
    if ((st = check_rope(rope, cache->head_dim))) return st;
    if ((st = check_append(n_rows, q_heads, q_out, ldqo, q, ldq, k, ldk, v, ldv, rope, positions, ld_pos, slots,
                           cache->kv_heads, cache->head_dim)))
        return st;
    if (n_rows == 0) return LORA_OK;
    QuantAppendArgs a{};
    a.n_rows = n_rows;
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.rot = rope->rot_dim;
    a.n_axes = rope->n_axes;
    a.shift = page_shift(cache->page_size);
    a.units_q = rope->interleaved ? cache->head_dim / 8 : cache->head_dim / 8 - rope->rot_dim / 16;
    a.units_kv = quant_blocks(cache->head_dim) * (kBlock / 8);
    a.n_q = (q_heads * a.units_q + 3) / 4 * 4;
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
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t units = a.n_q + 2 * (int64_t)a.kv_heads * a.units_kv;
    // One workgroup per row, unless there are too few rows to fill the CUs: then one per 256 units.
    const bool grouped = n_rows >= kFillRows;
    const int64_t groups = grouped ? 1 : std::min<int64_t>((units + 255) / 256, 64);
    const dim3 grid(grouped ? groups_of_rows(n_rows) : (unsigned)n_rows, (unsigned)groups);
    const int threads = (int)std::min<int64_t>((units + 63) / 64 * 64, 256);
    if ((st = check_rows(n_rows, threads, 8 * kRowGroup))) return st;
    const bool bf = cache->type == LORA_TYPE_BF16, four = cache->bits == 4;
    const bool stream_out = 2 * (int64_t)n_rows * q_heads * cache->head_dim > kStreamBytes;
#define LORA_QAPPEND3(T, INTER, BITS)                                                                           \
    (!grouped ? launch(lora_quant_append_kernel<T, INTER, BITS, false, false>, grid, threads, 0, s, a)          \
     : stream_out ? launch(lora_quant_append_kernel<T, INTER, BITS, true, true>, grid, threads, 0, s, a)        \
                  : launch(lora_quant_append_kernel<T, INTER, BITS, true, false>, grid, threads, 0, s, a))
#define LORA_QAPPEND(T, INTER) (four ? LORA_QAPPEND3(T, INTER, 4) : LORA_QAPPEND3(T, INTER, 8))
    if (rope->interleaved) {
        if (bf) LORA_QAPPEND(BF16, true);
        else LORA_QAPPEND(F16, true);
    } else {
        if (bf) LORA_QAPPEND(BF16, false);
        else LORA_QAPPEND(F16, false);
    }
#undef LORA_QAPPEND
#undef LORA_QAPPEND3
    return launch_status("quantising append");
}

int lora_quant_read(void *stream, int32_t n_rows, void *k_out, int64_t ldko, void *v_out, int64_t ldvo,
                    const int32_t *slots, const lora_quant_cache *cache)
{
    clear_error();
    int st = check_quant_cache(cache);
    if (st) return st;
    if (n_rows < 0) return fail(LORA_E_SHAPE, "n_rows = %d", n_rows);
    if ((int64_t)cache->kv_heads * cache->head_dim > 1 << 28) return fail(LORA_E_UNSUPPORTED, "%d key/value heads", cache->kv_heads);
    if (n_rows == 0) return LORA_OK;
    const int64_t cols = (int64_t)cache->kv_heads * cache->head_dim;
    if (!k_out && !v_out) return fail(LORA_E_NULL, "k_out and v_out are both NULL");
    if (k_out && (st = check_matrix(k_out, ldko, cols, "k_out"))) return st;
    if (v_out && (st = check_matrix(v_out, ldvo, cols, "v_out"))) return st;
    if ((st = check_apart(k_out, ldko, cols, v_out, ldvo, cols, n_rows, false, "k_out and v_out"))) return st;
    if (!slots) return fail(LORA_E_NULL, "slots is NULL");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t units = ((k_out ? 1 : 0) + (v_out ? 1 : 0)) * cols / 8;
    // Where there are rows enough, workgroups with 8 KB of codes or one row, four units a thread at a time; else one unit
    // a thread.  12,907 rows of 32 heads of 128: 4 bits 51.2 us with 4 KB and 44.9 with 8; 8 bits 64.3 with 8, 66.9 with 16.
    const int64_t share = 8192 / cache->bits;
    const bool many = n_rows * units >= kFillRows * (int64_t)1024;
    const int32_t rows = many ? (int32_t)std::max<int64_t>(1, share / units) : 1;
    const int64_t groups = many ? 1 : std::min<int64_t>((units + 255) / 256, 64);
    QuantReadArgs a{n_rows, cache->kv_heads, cache->head_dim, page_shift(cache->page_size), rows, (int32_t)units,
                    (uint32_t)((((uint64_t)1 << 32) + units - 1) / units), k_out, v_out, ldko, ldvo, slots, *cache};
    const dim3 grid((unsigned)((n_rows + (int64_t)rows - 1) / rows), (unsigned)groups);
    const int threads = (int)std::min<int64_t>((rows * units + 63) / 64 * 64, 256);
    if ((st = check_rows(n_rows, threads))) return st;
    const bool bf = cache->type == LORA_TYPE_BF16, four = cache->bits == 4;
    const bool stream_out = 16 * n_rows * units > kStreamBytes;
#define LORA_QREAD(T, BITS)                                                                      \
    (!many ? launch(lora_quant_read_kernel<T, BITS, false, 1>, grid, threads, 0, s, a)           \
     : stream_out ? launch(lora_quant_read_kernel<T, BITS, true, 4>, grid, threads, 0, s, a)     \
                  : launch(lora_quant_read_kernel<T, BITS, false, 4>, grid, threads, 0, s, a))
    if (four) bf ? LORA_QREAD(BF16, 4) : LORA_QREAD(F16, 4);
    else bf ? LORA_QREAD(BF16, 8) : LORA_QREAD(F16, 8);
#undef LORA_QREAD
    return launch_status("quantised read");
}

size_t lora_quant_attention_bytes(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim)
{
    if (n_rows < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 8 ||
        head_dim > LORA_KV_MAX_HEAD_DIM || head_dim % 8)
        return 0;
    const int32_t tiles = attn_tiles(q_heads, kv_heads);
    if (tiles > kAttnMaxTiles) return 0;
    const size_t slots = 2 * (size_t)quant_shares(tiles, head_dim, quant_solo(n_rows, tiles, head_dim)) * q_heads;
    return (kAttnCounters * sizeof(uint32_t) + slots * (head_dim + 2) * sizeof(float) + 255) & ~size_t(255);
}

int lora_quant_attention(void *stream, int32_t n_rows, int32_t q_heads, void *out, int64_t ldo, const void *q,
                         int64_t ldq, const lora_quant_cache *cache, int32_t n_req, const int32_t *block_table,
                         int64_t ld_table, int32_t max_blocks, const int32_t *kv_len, const int32_t *req, float scale,
                         int32_t window, float *lse, void *work, size_t work_bytes)
{
    clear_error();
    int st = check_quant_cache(cache);
    if (st) return st;
    if ((st = check_attention(n_rows, q_heads, out, ldo, q, ldq, n_req, block_table, ld_table, max_blocks, kv_len, scale,
                              window, lse, work, work_bytes, cache->kv_heads, cache->head_dim, cache->page_size,
                              lora_quant_attention_bytes(n_rows, q_heads, cache->kv_heads, cache->head_dim))))
        return st;
    if (n_rows == 0) return LORA_OK;
    QuantArgs a{};
    const int32_t tiles = attn_tiles(q_heads, cache->kv_heads);
    const bool solo = quant_solo(n_rows, tiles, cache->head_dim);
    const int32_t most = quant_shares(tiles, cache->head_dim, solo);
    // rows of two tiles at most are a wavefront's, too (one row of 17 tokens: 8.6 us in a gang, 7.8 alone)
    const bool alone = solo || std::min<int64_t>((int64_t)max_blocks * cache->page_size, window > 0 ? window : INT32_MAX) <= 2 * kQTile;
    auto fill = alone ? fill_attention<SoloLine> : fill_attention<GangLine>;
    if ((st = fill(a, n_rows, q_heads, out, ldo, q, ldq, n_req, block_table, ld_table, max_blocks, kv_len, req, scale, window,
                   lse, work, cache->kv_heads, cache->head_dim, cache->page_size, most)))
        return st;
    a.c = *cache;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (alone) quant_attention_launch<SoloLine>(a, attention_grid(a, kQWaves), s);
    else quant_attention_launch<GangLine>(a, attention_grid(a), s);
    return launch_status("quantised attention");
}

}  // extern "C"
