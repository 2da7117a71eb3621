// Row operators on activations: the 8-bit row quantizer, the root-mean-square
// norm with the residual's addition, and the gated product silu(a) * b. Each
// writes either 8-bit codes (int8 or E4M3) with one fp32 scale per row, or
// dense rows.
//
// Mathematics. With R = 127 (int8) or 448 (E4M3, the largest finite value) a
// row of values r * p_k, k = 0..K-1, becomes
//     code_k = rnd(R * p_k / P),   scale = r * P / R,   P = max_k |p_k|,
// rnd to the nearest code, ties to even. p is x (quantizer), h * weight with
// r = 1 / sqrt(mean(h^2) + eps) (norm, h = x + residual rounded once to the
// stream's type), or a / (1 + exp(-a)) * b (gated product). The common factor
// r cancels in the codes.
//
// The codes are those of the fp64 formula, as the weight quantizers' are, with
// quotients closer to a tie than fp64 can tell taken as ties. Two steps make
// that cheap:
//  - p * (R / P) is taken in fp32 with a factor slightly below and slightly
//    above R / P, further apart than the relative error Src::kDelta of the
//    fp32 quotient. Where both round to the same code that is the code;
//    elsewhere (about one element in 10^4) the element's p is loaded again and
//    the quotient taken in fp64.
//  - P itself is exact in fp32 for the quantizer. For the norm and the gated
//    product the row's candidates, those within 2 * kDelta of the fp32
//    maximum, are evaluated again in fp64: one element of most rows.
// Rows whose P lies outside [2^-60, 2^120], where fp32 products could lose
// bits to underflow or overflow, and rows with an infinity or a NaN, take
// every step in fp64.
//
// Sums of squares are fp64 (v_fma_f64 runs at the rate of v_fma_f32 here): no
// overflow for any finite fp32 row.
#include <rtq.h>

#include <float.h>

#include <type_traits>

#include "rtq_internal.h"

namespace rtq {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 8;                  // consecutive elements of one lane's load
constexpr int kOutQ8 = 0, kOutF8 = 1, kOutDense = 2;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(_Float16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float to_f(__bf16 v) { return static_cast<float>(v); }

// Forms of a row: K a multiple of eight, so no chunk is partial; any K from
// eight; K below eight.
constexpr int kWhole = 0, kTail = 1, kShort = 2;

// A chunk as it lies in memory. Loads are kept apart from what is done with
// them, so that a thread's loads are all in flight before the first is waited
// for; a chunk goes through memcpy: one 16-byte access per 16 bytes at any
// alignment of the row. A test around the load would be a branch with a wait
// in it, so a thread without a chunk (k beyond the row) reads the row's first
// and drops it, and a partial chunk is read as the row's last eight elements.
template <class T>
struct Raw {
    static constexpr int kWords = kChunk * sizeof(T) / 4;
    uint32_t u[kWords];
    // The chunk at k of the row p, n = K - k or more than eight elements.
    template <int FORM>
    __device__ __forceinline__ void load(const T* p, int64_t k, int n) {
        if constexpr (FORM == kShort) {
            T t[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j) t[j] = j < n ? p[k + j] : static_cast<T>(0.0f);
            __builtin_memcpy(u, t, sizeof(u));
        } else {
            const int64_t at = n >= kChunk ? k : FORM == kTail && n > 0 ? k + n - kChunk : 0;
            __builtin_memcpy(u, p + at, sizeof(u));
        }
        if constexpr (FORM == kWhole) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) u[j] = n > 0 ? u[j] : 0u;
        }
    }
    // The same for the norm, with a test around the load of a thread without a
    // chunk: nothing in the branch waits, and the weights' zeros need no select
    // that would wait for them before the row's loads are issued (2048 x 4096
    // bf16: 13.0 us, 14.1 with load(); the gated product of 8192 x 8192 prefers
    // load(): 64 us, 69 with this).
    template <int FORM>
    __device__ __forceinline__ void load_if(const T* p, int64_t k, int n) {
        if constexpr (FORM == kWhole) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) u[j] = 0u;
            if (n > 0) __builtin_memcpy(u, p + k, sizeof(u));
        } else {
            load<FORM>(p, k, n);
        }
    }
    // What load() read beside a partial chunk's n elements goes, zeros take its place.
    template <int FORM>
    __device__ __forceinline__ void settle(int n) {
        if constexpr (FORM == kTail) {
            if (n >= kChunk) return;
            const int s = n > 0 ? kChunk - n : kChunk;         // elements to drop
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    u[j] = s & 1 ? __builtin_amdgcn_alignbyte(j + 1 < kWords ? u[j + 1] : 0u, u[j], 2u) : u[j];
            }
#pragma unroll
            for (int by = 1; by <= kWords; by *= 2) {
                const bool drop = s & (by * 4 / static_cast<int>(sizeof(T)));
#pragma unroll
                for (int j = 0; j < kWords; ++j) u[j] = drop ? (j + by < kWords ? u[j + by] : 0u) : u[j];
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[kChunk]) const {
        T t[kChunk];
        __builtin_memcpy(t, u, sizeof(u));
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = to_f(t[j]);
    }
};

// The first n (1 .. 7) of eight elements of SIZE bytes, in three pieces at
// most: one branch each for 4, 2 and 1 elements, the rest moved down.
template <int SIZE>
__device__ __forceinline__ void store_some(uint8_t* p, int n, const uint32_t (&u)[2 * SIZE]) {
    uint32_t left[SIZE];
#pragma unroll
    for (int j = 0; j < SIZE; ++j) left[j] = u[j];
    if (n & 4) {
        __builtin_memcpy(p, left, 4 * SIZE);
#pragma unroll
        for (int j = 0; j < SIZE; ++j) left[j] = u[SIZE + j];
    }
    p += (n & 4) * SIZE;
    if (n & 2) {
        __builtin_memcpy(p, left, 2 * SIZE);
        if constexpr (SIZE == 1) left[0] >>= 16;
        else if constexpr (SIZE == 2) left[0] = left[1];
        else left[0] = left[2];
    }
    if (n & 1) __builtin_memcpy(p + (n & 2) * SIZE, left, SIZE);
}

template <int FORM, class T>
__device__ __forceinline__ void store_chunk(T* p, int n, const float (&v)[kChunk]) {
    if (FORM == kWhole ? n > 0 : n >= kChunk) {
        T t[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) t[j] = static_cast<T>(v[j]);
        __builtin_memcpy(p, t, sizeof(t));
    } else if (FORM != kWhole && n > 0) {
        T t[kChunk];
        uint32_t u[2 * sizeof(T)];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) t[j] = static_cast<T>(v[j]);
        __builtin_memcpy(u, t, sizeof(t));
        store_some<sizeof(T)>(reinterpret_cast<uint8_t*>(p), n, u);
    }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ float as_float(uint32_t b) { return __builtin_bit_cast(float, b); }

// ---- sources: p of one element in fp64 ----

template <class T>
struct PlainSrc {
    static constexpr float kDelta = 0x1p-22f;      // roundings of R / P, of each factor, of the product: 3 * 2^-24
    const T* x;
    __device__ __forceinline__ double exact(int64_t k) const { return static_cast<double>(to_f(x[k])); }
};

template <class T>
struct NormSrc {
    static constexpr float kDelta = 0x1p-21f;      // as above, and the rounding of h * w: 4 * 2^-24
    const T* h;              // the row that is normalised: x, or the stored sum
    const float* w;
    __device__ __forceinline__ double exact(int64_t k) const {
        return static_cast<double>(to_f(h[k])) * static_cast<double>(w[k]);
    }
};

__device__ __forceinline__ double silu_mul_exact(float a, float b) {
    const double d = a;
    return d / (1.0 + exp(-d)) * static_cast<double>(b);
}

// fp32 silu(a) * b = ab / (1 + exp(-a)); ab is returned too. exp(-a) = 2^hi *
// (1 + lo ln 2) with hi + lo = -a log2 e to about 2^-44, so its relative error
// is that of v_exp_f32 and two roundings at every a (a single fp32 product
// would lose |a| * 2^-24). exp stays finite because a is taken as -80 below
// that: the result is then too large, by less than |ab| * 2^-115 (exp(-80) <
// 2^-115), which the callers look at. a * b first: it overflows where a
// factor is huge (the callers see infinity), and where it underflows the
// result does.
__device__ __forceinline__ float silu_mul_fast(float a, float b, float& ab) {
    constexpr float kL = -0x1.715476p+0f, kLlo = -0x1.4ae0cp-26f;      // -log2 e, high and low part
    const float c = __builtin_fmaxf(a, -80.0f);
    const float hi = c * kL;
    const float lo = __builtin_fmaf(c, kLlo, __builtin_fmaf(c, kL, -hi));
    const float e0 = __builtin_amdgcn_exp2f(hi);
    const float e = __builtin_fmaf(e0, lo * 0x1.62e43p-1f, e0);
    ab = a * b;
    return ab * __builtin_amdgcn_rcpf(1.0f + e);
}

template <class T>
struct SiluSrc {
    // v_exp_f32 and v_rcp_f32 (1 ulp each) and four roundings in p, three as the quantizer's: 11 * 2^-24
    static constexpr float kDelta = 0x1p-20f;
    const T* a;
    const T* b;
    __device__ __forceinline__ double exact(int64_t k) const { return silu_mul_exact(to_f(a[k]), to_f(b[k])); }
};

// ---- rounding to codes ----

// fp64 -> fp32 rounded to odd: a later rounding to fewer bits is then that of
// the fp64 value itself.
__device__ __forceinline__ float round_to_odd(double t) {
    const float f = static_cast<float>(t);
    const double back = f;
    uint32_t b = __builtin_bit_cast(uint32_t, f);
    if (back != t) {
        if (__builtin_fabs(back) > __builtin_fabs(t)) --b;
        b |= 1u;
    }
    return __builtin_bit_cast(float, b);
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xffffu;
}

template <int OUT>
struct CodeOf {
    static constexpr float kTop = OUT == kOutQ8 ? 127.0f : 448.0f;
    // The code of the fp64 quotient R * p / P, first rounded to 47 bits. Rows
    // hold true ties (elements with the gate of the row's largest, b / b_max =
    // 9 / 16, or weights of one value); the roundings of p, P, R * p and the
    // quotient, 2^-53 each, would send those either way. 47 bits bring each
    // back to the tie, and move no other quotient by more than 2^-48 of it.
    static __device__ __forceinline__ uint32_t exact(double p, double P) {
        const uint64_t bits = __builtin_bit_cast(uint64_t, static_cast<double>(kTop) * p / P);
        const double t = __builtin_bit_cast(double, (bits + 32u) & ~uint64_t{63});
        if constexpr (OUT == kOutQ8) return static_cast<uint32_t>(static_cast<int>(__builtin_rint(t))) & 0xffu;
        else return e4m3_pair(round_to_odd(t), 0.0f) & 0xffu;
    }
};

// Codes of eight fp32 values v with factors lo < R / P < hi, packed. `differ`:
// nonzero bytes where the two factors give different codes.
template <int OUT>
__device__ __forceinline__ u32x2 fast_codes(const float (&v)[kChunk], float lo, float hi, u32x2& differ) {
    u32x2 w, d;
    if constexpr (OUT == kOutQ8) {
        // v * f + 1.5 * 2^23 rounds once, to a whole number, ties to even; its low byte is the code
        constexpr float kMagic = 12582912.0f;
        auto pack = [&](int j, float f) {
            uint32_t r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = __builtin_bit_cast(uint32_t, __builtin_fmaf(v[j + e], f, kMagic));
            const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x0c0c0400u);
            const uint32_t b = __builtin_amdgcn_perm(r[3], r[2], 0x04000c0cu);
            return a | b;
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = pack(4 * h, hi);
            d[h] = w[h] ^ pack(4 * h, lo);
        }
    } else {
        auto pack = [&](int j, float f) {
            int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[j] * f, v[j + 1] * f, 0, false);
            r = __builtin_amdgcn_cvt_pk_fp8_f32(v[j + 2] * f, v[j + 3] * f, r, true);
            return static_cast<uint32_t>(r);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = pack(4 * h, hi);
            d[h] = w[h] ^ pack(4 * h, lo);
        }
    }
    differ = d;
    return w;
}

// Bit j: byte j is not zero.
__device__ __forceinline__ uint32_t bytes_set(u32x2 d) {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) mask |= (d[j / 4] >> (8 * (j % 4))) & 0xffu ? 1u << j : 0u;
    return mask;
}

template <int FORM>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 w) {
    if (n >= kChunk) {
        __builtin_memcpy(p, &w, 8);
    } else if (FORM != kWhole && n > 0) {
        const uint32_t u[2] = {w[0], w[1]};
        store_some<1>(p, n, u);
    }
}

// ---- reductions over a wave (DPP: no LDS crossbar), result in every lane ----

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false));
}

// f(v, CTRL) over row_shr 1, 2, 4, 8, row_bcast 15 and 31: lane 63 ends with
// the whole wave's. Lanes without a source read 0.
template <class V, class F>
__device__ __forceinline__ V wave_scan(V v, F f) {
    v = f(v, std::integral_constant<int, 0x111>());
    v = f(v, std::integral_constant<int, 0x112>());
    v = f(v, std::integral_constant<int, 0x114>());
    v = f(v, std::integral_constant<int, 0x118>());
    v = f(v, std::integral_constant<int, 0x142>());
    return f(v, std::integral_constant<int, 0x143>());
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = wave_scan(v, [](uint32_t a, auto c) {
        const uint32_t b = dpp<decltype(c)::value>(a);
        return a > b ? a : b;
    });
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) {
    v = wave_scan(v, [](double a, auto c) {
        const uint64_t b = __builtin_bit_cast(uint64_t, a);
        const uint64_t o = static_cast<uint64_t>(dpp<decltype(c)::value>(static_cast<uint32_t>(b >> 32))) << 32 |
                           dpp<decltype(c)::value>(static_cast<uint32_t>(b));
        return a + __builtin_bit_cast(double, o);
    });
    return lane_value(v, 63);
}

// The largest of a value that few lanes hold (zero in the others).
__device__ __forceinline__ double wave_max_sparse(double v) {
    double best = 0.0;
    uint64_t lanes = __builtin_amdgcn_ballot_w64(v > 0.0);
    while (lanes) {
        best = __builtin_fmax(best, lane_value(v, __builtin_ctzll(lanes)));
        lanes &= lanes - 1;
    }
    return best;
}

struct RowArgs {
    const void* x;           // x, or a
    const void* r;           // residual or nullptr, or b
    void* sum;
    const float* weight;
    void* out;
    float* scale;
    int64_t ldx, ldr, lds;
    int64_t M, K;
    float eps;
};

// Sources of rows. load(): a chunk of the inputs; values(): what is kept of it
// in fp32: x, or h (the norm, which stores it), or p (the gated product;
// `top_ab` collects max |ab|).
template <class T>
struct PlainOp {
    typedef PlainSrc<T> Src;
    static constexpr bool kNorm = false, kSilu = false;
    Raw<T> x;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return Src{static_cast<const T*>(a.x) + row * a.ldx};
    }
    template <int FORM>
    __device__ __forceinline__ void load(const RowArgs& a, int64_t row, int64_t k, int n) {
        x.template load<FORM>(static_cast<const T*>(a.x) + row * a.ldx, k, n);
    }
    template <int FORM>
    __device__ __forceinline__ void values(const RowArgs&, int64_t, int64_t, int n, float (&p)[kChunk], uint32_t&) {
        x.template settle<FORM>(n);
        x.get(p);
    }
};

template <class T>
struct NormOp {
    typedef NormSrc<T> Src;
    static constexpr bool kNorm = true, kSilu = false;
    Raw<T> x, r;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return a.r ? Src{static_cast<const T*>(a.sum) + row * a.lds, a.weight}
                   : Src{static_cast<const T*>(a.x) + row * a.ldx, a.weight};
    }
    template <int FORM>
    __device__ __forceinline__ void load(const RowArgs& a, int64_t row, int64_t k, int n) {
        x.template load_if<FORM>(static_cast<const T*>(a.x) + row * a.ldx, k, n);
        if (a.r) r.template load_if<FORM>(static_cast<const T*>(a.r) + row * a.ldr, k, n);
    }
    // h = x + residual in fp32, rounded once to the stream's type: what is
    // stored is what is normalised.
    template <int FORM>
    __device__ __forceinline__ void values(const RowArgs& a, int64_t row, int64_t k, int n, float (&h)[kChunk], uint32_t&) {
        x.template settle<FORM>(n);
        x.get(h);
        if (a.r) {
            float b[kChunk];
            r.template settle<FORM>(n);
            r.get(b);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) h[j] = to_f(static_cast<T>(h[j] + b[j]));
            store_chunk<FORM>(static_cast<T*>(a.sum) + row * a.lds + k, n, h);
        }
    }
};

template <class T>
struct SiluOp {
    typedef SiluSrc<T> Src;
    static constexpr bool kNorm = false, kSilu = true;
    Raw<T> x, r;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return Src{static_cast<const T*>(a.x) + row * a.ldx, static_cast<const T*>(a.r) + row * a.ldr};
    }
    template <int FORM>
    __device__ __forceinline__ void load(const RowArgs& a, int64_t row, int64_t k, int n) {
        x.template load<FORM>(static_cast<const T*>(a.x) + row * a.ldx, k, n);
        r.template load<FORM>(static_cast<const T*>(a.r) + row * a.ldr, k, n);
    }
    template <int FORM>
    __device__ __forceinline__ void values(const RowArgs&, int64_t, int64_t, int n, float (&p)[kChunk], uint32_t& top_ab) {
        float b[kChunk];
        x.template settle<FORM>(n);
        r.template settle<FORM>(n);
        x.get(p);
        r.get(b);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            float ab;
            p[j] = silu_mul_fast(p[j], b[j], ab);
            top_ab = max(top_ab, abs_bits(ab));
        }
    }
    // Dense rows have no maximum to hide behind: gates below -80 and products
    // that overflow before the sigmoid are taken in fp64.
    template <int FORM>
    __device__ __forceinline__ void dense(const RowArgs& a, int64_t row, int64_t k, int n, float (&p)[kChunk]) {
        float b[kChunk];
        uint32_t mask = 0;
        x.template settle<FORM>(n);
        r.template settle<FORM>(n);
        x.get(p);
        r.get(b);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            float ab;
            const bool low = p[j] < -80.0f;
            p[j] = silu_mul_fast(p[j], b[j], ab);
            mask |= low || __builtin_fabsf(ab) > FLT_MAX ? 1u << j : 0u;
        }
        mask &= n >= kChunk ? 0xffu : (1u << max(n, 0)) - 1u;
        const Src s = src(a, row);
        while (mask) {
            const int h = __builtin_ctz(mask);
            mask &= mask - 1u;
            const float v = static_cast<float>(s.exact(k + h));
#pragma unroll
            for (int j = 0; j < kChunk; ++j) p[j] = j == h ? v : p[j];
        }
    }
};

// One row per TPR threads (64: four rows per workgroup of 256; else one), NV
// chunks of eight elements per thread held in registers: one pass over the
// data. NV = 0: rows of any length, read again for each step. Workgroups take
// rows in turn; the norm's weight stays in registers across them.
//
// Bound by memory: long inputs move at 4.5 to 5.7 TB/s, a copy of 1 GiB at 5.1
// (bf16 quantizer, 16384 x 8192: 70.0 us, 5.7 TB/s; bf16 norm with its sum,
// 2048 x 4096: 13.0 us, 4.5 TB/s; bf16 gated product, 8192 x 8192: 63.8 us, 5.3
// TB/s). One row of 512 takes 2.3 us: one load, two reductions, one store.
//
// Rows whose K is no multiple of eight cost the moves of one partial chunk and
// unaligned accesses (bf16, M K = 2^25, K = 4096 / 4095: quantizer 21.1 / 25.5
// us, gated product 34.9 / 47.2, norm to codes 55.6 / 70.7; with a test for
// every element of every chunk instead 31.8, 74.4 and 149.0).
template <class Op, int OUT, class OutT, int TPR, int NV, int FORM>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void row_kernel(RowArgs a) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    constexpr bool kNorm = Op::kNorm, kDense = OUT == kOutDense;
    constexpr bool kReduced = kNorm || !kDense;                // whether a row is reduced at all
    constexpr int W = TPR / 64;
    // By the row's parity: a row's slots are written again two rows later,
    // behind the barrier of the row between.
    __shared__ double sh_ss[2][W], sh_best[2][W];
    __shared__ uint32_t sh_top[2][W], sh_ab[2][W];
    const int lane = TPR == 64 ? static_cast<int>(threadIdx.x & 63) : static_cast<int>(threadIdx.x);
    const int wave = threadIdx.x >> 6;
    const int per = NV > 0 ? NV : static_cast<int>((a.K + kChunk * TPR - 1) / (kChunk * TPR));
    auto chunk_k = [&](int i) { return static_cast<int64_t>(i * TPR + lane) * kChunk; };
    auto chunk_n = [&](int64_t k) {                                                       // <= 0: none
        if constexpr (FORM == kWhole) return k < a.K ? kChunk : 0;
        else return static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk);
    };

    float w[kNorm && NV > 0 ? NV : 1][kChunk];
    if constexpr (kNorm && NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Raw<float> g;
            g.load_if<FORM>(a.weight, chunk_k(i), chunk_n(chunk_k(i)));
            g.settle<FORM>(chunk_n(chunk_k(i)));
            g.get(w[i]);
        }
    }

    int parity = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + (TPR == 64 ? wave : 0); row < a.M;
         row += static_cast<int64_t>(gridDim.x) * RPB, parity ^= 1) {
        const typename Op::Src src = Op::src(a, row);
        float v[NV > 0 ? NV : 1][kChunk];
        uint32_t top = 0, top_ab = 0;
        double ss = 0.0;

        auto values = [&](Op& op, int i, float (&x)[kChunk]) {
            const int64_t k = chunk_k(i);
            if constexpr (Op::kSilu && kDense) op.template dense<FORM>(a, row, k, chunk_n(k), x);
            else op.template values<FORM>(a, row, k, chunk_n(k), x, top_ab);
        };
        auto take = [&](int i, float (&x)[kChunk]) {
            Op op;
            op.template load<FORM>(a, row, chunk_k(i), chunk_n(chunk_k(i)));
            values(op, i, x);
        };
        auto weight = [&](int i) {
            Raw<float> g;
            g.load_if<FORM>(a.weight, chunk_k(i), chunk_n(chunk_k(i)));
            g.settle<FORM>(chunk_n(chunk_k(i)));
            g.get(w[0]);
        };
        // The same values once more, of a row that values() has been through.
        auto again = [&](int i, float (&x)[kChunk]) {
            if constexpr (kNorm) {
                Raw<std::remove_const_t<std::remove_pointer_t<decltype(src.h)>>> h;
                h.template load_if<FORM>(src.h, chunk_k(i), chunk_n(chunk_k(i)));
                h.template settle<FORM>(chunk_n(chunk_k(i)));
                h.get(x);
                weight(i);
            } else {
                take(i, x);
            }
        };
        auto look = [&](const float (&x)[kChunk], const float (&wx)[kChunk]) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                if constexpr (kNorm) {
                    const double h = x[j];
                    ss = __builtin_fma(h, h, ss);
                }
                if constexpr (!kDense) top = max(top, abs_bits(kNorm ? x[j] * wx[j] : x[j]));
            }
        };
        if constexpr (NV > 0) {
            Op op[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) op[i].template load<FORM>(a, row, chunk_k(i), chunk_n(chunk_k(i)));
#pragma unroll
            for (int i = 0; i < NV; ++i) values(op[i], i, v[i]);
            if constexpr (kReduced) {
#pragma unroll
                for (int i = 0; i < NV; ++i) look(v[i], w[kNorm ? i : 0]);
            }
        } else if constexpr (kReduced) {
            for (int i = 0; i < per; ++i) {
                take(i, v[0]);
                if constexpr (kNorm) weight(i);
                look(v[0], w[0]);
            }
        }
        const uint32_t lane_top = top;
        if constexpr (kReduced) {
            if constexpr (kNorm) ss = wave_sum(ss);
            if constexpr (!kDense) top = wave_max(top);
            if constexpr (Op::kSilu) top_ab = wave_max(top_ab);
            if constexpr (TPR > 64) {
                if ((threadIdx.x & 63) == 0) {
                    if constexpr (kNorm) sh_ss[parity][wave] = ss;
                    sh_top[parity][wave] = top;
                    if constexpr (Op::kSilu) sh_ab[parity][wave] = top_ab;
                }
                __syncthreads();
                ss = 0.0;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if constexpr (kNorm) ss += sh_ss[parity][i];
                    top = max(top, sh_top[parity][i]);
                    if constexpr (Op::kSilu) top_ab = max(top_ab, sh_ab[parity][i]);
                }
            }
        }
        double r = 1.0;
        if constexpr (kNorm) r = 1.0 / __builtin_sqrt(ss / static_cast<double>(a.K) + static_cast<double>(a.eps));

        if constexpr (kDense) {
            OutT* out = static_cast<OutT*>(a.out) + row * a.K;
            const float rf = static_cast<float>(r);
            auto put = [&](int i, float (&x)[kChunk], const float (&wx)[kChunk]) {
                const int64_t k = chunk_k(i);
                const int n = chunk_n(k);
                if (n <= 0) return;
                if constexpr (kNorm) {
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) x[j] = x[j] * rf * wx[j];
                }
                store_chunk<FORM>(out + k, n, x);
            };
            if constexpr (NV > 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) put(i, v[i], w[kNorm ? i : 0]);
            } else {
                for (int i = 0; i < per; ++i) {
                    again(i, v[0]);
                    put(i, v[0], w[0]);
                }
            }
        } else {
            typedef CodeOf<OUT> Code;
            constexpr float kDelta = Op::Src::kDelta;
            const float pf = as_float(top);
            bool fast = pf >= 0x1p-60f && pf <= 0x1p120f;            // false for NaN
            // the gates below -80: their error stays under 2^-40 of P
            if constexpr (Op::kSilu) fast = fast && as_float(top_ab) <= pf * 0x1p75f;
            double P = static_cast<double>(pf);
            if (kNorm || Op::kSilu || !fast) {
                const float near = pf * (1.0f - 2.0f * kDelta);
                double best = 0.0;
                if (!fast) {
                    for (int i = 0; i < per; ++i) {
                        const int64_t k = chunk_k(i);
                        const int n = chunk_n(k);
                        for (int j = 0; j < n; ++j) {
                            const double p = __builtin_fabs(src.exact(k + j));
                            best = __builtin_fmax(best, p <= DBL_MAX ? p : static_cast<double>(__builtin_inff()));
                        }
                    }
                } else if (as_float(lane_top) >= near) {
                    auto candidates = [&](const float (&x)[kChunk], const float (&wx)[kChunk]) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int j = 0; j < kChunk; ++j)
                            mask |= __builtin_fabsf(kNorm ? x[j] * wx[j] : x[j]) >= near ? 1u << j : 0u;
                        return mask;
                    };
                    auto settle = [&](int i0, uint32_t mask) {
                        while (mask) {
                            const int b = __builtin_ctz(mask);
                            mask &= mask - 1u;
                            best = __builtin_fmax(best, __builtin_fabs(src.exact(chunk_k(i0 + b / kChunk) + b % kChunk)));
                        }
                    };
                    if constexpr (NV > 0) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int i = 0; i < NV; ++i) mask |= candidates(v[i], w[kNorm ? i : 0]) << (kChunk * i);
                        settle(0, mask);
                    } else {
                        for (int i = 0; i < per; ++i) {
                            again(i, v[0]);
                            settle(i, candidates(v[0], w[0]));
                        }
                    }
                }
                P = wave_max_sparse(best);
                if constexpr (TPR > 64) {
                    if ((threadIdx.x & 63) == 0) sh_best[parity][wave] = P;
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < W; ++i) P = __builtin_fmax(P, sh_best[parity][i]);
                }
            }
            const float scale = static_cast<float>(P * r / static_cast<double>(Code::kTop));
            const bool fine = scale <= FLT_MAX;                      // false for NaN and infinity
            if (lane == 0) a.scale[row] = fine ? scale : __builtin_nanf("");
            uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.K;
            const bool zero = !fine || P == 0.0, quick = fast && fine;
            const float inv = static_cast<float>(static_cast<double>(Code::kTop) / P);
            const float lo = inv * (1.0f - kDelta), hi = inv * (1.0f + kDelta);
            // Stores the codes of chunk i; returns the elements still to be taken in fp64.
            auto put = [&](int i, const float (&x)[kChunk], const float (&wx)[kChunk]) {
                const int64_t k = chunk_k(i);
                const int n = chunk_n(k);
                if (n <= 0) return 0u;
                u32x2 c = {0u, 0u};
                uint32_t mask = zero ? 0u : 0xffu;
                if (quick) {
                    float p[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) p[j] = kNorm ? x[j] * wx[j] : x[j];
                    u32x2 d;
                    c = fast_codes<OUT>(p, lo, hi, d);
                    mask = d[0] | d[1] ? bytes_set(d) : 0u;
                }
                store_codes<FORM>(out + k, n, c);
                return n >= kChunk ? mask : mask & ((1u << n) - 1u);
            };
            // The same thread stored these elements' chunk, so the bytes land in this order.
            auto settle = [&](int i0, uint32_t mask) {
                while (mask) {
                    const int b = __builtin_ctz(mask);
                    mask &= mask - 1u;
                    const int64_t k = chunk_k(i0 + b / kChunk) + b % kChunk;
                    out[k] = static_cast<uint8_t>(Code::exact(src.exact(k), P));
                }
            };
            if constexpr (NV > 0) {
                uint32_t mask = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) mask |= put(i, v[i], w[kNorm ? i : 0]) << (kChunk * i);
                settle(0, mask);
            } else {
                for (int i = 0; i < per; ++i) {
                    again(i, v[0]);
                    settle(i, put(i, v[0], w[0]));
                }
            }
        }
    }
}

constexpr int64_t kMaxGrid = 1 << 20;

template <class Op, int OUT, class OutT, int TPR, int NV, int FORM>
hipError_t launch_rows(const RowArgs& a, hipStream_t stream) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    const int64_t blocks = (a.M + RPB - 1) / RPB;
    row_kernel<Op, OUT, OutT, TPR, NV, FORM><<<static_cast<uint32_t>(blocks < kMaxGrid ? blocks : kMaxGrid),
                                                TPR == 64 ? 256 : TPR, 0, stream>>>(a);
    return hipGetLastError();
}

// Threads and chunks per row by its length alone. Measured on bf16 rows, us,
// norm / quantizer / gated product: K = 1024, M = 16384: 64 threads x 2 chunks
// 26.8 / 10.3 / 19.9, 128 x 1 31.4 / 12.1 / 23.1. K = 2048, M = 8192: 128 x 2
// 26.4 / 10.5 / 20.0, 256 x 1 29.1 / 11.7 / 21.5, 64 x 4 26.3 / 10.2 / 20.4
// (fp32 norm 43.4, 42.2, 49.7). K = 4096: 256 x 2 14.0 (norm, M = 2048), 128 x
// 4 15.5. K = 8192: 256 x 4 71.5 (quantizer, M = 16384) and 69.9 (gated
// product, M = 8192), 512 x 2 71.8 and 83.7. K = 16384, M = 1024: 512 x 4 32.0
// / 11.1 / 21.3, 1024 x 2 32.9 / 11.4 / 24.7, 256 x 8 40.9 / 11.4 / 23.6.
template <class Op, int OUT, class OutT, int FORM>
hipError_t launch_by_length(const RowArgs& a, hipStream_t stream) {
    if (a.K <= 64 * 8) return launch_rows<Op, OUT, OutT, 64, 1, FORM>(a, stream);
    if (a.K <= 64 * 16) return launch_rows<Op, OUT, OutT, 64, 2, FORM>(a, stream);
    if (a.K <= 128 * 16) return launch_rows<Op, OUT, OutT, 128, 2, FORM>(a, stream);
    if (a.K <= 256 * 16) return launch_rows<Op, OUT, OutT, 256, 2, FORM>(a, stream);
    if (a.K <= 256 * 32) return launch_rows<Op, OUT, OutT, 256, 4, FORM>(a, stream);
    if (a.K <= 512 * 32) return launch_rows<Op, OUT, OutT, 512, 4, FORM>(a, stream);
    return launch_rows<Op, OUT, OutT, 1024, 0, FORM>(a, stream);
}

template <class Op, int OUT, class OutT>
hipError_t launch_by_form(const RowArgs& a, hipStream_t stream) {
    if (a.K % kChunk == 0) return launch_by_length<Op, OUT, OutT, kWhole>(a, stream);
    if (a.K > kChunk) return launch_by_length<Op, OUT, OutT, kTail>(a, stream);
    return launch_rows<Op, OUT, OutT, 64, 1, kShort>(a, stream);
}

template <template <class> class Op, class T>
hipError_t launch_by_out(const RowArgs& a, int fmt, int out_dtype, hipStream_t stream) {
    if (fmt == RTQ_FMT_Q8) return launch_by_form<Op<T>, kOutQ8, uint8_t>(a, stream);
    if (fmt == RTQ_FMT_F8) return launch_by_form<Op<T>, kOutF8, uint8_t>(a, stream);
    if constexpr (!__is_same(Op<T>, PlainOp<T>)) {
        if (out_dtype == RTQ_F32) return launch_by_form<Op<T>, kOutDense, float>(a, stream);
        return launch_by_form<Op<T>, kOutDense, T>(a, stream);
    }
    return hipErrorInvalidValue;
}

template <template <class> class Op>
hipError_t launch_by_dtype(const RowArgs& a, int dtype, int fmt, int out_dtype, hipStream_t stream) {
    switch (dtype) {
        case RTQ_F32: return launch_by_out<Op, float>(a, fmt, out_dtype, stream);
        case RTQ_F16: return launch_by_out<Op, _Float16>(a, fmt, out_dtype, stream);
        default: return launch_by_out<Op, __bf16>(a, fmt, out_dtype, stream);
    }
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int64_t ldx, int dtype, int fmt, void* codes, float* scale, int64_t M,
                                int64_t K, hipStream_t stream) {
    const RowArgs a{x, nullptr, nullptr, nullptr, codes, scale, ldx, 0, 0, M, K, 0.0f};
    return launch_by_dtype<PlainOp>(a, dtype, fmt, 0, stream);
}

hipError_t launch_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* sum, int64_t lds,
                           const float* weight, float eps, int dtype, int fmt, int out_dtype, void* out, float* scale,
                           int64_t M, int64_t K, hipStream_t stream) {
    const RowArgs a{x, residual, sum, weight, out, scale, ldx, ldr, lds, M, K, eps};
    return launch_by_dtype<NormOp>(a, dtype, fmt, out_dtype, stream);
}

hipError_t launch_silu_mul(const void* x, int64_t lda, const void* b, int64_t ldb, int dtype, int fmt, int out_dtype,
                           void* out, float* scale, int64_t M, int64_t K, hipStream_t stream) {
    const RowArgs a{x, b, nullptr, nullptr, out, scale, lda, ldb, 0, M, K, 0.0f};
    return launch_by_dtype<SiluOp>(a, dtype, fmt, out_dtype, stream);
}

}  // namespace rtq
