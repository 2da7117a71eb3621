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
// The codes are those of the fp64 formula, as the weight quantizers' are. Two
// steps make that cheap:
//  - t = R * p / P is first taken in fp32, whose relative error is below
//    Src::kDelta. Only where t lies that close to a rounding border (about one
//    element in 10^4) is the element's p loaded again and the quotient taken
//    in fp64.
//  - P itself: exact in fp32 for the quantizer; kept in fp64 for the norm (the
//    multiply and the maximum run beside the sum of squares); for the gated
//    product the row's candidates, those within 2 * kDelta of the fp32
//    maximum, are evaluated again in fp64.
// Rows whose P lies outside [2^-60, 2^120], where fp32 products could lose
// bits to underflow or overflow, and rows with an infinity or a NaN, take
// every step in fp64.
//
// Sums of squares are fp64: no overflow for any finite fp32 row.
#include <rtq.h>

#include <float.h>

#include "rtq_internal.h"

namespace rtq {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 8;                  // consecutive elements of one lane's load
constexpr int kOutQ8 = 0, kOutF8 = 1, kOutDense = 2;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(_Float16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float to_f(__bf16 v) { return static_cast<float>(v); }

// Loads and stores of a whole chunk go through memcpy: one 16-byte access per
// 16 bytes at any alignment of the row.
template <class T>
__device__ __forceinline__ void load_chunk(const T* p, int n, float (&v)[kChunk]) {
    if (n >= kChunk) {
        T t[kChunk];
        __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = to_f(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = j < n ? to_f(p[j]) : 0.0f;
    }
}

template <class T>
__device__ __forceinline__ void store_chunk(T* p, int n, const float (&v)[kChunk]) {
    if (n >= kChunk) {
        T t[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) t[j] = static_cast<T>(v[j]);
        __builtin_memcpy(p, t, sizeof(t));
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (j < n) p[j] = static_cast<T>(v[j]);
    }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ float as_float(uint32_t b) { return __builtin_bit_cast(float, b); }

// ---- sources: fast(k) in fp32, exact(k) in fp64, of one row ----

template <class T>
struct PlainSrc {
    static constexpr bool kNorm = false, kCandidates = false;
    // t carries the rounding of R / P and of the product
    static constexpr float kDelta = 0x1p-21f;
    const T* x;
    __device__ __forceinline__ double exact(int64_t k) const { return static_cast<double>(to_f(x[k])); }
};

template <class T>
struct NormSrc {
    static constexpr bool kNorm = true, kCandidates = false;
    // the rounding of h * w, of R / P and of the product
    static constexpr float kDelta = 0x1p-21f;
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

// fp32 silu(a) * b. exp(-a) = 2^hi * (1 + lo ln 2) with hi + lo = -a log2 e to
// about 2^-44, so its relative error is that of v_exp_f32 and two roundings
// at every a (a single fp32 product would lose |a| * 2^-24). `hard` is set
// where fp32 cannot hold a factor to full precision (exp overflows, or the
// sigmoid's product is tiny): that element is taken in fp64.
__device__ __forceinline__ float silu_mul_fast(float a, float b, bool& hard) {
    constexpr float kL = -0x1.715476p+0f, kLlo = -0x1.4ae0cp-26f;      // -log2 e, high and low part
    const float hi = a * kL;
    const float lo = __builtin_fmaf(a, kLlo, __builtin_fmaf(a, kL, -hi));
    const float e0 = __builtin_amdgcn_exp2f(hi);
    const float e = __builtin_fmaf(e0, lo * 0x1.62e43p-1f, e0);
    const float u = a * __builtin_amdgcn_rcpf(1.0f + e);
    hard = a < -80.0f || (__builtin_fabsf(u) < 0x1p-100f && a != 0.0f);
    return u * b;
}

template <class T>
struct SiluSrc {
    static constexpr bool kNorm = false, kCandidates = true;
    // v_exp_f32 and v_rcp_f32 (1 ulp each) and six more roundings, twice (in p and in P)
    static constexpr float kDelta = 0x1p-18f;
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
    // The code of the fp64 quotient R * p / P.
    static __device__ __forceinline__ uint32_t exact(double p, double P) {
        const double t = static_cast<double>(kTop) * p / P;
        if constexpr (OUT == kOutQ8) return static_cast<uint32_t>(static_cast<int>(__builtin_rint(t))) & 0xffu;
        else return e4m3_pair(round_to_odd(t), 0.0f) & 0xffu;
    }
};

// Codes of eight fp32 values v with factor inv = R / P, packed; bit j of the
// result's mask: element j is within `delta` of a rounding border.
template <int OUT>
__device__ __forceinline__ u32x2 fast_codes(const float (&v)[kChunk], float inv, float delta, uint32_t& mask) {
    u32x2 w = {0u, 0u};
    mask = 0;
    if constexpr (OUT == kOutQ8) {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float t = v[j] * inv;
            const float n = __builtin_rintf(t);
            const float d = __builtin_fabsf(t - n);
            if (d > __builtin_fmaf(-delta, __builtin_fabsf(t), 0.5f)) mask |= 1u << j;
            w[j / 4] |= (static_cast<uint32_t>(static_cast<int>(n)) & 0xffu) << (8 * (j % 4));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; j += 2) {
            const float t0 = v[j] * inv, t1 = v[j + 1] * inv;
            const uint32_t lo = e4m3_pair(t0 * (1.0f - delta), t1 * (1.0f - delta));
            const uint32_t hi = e4m3_pair(t0 * (1.0f + delta), t1 * (1.0f + delta));
            const uint32_t x = lo ^ hi;
            if (x & 0xffu) mask |= 1u << j;
            if (x & 0xff00u) mask |= 2u << j;
            w[j / 4] |= hi << (8 * (j % 4));
        }
    }
    return w;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 w) {
    if (n >= kChunk) {
        __builtin_memcpy(p, &w, 8);
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (j < n) p[j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
    }
}

// ---- reductions over the TPR threads of a row ----

template <class V, class F>
__device__ __forceinline__ V wave_reduce(V v, F f) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = f(v, __shfl_xor(v, s));
    return v;
}

// All threads of the row get the result. `slot` is LDS of TPR / 64 entries of
// its own for each use within a row.
template <int TPR, class V, class F>
__device__ __forceinline__ V row_reduce(V v, V* slot, F f) {
    v = wave_reduce(v, f);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = f(v, slot[i]);
    }
    return v;
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

struct Max32 {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct Max64 {
    __device__ __forceinline__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
};
struct Add64 {
    __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};

template <class T>
struct PlainOp {
    typedef PlainSrc<T> Src;
    typedef T In;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return Src{static_cast<const T*>(a.x) + row * a.ldx};
    }
    // The chunk's p in fp32 (zeros past n) and, for the norm, h itself.
    static __device__ __forceinline__ void first(const RowArgs& a, int64_t row, int64_t k, int n, float (&p)[kChunk],
                                                 float (&)[kChunk]) {
        load_chunk(static_cast<const T*>(a.x) + row * a.ldx + k, n, p);
    }
};

template <class T>
struct NormOp {
    typedef NormSrc<T> Src;
    typedef T In;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return a.r ? Src{static_cast<const T*>(a.sum) + row * a.lds, a.weight}
                   : Src{static_cast<const T*>(a.x) + row * a.ldx, a.weight};
    }
    // h = x + residual in fp32, rounded once to the stream's type: what is
    // stored is what is normalised.
    static __device__ __forceinline__ void first(const RowArgs& a, int64_t row, int64_t k, int n, float (&h)[kChunk],
                                                 float (&w)[kChunk]) {
        load_chunk(static_cast<const T*>(a.x) + row * a.ldx + k, n, h);
        load_chunk(a.weight + k, n, w);
        if (a.r) {
            float r[kChunk];
            load_chunk(static_cast<const T*>(a.r) + row * a.ldr + k, n, r);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) h[j] = to_f(static_cast<T>(h[j] + r[j]));
            store_chunk(static_cast<T*>(a.sum) + row * a.lds + k, n, h);
        }
    }
};

template <class T>
struct SiluOp {
    typedef SiluSrc<T> Src;
    typedef T In;
    static __device__ __forceinline__ Src src(const RowArgs& a, int64_t row) {
        return Src{static_cast<const T*>(a.x) + row * a.ldx, static_cast<const T*>(a.r) + row * a.ldr};
    }
    static __device__ __forceinline__ void first(const RowArgs& a, int64_t row, int64_t k, int n, float (&p)[kChunk],
                                                 float (&)[kChunk]) {
        float b[kChunk];
        load_chunk(static_cast<const T*>(a.x) + row * a.ldx + k, n, p);
        load_chunk(static_cast<const T*>(a.r) + row * a.ldr + k, n, b);
uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            bool hard;
            p[j] = silu_mul_fast(p[j], b[j], hard);
            mask |= hard ? 1u << j : 0u;
        }
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
// data. NV = 0: rows of any length, read a second time for the codes.
template <class Op, int OUT, class OutT, int TPR, int NV>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void row_kernel(RowArgs a) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    constexpr bool kNorm = Op::Src::kNorm;
    constexpr int W = TPR / 64;
    __shared__ double sh_d[3][W];
    __shared__ uint32_t sh_u[W];
    const int lane = TPR == 64 ? static_cast<int>(threadIdx.x & 63) : static_cast<int>(threadIdx.x);
    const int chunks = static_cast<int>((a.K + kChunk - 1) / kChunk);
    const int per = NV > 0 ? NV : (chunks + TPR - 1) / TPR;

    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + (TPR == 64 ? threadIdx.x >> 6 : 0); row < a.M;
         row += static_cast<int64_t>(gridDim.x) * RPB) {
        float keep[NV > 0 ? NV : 1][kChunk];
        float keep_w[NV > 0 && kNorm ? NV : 1][kChunk];
        uint32_t top = 0;
        double top_d = 0.0, ss = 0.0;

        auto chunk_n = [&](int i) { return static_cast<int64_t>(i * TPR + lane) * kChunk; };
        auto take = [&](int i, float (&v)[kChunk], float (&w)[kChunk]) {
            const int64_t k = chunk_n(i);
            const int n = k < a.K ? static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk) : 0;
            if (n > 0) {
                Op::first(a, row, k, n, v, w);
            } else {
#pragma unroll
                for (int j = 0; j < kChunk; ++j) v[j] = w[j] = 0.0f;
            }
        };
        auto look = [&](float (&v)[kChunk], const float (&w)[kChunk]) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                if constexpr (kNorm) {
                    const double h = v[j];
                    ss = __builtin_fma(h, h, ss);
                    if constexpr (OUT != kOutDense) {
                        top_d = __builtin_fmax(top_d, __builtin_fabs(h * static_cast<double>(w[j])));
                        top = Max32()(top, abs_bits(v[j] * w[j]));
                    }
                } else if constexpr (OUT != kOutDense) {
                    top = Max32()(top, abs_bits(v[j]));
                }
            }
        };
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) take(i, keep[i], keep_w[kNorm ? i : 0]);
#pragma unroll
            for (int i = 0; i < NV; ++i) look(keep[i], keep_w[kNorm ? i : 0]);
        } else {
            for (int i = 0; i < per; ++i) {
                take(i, keep[0], keep_w[0]);
                look(keep[0], keep_w[0]);
            }
        }
        // The row's slots of the last row may still be read.
        if constexpr (TPR > 64) __syncthreads();
        double r = 1.0;
        if constexpr (kNorm) {
            ss = row_reduce<TPR>(ss, sh_d[0], Add64());
            r = 1.0 / __builtin_sqrt(ss / static_cast<double>(a.K) + static_cast<double>(a.eps));
        }

        const typename Op::Src src = Op::src(a, row);
        if constexpr (OUT == kOutDense) {
            OutT* out = static_cast<OutT*>(a.out) + row * a.K;
            const float rf = static_cast<float>(r);
            auto put = [&](int i, float (&v)[kChunk], const float (&w)[kChunk]) {
                const int64_t k = chunk_n(i);
                if (k >= a.K) return;
                const int n = static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk);
                if constexpr (kNorm) {
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) v[j] = v[j] * rf * w[j];
                }
                store_chunk(out + k, n, v);
            };
            if constexpr (NV > 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) put(i, keep[i], keep_w[kNorm ? i : 0]);
            } else {
                for (int i = 0; i < per; ++i) {
                    if constexpr (kNorm) {
                        const int64_t k = chunk_n(i);
                        const int n = k < a.K ? static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk) : 0;
                        load_chunk(src.h + k, n, keep[0]);
                        load_chunk(src.w + k, n, keep_w[0]);
                    } else {
                        take(i, keep[0], keep_w[0]);
                    }
                    put(i, keep[0], keep_w[0]);
                }
            }
        } else {
            typedef CodeOf<OUT> Code;
            top = row_reduce<TPR>(top, sh_u, Max32());
            const float pf = as_float(top);
            const bool fast = pf >= 0x1p-60f && pf <= 0x1p120f;      // false for NaN
            double P;
            if (fast) {
                if constexpr (kNorm) {
                    P = row_reduce<TPR>(top_d, sh_d[1], Max64());
                } else if constexpr (Op::Src::kCandidates) {
                    const float near = pf * (1.0f - 2.0f * Op::Src::kDelta);
                    double best = 0.0;
                    auto candidates = [&](const float (&v)[kChunk]) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) mask |= __builtin_fabsf(v[j]) >= near ? 1u << j : 0u;
                        return mask;
                    };
                    auto settle = [&](int i0, uint32_t mask) {
                        while (mask) {
                            const int b = __builtin_ctz(mask);
                            mask &= mask - 1u;
                            best = __builtin_fmax(best, __builtin_fabs(src.exact(chunk_n(i0 + b / kChunk) + b % kChunk)));
                        }
                    };
                    if constexpr (NV > 0) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int i = 0; i < NV; ++i) mask |= candidates(keep[i]) << (kChunk * i);
                        settle(0, mask);
                    } else {
                        for (int i = 0; i < per; ++i) {
                            take(i, keep[0], keep_w[0]);
                            settle(i, candidates(keep[0]));
                        }
                    }
                    P = row_reduce<TPR>(best, sh_d[1], Max64());
                } else {
                    P = static_cast<double>(pf);
                }
            } else {
                double best = 0.0;
                for (int i = 0; i < per; ++i) {
                    const int64_t k = chunk_n(i);
                    for (int j = 0; j < kChunk; ++j) {
                        if (k + j >= a.K) continue;
                        const double p = __builtin_fabs(src.exact(k + j));
                        best = __builtin_fmax(best, p <= DBL_MAX ? p : static_cast<double>(__builtin_inff()));
                    }
                }
                P = row_reduce<TPR>(best, sh_d[1], Max64());
            }
            const float scale = static_cast<float>(P * r / static_cast<double>(Code::kTop));
            const bool fine = scale <= FLT_MAX;                      // false for NaN and infinity
            if (lane == 0) a.scale[row] = fine ? scale : __builtin_nanf("");
            uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.K;
            const bool zero = !fine || P == 0.0;
            const float inv = static_cast<float>(static_cast<double>(Code::kTop) / P);
            // Stores the codes of chunk i; returns the elements still to be taken in fp64.
            auto put = [&](int i, const float (&v)[kChunk], const float (&w)[kChunk]) {
                const int64_t k = chunk_n(i);
                if (k >= a.K) return 0u;
                const int n = static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk);
                u32x2 c = {0u, 0u};
                uint32_t mask = zero ? 0u : 0xffu;
                if (fast && fine) {
                    float p[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) p[j] = kNorm ? v[j] * w[j] : v[j];
                    c = fast_codes<OUT>(p, inv, Op::Src::kDelta, mask);
                }
                store_codes(out + k, n, c);
                return mask & ((1u << n) - 1u);
            };
            // The same thread stored these elements' chunk, so the bytes land in this order.
            auto settle = [&](int i0, uint32_t mask) {
                while (mask) {
                    const int b = __builtin_ctz(mask);
                    mask &= mask - 1u;
                    const int64_t k = chunk_n(i0 + b / kChunk) + b % kChunk;
                    out[k] = static_cast<uint8_t>(Code::exact(src.exact(k), P));
                }
            };
            if constexpr (NV > 0) {
                uint32_t mask = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) mask |= put(i, keep[i], keep_w[kNorm ? i : 0]) << (kChunk * i);
                settle(0, mask);
            } else {
                for (int i = 0; i < per; ++i) {
                    if constexpr (kNorm) {
                        const int64_t k = chunk_n(i);
                        const int n = k < a.K ? static_cast<int>(a.K - k < kChunk ? a.K - k : kChunk) : 0;
                        load_chunk(src.h + k, n, keep[0]);
                        load_chunk(src.w + k, n, keep_w[0]);
                    } else {
                        take(i, keep[0], keep_w[0]);
                    }
                    settle(i, put(i, keep[0], keep_w[0]));
                }
            }
        }
    }
}

constexpr int64_t kMaxGrid = 1 << 20;

template <class Op, int OUT, class OutT, int TPR, int NV>
hipError_t launch_rows(const RowArgs& a, hipStream_t stream) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    const int64_t blocks = (a.M + RPB - 1) / RPB;
    row_kernel<Op, OUT, OutT, TPR, NV><<<static_cast<uint32_t>(blocks < kMaxGrid ? blocks : kMaxGrid),
                                         TPR == 64 ? 256 : TPR, 0, stream>>>(a);
    return hipGetLastError();
}

// Threads and chunks per row by its length alone.
template <class Op, int OUT, class OutT>
hipError_t launch_by_length(const RowArgs& a, hipStream_t stream) {
    if (a.K <= 64 * 8) return launch_rows<Op, OUT, OutT, 64, 1>(a, stream);
    if (a.K <= 64 * 16) return launch_rows<Op, OUT, OutT, 64, 2>(a, stream);
    if (a.K <= 256 * 8) return launch_rows<Op, OUT, OutT, 256, 1>(a, stream);
    if (a.K <= 256 * 16) return launch_rows<Op, OUT, OutT, 256, 2>(a, stream);
    if (a.K <= 256 * 32) return launch_rows<Op, OUT, OutT, 256, 4>(a, stream);
    if (a.K <= 1024 * 16) return launch_rows<Op, OUT, OutT, 1024, 2>(a, stream);
    return launch_rows<Op, OUT, OutT, 1024, 0>(a, stream);
}

template <template <class> class Op, class T>
hipError_t launch_by_out(const RowArgs& a, int fmt, int out_dtype, hipStream_t stream) {
    if (fmt == RTQ_FMT_Q8) return launch_by_length<Op<T>, kOutQ8, uint8_t>(a, stream);
    if (fmt == RTQ_FMT_F8) return launch_by_length<Op<T>, kOutF8, uint8_t>(a, stream);
    if constexpr (!__is_same(Op<T>, PlainOp<T>)) {
        if (out_dtype == RTQ_F32) return launch_by_length<Op<T>, kOutDense, float>(a, stream);
        return launch_by_length<Op<T>, kOutDense, T>(a, stream);
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
