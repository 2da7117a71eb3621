// Matrix product of 8-bit activations with 8-bit weights:
//     y[m][n] = sx[m] * sw[n] * sum_k x[m][k] * w[n][k]  (+ bias[n])
// x and w both int8 or both E4M3 (no channel scale). The scales, the bias and
// the rounding to y's type are the epilogue, in fp32.
//
// Sums by kind:
//  - int8: v_mfma_i32_16x16x64_i8, exact in int32 (K < 2^17).
//  - E4M3 with a 16-bit y: v_mfma_f32_16x16x128_f8f6f4. Measured on the
//    instruction: it adds each group of 8 consecutive k of a lane in fixed
//    point with a unit of 2^-13 of the group's largest product (truncating),
//    and the groups' sums in fp32. A group loses at most 7 units, so a sum is
//    off by less than 7 * 2^-13 * sum|x w|; on normal data by 1e-5 of its
//    norm, far below y's own rounding.
//  - E4M3 with an fp32 y: the codes, exact in bf16, go through
//    v_mfma_f32_16x16x32_bf16, whose sums are fp32, at half the rate.
#include <rtq.h>

#include "rtq_internal.h"
#include "split_device.h"

namespace rtq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBK = 128;                   // bytes (= elements) of K per stage

template <int KIND>
struct Acc {
    typedef floatx4 T;
};
template <>
struct Acc<kA8Int> {
    typedef i32x4 T;
};

// Eight E4M3 codes -> bf16, exactly.
__device__ __forceinline__ bf16x8 f8_to_bf16(int w0, int w1) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One 16 x 16 block, 128 of K: each lane holds 32 bytes of one row of each
// operand (the same k of both, so their order within the lane is free).
template <int KIND>
__device__ __forceinline__ typename Acc<KIND>::T mma(i32x4 a0, i32x4 a1, i32x4 b0, i32x4 b1, typename Acc<KIND>::T c) {
    if constexpr (KIND == kA8Int) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, b0, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, b1, c, 0, 0, 0);
    } else if constexpr (KIND == kA8F8) {
        const i32x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const i32x4 a = h < 2 ? a0 : a1, b = h < 2 ? b0 : b1;
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_to_bf16(a[2 * (h & 1)], a[2 * (h & 1) + 1]),
                                                        f8_to_bf16(b[2 * (h & 1)], b[2 * (h & 1) + 1]), c, 0, 0, 0);
        }
        return c;
    }
}

// Four outputs y[m][n .. n+3].
__device__ __forceinline__ void store4(const A8Task& t, int64_t m, int64_t n, const float (&v)[4]) {
    const int64_t at = m * t.ldy + n;
    const int left = static_cast<int>(t.N - n < 4 ? t.N - n : 4);
    auto put = [&](auto* y) {
        typedef __remove_reference_t(decltype(*y)) T;
        T w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = static_cast<T>(v[j]);
        if (left == 4) {
            __builtin_memcpy(y + at, w, sizeof(w));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) y[at + j] = w[j];
        }
    };
    if (t.y_dtype == RTQ_F32) put(static_cast<float*>(t.y));
    else if (t.y_dtype == RTQ_F16) put(static_cast<_Float16*>(t.y));
    else put(static_cast<__bf16*>(t.y));
}

// 16 bytes of a row at k (any alignment), zeros past K.
__device__ __forceinline__ i32x4 load16(const uint8_t* row, int k, int K) {
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K) {
#pragma unroll
        for (int j = 0; j < 15; ++j)
            if (k + j < K) v[j / 4] |= static_cast<int>(row[k + j]) << (8 * (j % 4));
    }
    return v;
}

// LDS: rows of 128 bytes, the 16-byte chunk c of row r at slot c ^ (r & 7).
__device__ __forceinline__ int lds_at(int r, int c) { return r * kBK + ((c ^ (r & 7)) << 4); }

template <int KIND, int BM, int BN>
__global__ __launch_bounds__(256) void tile_kernel(const A8Args args) {
    constexpr int WM = BM / 2, WN = BN / 2;                    // four waves, 2 x 2
    __shared__ __align__(16) uint8_t sx[BM * kBK];
    __shared__ __align__(16) uint8_t sw[BN * kBK];
    int j = 0;
    while (j + 1 < args.count && static_cast<uint32_t>(args.begin[j + 1]) <= blockIdx.x) ++j;
    const A8Task& t = args.task[j];
    const int tile = blockIdx.x - args.begin[j];
    const int tiles_n = (t.N + BN - 1) / BN;
    const int64_t m0 = static_cast<int64_t>(tile / tiles_n) * BM;
    const int64_t n0 = static_cast<int64_t>(tile % tiles_n) * BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave & 1) * WM, wn = (wave >> 1) * WN;
    const int r16 = lane & 15, g = lane >> 4;
    typename Acc<KIND>::T acc[WN / 16][WM / 16] = {};

    for (int k0 = 0; k0 < t.K; k0 += kBK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < BM * 8 / 256; ++i) {
            const int at = i * 256 + threadIdx.x, r = at >> 3, c = at & 7;
            const int64_t m = m0 + r < args.M ? m0 + r : args.M - 1;       // rows past the end: not stored
            *reinterpret_cast<i32x4*>(sx + lds_at(r, c)) = load16(t.x + m * t.K, k0 + c * 16, t.K);
        }
#pragma unroll
        for (int i = 0; i < BN * 8 / 256; ++i) {
            const int at = i * 256 + threadIdx.x, r = at >> 3, c = at & 7;
            const int64_t n = n0 + r < t.N ? n0 + r : t.N - 1;
            *reinterpret_cast<i32x4*>(sw + lds_at(r, c)) = load16(t.w + n * t.K, k0 + c * 16, t.K);
        }
        __syncthreads();
        i32x4 b[WM / 16][2];
#pragma unroll
        for (int i = 0; i < WM / 16; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[i][h] = *reinterpret_cast<const i32x4*>(sx + lds_at(wm + i * 16 + r16, g + 4 * h));
#pragma unroll
        for (int i = 0; i < WN / 16; ++i) {
            i32x4 a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                a[h] = *reinterpret_cast<const i32x4*>(sw + lds_at(wn + i * 16 + r16, g + 4 * h));
#pragma unroll
            for (int q = 0; q < WM / 16; ++q) acc[i][q] = mma<KIND>(a[0], a[1], b[q][0], b[q][1], acc[i][q]);
        }
    }

    // Lane: column m = lane % 16, rows n = 4 (lane / 16) .. + 3 of each block.
#pragma unroll
    for (int q = 0; q < WM / 16; ++q) {
        const int64_t m = m0 + wm + q * 16 + r16;
        if (m >= args.M) continue;
        const float s = t.x_scale[m];
#pragma unroll
        for (int i = 0; i < WN / 16; ++i) {
            const int64_t n = n0 + wn + i * 16 + g * 4;
            if (n >= t.N) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = n + e < t.N ? n + e : t.N - 1;
                const float f = t.w_scale ? s * t.w_scale[at] : s;
                v[e] = static_cast<float>(acc[i][q][e]) * f;
                if (t.bias) v[e] += t.bias[at];
            }
            store4(t, m, n, v);
        }
    }
}

template <int KIND, int BM, int BN>
hipError_t launch_tiles(A8Args& args, hipStream_t stream) {
    int64_t tiles = 0;
    for (int j = 0; j < args.count; ++j) {
        args.begin[j] = static_cast<uint32_t>(tiles);
        tiles += ((args.M + BM - 1) / BM) * ((args.task[j].N + BN - 1) / BN);
    }
    tile_kernel<KIND, BM, BN><<<static_cast<uint32_t>(tiles), 256, 0, stream>>>(args);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_a8(const A8Task* tasks, int count, int64_t M, hipStream_t stream) {
    // Rows of one launch: its tiles stay below 2^23 whatever N is (a grid
    // holds fewer than 2^32 threads).
    constexpr int64_t kMaxTiles = int64_t(1) << 23;
    A8Args args;
    for (int kind = 0; kind < kA8Kinds; ++kind) {
        for (int at = 0; at < count;) {
            int64_t tiles_n = 0;
            const A8Task* slot[kA8Slots];
            args.count = 0;
            for (; at < count && args.count < kA8Slots; ++at) {
                if (tasks[at].kind != kind) continue;
                slot[args.count++] = &tasks[at];
                tiles_n += (tasks[at].N + 63) / 64;
            }
            if (!args.count) break;
            const int64_t most = kMaxTiles / tiles_n > 0 ? kMaxTiles / tiles_n * 64 : 64;
            for (int64_t m = 0; m < M; m += most) {
                args.M = M - m < most ? M - m : most;
                for (int j = 0; j < args.count; ++j) {
                    A8Task& t = args.task[j] = *slot[j];
                    t.x += m * t.K;
                    t.x_scale += m;
                    t.y = static_cast<uint8_t*>(t.y) + m * t.ldy * (t.y_dtype == RTQ_F32 ? 4 : 2);
                }
                const hipError_t e = kind == kA8Int  ? launch_tiles<kA8Int, 64, 64>(args, stream)
                                     : kind == kA8F8 ? launch_tiles<kA8F8, 64, 64>(args, stream)
                                                     : launch_tiles<kA8F8Wide, 64, 64>(args, stream);
                if (e != hipSuccess) return e;
            }
        }
    }
    return hipSuccess;
}

}  // namespace rtq
