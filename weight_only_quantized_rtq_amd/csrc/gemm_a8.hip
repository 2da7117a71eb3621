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

#include <type_traits>

#include "rtq_internal.h"
#include "split_device.h"

namespace rtq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBK = 128;                   // bytes (= elements) of K per stage
constexpr int kBand = 4;                   // tiles of m that a band of tiles covers

constexpr bool is_int(int kind) { return kind == kA8Int || kind == kA8IntWide; }
constexpr bool is_wide(int kind) { return kind == kA8IntWide || kind == kA8F8Wide; }

template <int KIND>
struct Acc {
    typedef std::conditional_t<is_int(KIND), i32x4, floatx4> T;
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
    if constexpr (is_int(KIND)) {
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

// 16 bytes v, the first `s` dropped (s >= 0; zeros come in behind).
__device__ __forceinline__ i32x4 drop_bytes(i32x4 v, int s) {
    const int zero = 0, q = s >> 2;
    i32x4 a, b, c;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = q & 1 ? (j < 3 ? v[j + 1] : zero) : v[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = q & 2 ? (j < 2 ? a[j + 2] : zero) : a[j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = static_cast<int>(__builtin_amdgcn_alignbyte(static_cast<uint32_t>(j < 3 ? b[j + 1] : zero),
                                                           static_cast<uint32_t>(b[j]), static_cast<uint32_t>(s & 3)));
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = s < 16 ? c[j] : zero;
    return c;
}

// 16 bytes of a row of K >= 16 at k, zeros past K. A chunk that the row ends
// in is the row's last 16 bytes, shifted: one load without a branch.
__device__ __forceinline__ i32x4 load16(const uint8_t* row, int k, int K) {
    i32x4 v;
    const int at = min(k, K - 16);
    __builtin_memcpy(&v, row + at, 16);
    return drop_bytes(v, k - at);
}

// 16 bytes at any address, from the aligned words that hold them. Each word
// holds at least one of the 16 bytes, so none lies outside the tensor's words.
__device__ __forceinline__ i32x4 load_words(const uint8_t* p) {
    typedef int W4 __attribute__((ext_vector_type(4), aligned(4)));
    const uint32_t r = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3u;
    const W4 v = *reinterpret_cast<const W4*>(p - r);
    const int last = *reinterpret_cast<const int*>(p + (15u - ((r + 15u) & 3u)));
    i32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = static_cast<int>(__builtin_amdgcn_alignbyte(static_cast<uint32_t>(j < 3 ? v[j + 1] : last),
                                                           static_cast<uint32_t>(v[j]), r));
    return o;
}

// load16 for K < 16, byte by byte.
__device__ __forceinline__ i32x4 load_bytes(const uint8_t* row, int k, int K) {
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (k + j < K) v[j / 4] |= static_cast<int>(row[k + j]) << (8 * (j % 4));
    return v;
}

// The workgroup's task and its number among the task's workgroups.
__device__ __forceinline__ const A8Task& task_of(const A8Args& args, uint32_t w, int& at) {
    int j = 0;
#pragma unroll
    for (int i = 1; i < kA8Slots; ++i) j += i < args.count && args.begin[i] <= w;
    j = __builtin_amdgcn_readfirstlane(j);
    at = static_cast<int>(w - args.begin[j]);
    return args.task[j];
}

// Four fp32 values of a vector at n, those past N from its last element; `none` without a vector.
__device__ __forceinline__ floatx4 channels(const float* p, int n, int N, float none) {
    floatx4 v = {none, none, none, none};
    if (!p) return v;
    if (n + 4 <= N) {
        __builtin_memcpy(&v, p + n, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p[min(n + e, N - 1)];
    }
    return v;
}

// An output in fp32: sum * (row scale * channel scale) + bias.
template <class T>
__device__ __forceinline__ float scaled(T sum, float s, float sw, float bias) {
    return __builtin_fmaf(static_cast<float>(sum), s * sw, bias);
}

// y[n .. n+C-1] of one row, in one store of up to 16 bytes. Nontemporal: y is not read
// here, and lines held back to be completed in L2 evict what is (65536 x 2048
// x 512 int8 to fp32: 201 us without, 168 with).
template <int C, class T>
__device__ __forceinline__ void put(T* y, int n, int N, const float (&v)[C]) {
    typedef T V __attribute__((ext_vector_type(C), aligned(sizeof(T))));
    V w;
#pragma unroll
    for (int e = 0; e < C; ++e) {
        float f = v[e];
        // the fp32 value itself: fused with the conversion to fp16 the last
        // operation would round once, in some kernels and not in others
        if constexpr (__is_same(T, _Float16)) asm("" : "+v"(f));
        w[e] = static_cast<T>(f);
    }
    if (n + C <= N) {
        __builtin_nontemporal_store(w, reinterpret_cast<V*>(y + n));
    } else {
#pragma unroll
        for (int e = 0; e < C; ++e)
            if (n + e < N) y[n + e] = w[e];
    }
}

// f(pointer of y's type)
template <int KIND, class F>
__device__ __forceinline__ void by_type(const A8Task& t, F f) {
    if constexpr (is_wide(KIND)) {
        f(static_cast<float*>(t.y));
    } else {
        if (t.y_dtype == RTQ_F16) f(static_cast<_Float16*>(t.y));
        else f(static_cast<__bf16*>(t.y));
    }
}

// ---- few rows: weights straight to registers, K split over the waves ----
//
// A workgroup of W waves owns 16 n and 16 MT m. Each wave takes every W-th
// 128 of K, reads its operands from global memory into registers (each weight
// byte once over the whole grid for M <= 16 MT) and the waves' sums meet in
// LDS, in the order of the waves. Bound by the weight stream: 1 x 8192 x 8192
// int8 takes 13.7 us, 4.9 TB/s of weights. Through LDS one row would leave 31
// of 32 rows of a stage's copies empty.
template <int KIND, int MT, int W, bool ALIGNED>
__global__ __launch_bounds__(W * 64) void skinny_kernel(const A8Args args) {
    typedef typename Acc<KIND>::T V;
    __shared__ V part[W][MT][64];
    int tile;
    const A8Task& t = task_of(args, blockIdx.x, tile);
    const int tiles_n = (t.N + 15) / 16;
    const int64_t m0 = static_cast<int64_t>(tile / tiles_n) * (16 * MT);
    const int n0 = tile % tiles_n * 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int K = t.K;
    // rows past the end repeat the last one; their outputs are not stored
    const uint8_t* w = t.w + static_cast<int64_t>(min(n0 + r16, t.N - 1)) * K + g * 16;
    const uint8_t* x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + i * 16 + r16;
        x[i] = t.x + (m < args.M ? m : args.M - 1) * K + g * 16;
    }
    V acc[MT] = {};
    int k = wave * kBK;
    auto whole_steps = [&](auto load) {
        for (; k + kBK <= K; k += W * kBK) {
            const i32x4 a0 = load(w + k), a1 = load(w + k + 64);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = mma<KIND>(a0, a1, load(x[i] + k), load(x[i] + k + 64), acc[i]);
        }
    };
    // Rows off the words go through words: 80 x 512 x 2049 takes 6.3 us, 10.4
    // with loads at the bytes' own addresses. Rows on the words take those
    // addresses: 80 x 512 x 2056 takes 4.3 us, 5.2 through words.
    if (!ALIGNED && ((static_cast<uint32_t>(K) | static_cast<uint32_t>(reinterpret_cast<uintptr_t>(t.x)) |
                      static_cast<uint32_t>(reinterpret_cast<uintptr_t>(t.w))) & 3u))
        whole_steps([](const uint8_t* p) { return load_words(p); });
    else
        whole_steps([](const uint8_t* p) {
            i32x4 v;
            __builtin_memcpy(&v, p, 16);
            return v;
        });
    if (k < K) {                                               // the last, partial step
        auto last = [&](const uint8_t* p, int at) {            // p is 16 g into its row
            if constexpr (ALIGNED) {
                i32x4 v = {0, 0, 0, 0};
                if (at + g * 16 < K) __builtin_memcpy(&v, p + at, 16);
                return v;
            } else {
                return K >= 16 ? load16(p - g * 16, at + g * 16, K) : load_bytes(p - g * 16, at + g * 16, K);
            }
        };
        const i32x4 a0 = last(w, k), a1 = last(w, k + 64);
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = mma<KIND>(a0, a1, last(x[i], k), last(x[i], k + 64), acc[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * 64; q += W * 64) {
        const int i = q >> 6;
        V sum = part[0][i][lane];
#pragma unroll
        for (int v = 1; v < W; ++v) sum += part[v][i][lane];
        const int64_t m = m0 + i * 16 + r16;
        const int n = n0 + g * 4;
        if (m < args.M && n < t.N) {
            const floatx4 sw = channels(t.w_scale, n, t.N, 1.0f), bias = channels(t.bias, n, t.N, 0.0f);
            const float s = t.x_scale[m];
            float y4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y4[e] = scaled(sum[e], s, sw[e], bias[e]);
            by_type<KIND>(t, [&](auto* y) { put(y + m * t.ldy, n, t.N, y4); });
        }
    }
}

// ---- tiles through LDS ----

// Which n of a wave's tile is row a (0 .. 15) of its block i. A lane ends with
// rows 4g .. 4g+3 of every block (g = lane / 16); with a 16-bit y the rows of
// two blocks interleave in fours, so a lane's eight n of a pair are adjacent
// and leave in one 16-byte store.
template <bool WIDE>
__device__ __forceinline__ int n_row(int i, int a) {
    if constexpr (WIDE) return i * 16 + a;
    else return (i >> 1) * 32 + (a >> 2) * 8 + (i & 1) * 4 + (a & 3);
}

// LDS: rows of 128 bytes, the 16-byte chunk c of row r at slot c ^ key(r): the
// eight rows that are read together have eight keys, so they cover all banks.
// key is r & 7 where those are rows 0 .. 7 or 8 .. 15, and for the interleaved
// n rows, 0 .. 3 with 8 .. 11, bit 3 of r takes the place of bit 2.
template <bool PLAIN>
__device__ __forceinline__ int lds_key(int r) {
    return PLAIN ? r & 7 : (r & 3) | ((r >> 1) & 4);
}
template <bool PLAIN>
__device__ __forceinline__ int lds_at(int r, int c) { return r * kBK + ((c ^ lds_key<PLAIN>(r)) << 4); }

__device__ const uint32_t zero_chunk[4] = {0, 0, 0, 0};

template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70 | 0xf00);
}

__device__ __forceinline__ void dma16(const uint8_t* src, uint8_t* lds_base) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)lds_base, 16, 0, 0);
}

// BM x BN outputs by WM x WN waves, stages of 128 of K in S LDS buffers: the
// next S - 1 stages are copied (DMA to LDS, or through registers, S = 2, where
// rows are not 16-byte aligned) while one is multiplied. KS teams of such
// waves, each with its own buffers, take every KS-th stage, and their sums
// meet in LDS at the end: where a CU has one workgroup, a stage takes as long
// as its copies' latency, and the teams' overlap.
//
// 8192^3 E4M3 to bf16 takes 406 us (2.7 PFLOP/s): bound by the matrix
// instructions. 65536 x 2048 x 512 int8 to fp32 takes 145 us (4.0 TB/s, 97 us
// with the stores left out): bound by y's stores and, at four stages a tile, by
// the ends of tiles that nothing overlaps.
template <int KIND, int BM, int BN, int WM, int WN, int S, int KS, bool ALIGNED>
__global__ __launch_bounds__(WM * WN * KS * 64) void tile_kernel(const A8Args args) {
    constexpr int NW = WM * WN, ROWS = BM + BN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int OPS = ROWS / 8 / NW;                         // 1 KB copies of 8 rows, per wave and stage
    static_assert(ROWS % (8 * NW) == 0 && BM % (8 * NW) == 0, "copies divide over the waves");
    static_assert(NW % 2 == 0 && BM % 16 == 0 && TN % 2 == 0, "keys and pairs of blocks");
    static_assert(ALIGNED || S == 2, "copies through registers run one stage ahead");
    __shared__ __align__(1024) uint8_t lds_all[KS][S][ROWS * kBK];     // rows 0 .. BM-1: x, then the weights
    int tile;
    const A8Task& t = task_of(args, xcd_remap_split(blockIdx.x, args.total), tile);
    const int K = t.K;
    // Each XCD works on a run of tiles; a run goes through bands of kBand
    // tiles of m, so the tiles in flight on it share rows and weights in its L2.
    const int tiles_n = (t.N + BN - 1) / BN, tiles_m = static_cast<int>((args.M + BM - 1) / BM);
    const int band = tile / (kBand * tiles_n), in_band = tile % (kBand * tiles_n);
    const int high = min(kBand, tiles_m - band * kBand);
    const int64_t m0 = static_cast<int64_t>(band * kBand + in_band % high) * BM;
    const int n0 = in_band / high * BN;
    const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int team = KS == 1 ? 0 : wave_all / NW, wave = KS == 1 ? wave_all : wave_all % NW;
    uint8_t(&lds)[S][ROWS * kBK] = lds_all[team];
    const int wm = wave % WM * (TM * 16), wn = wave / WM * (TN * 16);
    const int r16 = lane & 15, g = lane >> 4;
    const uint8_t* xb = t.x + m0 * K;
    const uint8_t* wb = t.w + static_cast<int64_t>(n0) * K;

    // Copy j of this wave: rows 8 (j NW + wave) .. + 7, lane: row lane / 8, slot lane % 8.
    // The key of such a row depends on lane / 8 and, for the weights' interleave,
    // on the parity of wave (NW and BM / 8 are even).
    constexpr bool kWide = is_wide(KIND);
    const int chunk_x = ((lane & 7) ^ lds_key<true>(lane >> 3)) * 16;
    const int chunk_w = ((lane & 7) ^ lds_key<kWide>((lane >> 3) + 8 * (wave & 1))) * 16;
    uint32_t off[OPS];
#pragma unroll
    for (int j = 0; j < OPS; ++j) {
        const int r = 8 * (j * NW + wave) + (lane >> 3);
        // rows past the end repeat the last one; their outputs are not stored
        const int64_t left = r < BM ? args.M - 1 - m0 : static_cast<int64_t>(t.N) - 1 - n0;
        const int row = r < BM ? r : r - BM;
        off[j] = static_cast<uint32_t>(row < left ? row : static_cast<int>(left)) * static_cast<uint32_t>(K);
    }
    i32x4 hold[ALIGNED ? 1 : OPS];
    auto issue = [&](int step, int buf) {
        const int k0 = (step * KS + team) * kBK;
        const uint8_t *x0 = xb + k0, *w0 = wb + k0;
        if (k0 + kBK <= K) {
#pragma unroll
            for (int j = 0; j < OPS; ++j) {
                const bool is_x = j * NW * 8 < BM;
                const uint8_t* src = (is_x ? x0 : w0) + (off[j] + static_cast<uint32_t>(is_x ? chunk_x : chunk_w));
                if constexpr (ALIGNED) dma16(src, &lds[buf][(j * NW + wave) * 1024]);
                else {
                    i32x4 v;
                    __builtin_memcpy(&v, src, 16);
                    hold[j] = v;
                }
            }
        } else {                                               // the last stage: zeros past K
#pragma unroll
            for (int j = 0; j < OPS; ++j) {
                const bool is_x = j * NW * 8 < BM;
                const int chunk = is_x ? chunk_x : chunk_w;
                const uint8_t* row = (is_x ? xb : wb) + off[j];
                if constexpr (ALIGNED) {
                    const uint8_t* src = k0 + chunk < K ? row + k0 + chunk : reinterpret_cast<const uint8_t*>(zero_chunk);
                    dma16(src, &lds[buf][(j * NW + wave) * 1024]);
                } else {
                    hold[j] = load16(row, k0 + chunk, K);
                }
            }
        }
    };
    auto settle = [&](int buf) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int j = 0; j < OPS; ++j)
                *reinterpret_cast<i32x4*>(&lds[buf][(j * NW + wave) * 1024 + lane * 16]) = hold[j];
        }
    };

    typename Acc<KIND>::T acc[TN][TM] = {};
    const int stages = (K + kBK - 1) / kBK;                    // mine: this team's
    const int steps = (stages + KS - 1) / KS, mine = KS == 1 ? steps : (stages - team + KS - 1) / KS;
    // Every buffer is free at the start, so S stages are on their way; from the
    // second step on each step issues the one that its predecessor made room for.
    constexpr int kStart = ALIGNED ? S : 1;
#pragma unroll
    for (int j = 0; j < kStart; ++j)
        if (j < mine) issue(j, j);
    settle(0);
    auto stage = [&](int step, auto buf_c) {
        constexpr int buf = decltype(buf_c)::value, ahead = (buf + S - 1) % S;
        if constexpr (ALIGNED) {
            // Nothing moves past here: the last stage's LDS reads are all
            // used, so complete, before the barrier that frees their buffer.
            __builtin_amdgcn_sched_barrier(0);
            // This wave's part of the stage. The stages issued after it may stay
            // in flight: S - 2 of them, at the first step S - 1 (with fewer
            // steps left than that, wait for all).
            if (step == 0 && mine >= S) wait_vm<(S - 1) * OPS>();
            else if (S == 2 || step + S - 1 > mine) wait_vm<0>();
            else wait_vm<(S - 2) * OPS>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        } else {
            __syncthreads();
        }
        if (KS > 1 && step >= mine) return;
        const bool more = step + S - 1 < mine && (!ALIGNED || step > 0);
        const uint8_t* xs = lds[buf] + wm * kBK;
        const uint8_t* ws = lds[buf] + (BM + wn) * kBK;
        i32x4 b[TM][2], a[TN][2];
        auto read_a = [&](int i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                a[i][h] = *reinterpret_cast<const i32x4*>(ws + lds_at<kWide>(n_row<kWide>(i, r16), g + 4 * h));
        };
        // Enough operands for the first products are on their way before the
        // copies are issued (LDS reads do not move across those).
        constexpr int kFirst = TN < 2 ? TN : 2;
#pragma unroll
        for (int q = 0; q < TM; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[q][h] = *reinterpret_cast<const i32x4*>(xs + lds_at<true>(q * 16 + r16, g + 4 * h));
#pragma unroll
        for (int i = 0; i < kFirst; ++i) read_a(i);
        if (more) issue(step + S - 1, ahead);
        // While one wave of a SIMD reads operands the other's matrix instructions
        // go first (8192^3 E4M3: 414 -> 409 us; with the bf16 conversions between
        // them it costs instead, 55.7 -> 66.7 us for 16384 x 2048 x 512).
        if constexpr (KIND != kA8F8Wide) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = kFirst; i < TN; ++i) read_a(i);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < TM; ++q) acc[i][q] = mma<KIND>(a[i][0], a[i][1], b[q][0], b[q][1], acc[i][q]);
        if constexpr (KIND != kA8F8Wide) __builtin_amdgcn_s_setprio(0);
        if (more) settle(ahead);
    };
    for (int step = 0; step < steps; step += S) {              // buffers by constant numbers
        stage(step, std::integral_constant<int, 0>());
        if constexpr (S > 1) { if (step + 1 < steps) stage(step + 1, std::integral_constant<int, 1 % S>()); }
        if constexpr (S > 2) { if (step + 2 < steps) stage(step + 2, std::integral_constant<int, 2 % S>()); }
        if constexpr (S > 3) { if (step + 3 < steps) stage(step + 3, std::integral_constant<int, 3 % S>()); }
    }

    if constexpr (KS > 1) {                                    // the teams' sums, in their order
        typedef typename Acc<KIND>::T V;
        static_assert(sizeof(V) == 16 && BM * BN * 4 <= S * ROWS * kBK, "a team's sums fit its buffers");
        __syncthreads();
        if (team > 0) {
            V* part = reinterpret_cast<V*>(&lds[0][0]) + wave * (TN * TM * 64) + lane;
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int q = 0; q < TM; ++q) part[(i * TM + q) * 64] = acc[i][q];
        }
        __syncthreads();
        if (team > 0) return;
#pragma unroll
        for (int v = 1; v < KS; ++v) {
            const V* part = reinterpret_cast<const V*>(&lds_all[v][0][0]) + wave * (TN * TM * 64) + lane;
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int q = 0; q < TM; ++q) acc[i][q] += part[(i * TM + q) * 64];
        }
    }

    // Lane: m = lane % 16 of each block q; C adjacent n of each group of
    // blocks, as n_row puts them.
    constexpr int C = kWide ? 4 : 8, P = C / 4;                // n of a store, blocks it takes
    const int mq = wm + r16, nq = n0 + wn + g * C;
    const int M = args.M - m0 < BM ? static_cast<int>(args.M - m0) : BM;     // rows of this tile
    float sx[TM];
#pragma unroll
    for (int q = 0; q < TM; ++q) sx[q] = t.x_scale[m0 + min(mq + q * 16, M - 1)];
    by_type<KIND>(t, [&](auto* y) {
        y += m0 * t.ldy;
        auto finish = [&](int rows, int N) {
#pragma unroll
            for (int i = 0; i < TN; i += P) {
                const int n = nq + i * 16;
                if (n >= N) continue;
                floatx4 sw[P], bias[P];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    sw[p] = channels(t.w_scale, n + 4 * p, N, 1.0f);
                    bias[p] = channels(t.bias, n + 4 * p, N, 0.0f);
                }
#pragma unroll
                for (int q = 0; q < TM; ++q) {
                    if (mq + q * 16 >= rows) continue;
                    float v[C];
#pragma unroll
                    for (int e = 0; e < C; ++e)
                        v[e] = scaled(acc[i + e / 4][q][e % 4], sx[q], sw[e / 4][e % 4], bias[e / 4][e % 4]);
                    put(y + (mq + q * 16) * t.ldy, n, N, v);
                }
            }
        };
        if (M == BM && n0 + BN <= t.N) finish(1 << 30, 1 << 30);       // a whole tile: no tests
        else finish(M, t.N);
    });
}

// Workgroups of every task of a launch, BM x BN outputs each.
uint32_t number(A8Args& args, int BM, int BN) {
    int64_t tiles = 0;
    for (int j = 0; j < args.count; ++j) {
        args.begin[j] = static_cast<uint32_t>(tiles);
        tiles += ((args.M + BM - 1) / BM) * ((args.task[j].N + BN - 1) / BN);
    }
    args.total = static_cast<int32_t>(tiles);
    return static_cast<uint32_t>(tiles);
}

// Whether 256 x 256 tiles, one a CU, pay where there are enough of them. An
// fp32 y of a short K is all stores, which two smaller tiles a CU overlap
// better with loads (65536 x 2048 x 512: 153 us of 128 x 128, 165 us of 256 x
// 256; 65536 x 512 x 2048: 125 and 91; a bf16 y of K = 512: 117 and 104).
template <int KIND, bool ALIGNED>
bool large_pays(const A8Args& args) {
    if constexpr (!ALIGNED && KIND == kA8F8Wide) return false;     // its staging does not fit the registers
    if (!is_wide(KIND)) return true;
    for (int j = 0; j < args.count; ++j)
        if (args.task[j].K < 1024) return false;
    return true;
}

template <int KIND, bool ALIGNED>
hipError_t launch_kind(A8Args& args, hipStream_t stream) {
    auto skinny = [&](auto mt, auto w) {
        constexpr int MT = decltype(mt)::value, W = decltype(w)::value;
        skinny_kernel<KIND, MT, W, ALIGNED><<<number(args, 16 * MT, 16), W * 64, 0, stream>>>(args);
        return hipGetLastError();
    };
    auto tiles = [&](auto bm, auto bn, auto wm, auto wn, auto stages, auto teams) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
        constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value, S = ALIGNED ? decltype(stages)::value : 2;
        constexpr int KS = decltype(teams)::value;
        tile_kernel<KIND, BM, BN, WM, WN, S, KS, ALIGNED><<<number(args, BM, BN), WM * WN * KS * 64, 0, stream>>>(args);
        return hipGetLastError();
    };
    constexpr std::integral_constant<int, 1> c1{};
    constexpr std::integral_constant<int, 2> c2{};
    constexpr std::integral_constant<int, 4> c4{};
    constexpr std::integral_constant<int, 8> c8{};
    constexpr std::integral_constant<int, 32> c32{};
    constexpr std::integral_constant<int, 64> c64{};
    constexpr std::integral_constant<int, 128> c128{};
    constexpr std::integral_constant<int, 256> c256{};
    // Larger blocks read less, smaller ones keep 256 CUs busy: by the call's
    // count of blocks of each size. us, int8 to bf16, M x N x K, as graph
    // replays (the count in brackets):
    //   16 x 16 straight to registers / 32 x 64 tiles: 80 x 512 x 512 (160) 3.3 / 3.8;
    //     96 x 512 x 8192 (192) 9.9 / 11.0; 64 x 2048 x 1024 (512) 4.3 / 4.4; 64 x 2048 x 8192 (512) 13.8 / 12.0
    //   one / two blocks of m a wave: 96 x 512 x 8192 (192) 9.9 / 13.5; 200 x 512 x 8192 (416) 17.2 / 13.7
    //   one / two teams on K, 32 x 64: 80 x 2048 x 512 (96) 3.7 / 4.0; 80 x 2048 x 8192 (96) 14.7 / 11.8;
    //     512 x 2048 x 8192 (512) 20.5 / 23.0; 64 x 64: 512 x 2048 x 8192 (256) 18.8 / 16.0; 1024 x 2048 x 8192 (512) 27.2 / 29.3
    //   32 x 64 / 64 x 64: 700 x 512 x 2048 (176) 6.3 / 7.2; 700 x 2048 x 8192 (704) 29.2 / 25.6
    //   64 x 64 / 128 x 128: 1500 x 512 x 8192 (192) 18.6 / 33.4; 1500 x 2048 x 8192 (768) 43.6 / 36.5
    //   128 x 128 of eight waves and four stages, one a CU / of four waves and
    //     two stages, two a CU: 1500 x 2048 x 8192 (192) 36.5 / 46.2; 3000 x 2048 x 8192 (384) 70.5 / 55.3
    //   128 x 128 / 256 x 256: a round of 512 takes 4/7 of a round of 256 of
    //     the large ones: 1500 x 8192 x 8192 (768, 192) 106.6 / 94.0; 3000 x 8192 x 8192 (1536, 384) 188.7 / 195.9
    // Where rows are not 16-byte aligned: 16 x 16 / 32 x 64: 200 x 512 x 8190
    // (416) 18.7 / 24.9; 300 x 512 x 2049 (608) 12.5 / 8.9. One / two / four
    // teams: 32 x 64, 150 x 2048 x 8190 (160) 41.5 / 30.4 / 24.7; 64 x 64,
    // 500 x 2048 x 2049 (256) 16.2 / 13.8 / 12.5; 128 x 128 of eight waves,
    // one team or two of four waves: 2048 x 2048 x 8190 (256) 69.4 / 59.5.
    const int64_t n16 = number(args, 16, 16);
    bool short_k = false, long_k = false;
    for (int j = 0; j < args.count; ++j) {
        short_k |= args.task[j].K < 16;                        // the tiles load 16 bytes of a row at a time
        long_k |= args.task[j].K > 8 * kBK;
    }
    if (args.M <= 16 || short_k || n16 <= 256) return skinny(c1, c8);
    if (n16 <= 512 && !(ALIGNED && long_k)) return skinny(c2, c8);
    constexpr std::integral_constant<int, ALIGNED ? 2 : 4> teams{};
    if (long_k && number(args, 32, 64) <= 256) return tiles(c32, c64, c2, c2, c4, teams);
    if (long_k && number(args, 64, 64) <= 256) return tiles(c64, c64, c2, c2, c4, teams);
    if (number(args, 32, 64) <= 512) return tiles(c32, c64, c2, c2, c4, c1);
    if (number(args, 64, 64) <= 512) return tiles(c64, c64, c2, c2, c4, c1);
    const int64_t n128 = number(args, 128, 128), n256 = number(args, 256, 256);
    if (n128 <= 256) {
        if (!ALIGNED && long_k) return tiles(c128, c128, c2, c2, c2, c2);
        return tiles(c128, c128, c4, c2, c4, c1);
    }
    const int64_t rounds128 = (n128 + 511) / 512 * 4, rounds256 = (n256 + 255) / 256 * 7;
    if (rounds128 < rounds256 || !large_pays<KIND, ALIGNED>(args)) return tiles(c128, c128, c2, c2, c2, c1);
    if constexpr (ALIGNED || KIND != kA8F8Wide) return tiles(c256, c256, c4, c2, c2, c1);
    return tiles(c128, c128, c2, c2, c2, c1);
}

bool task_aligned(const A8Task& t) {
    return t.K % 16 == 0 && ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.w)) & 15) == 0;
}

}  // namespace

hipError_t launch_a8(const A8Task* tasks, int count, int64_t M, hipStream_t stream) {
    // A grid holds fewer than 2^32 threads: one launch covers at most 2^22 of
    // the smallest blocks (16 x 16, 512 threads), so wide tasks go in pieces
    // of columns and tall ones in pieces of rows.
    constexpr int64_t kMaxBlocks = int64_t(1) << 22;
    constexpr int kMaxCols = static_cast<int>(kMaxBlocks / kA8Slots * 16);
    A8Args args;
    // One launch holds tasks of one kind, and of one of the two ways to load.
    for (int pass = 0; pass < kA8Kinds * 2; ++pass) {
        const int kind = pass / 2;
        const bool whole = pass % 2 == 0;
        int at = 0, col = 0;                                   // the next task and its first column
        while (at < count) {
            int64_t blocks_n = 0;
            A8Task slot[kA8Slots];
            args.count = 0;
            while (at < count && args.count < kA8Slots) {
                if (tasks[at].kind != kind || task_aligned(tasks[at]) != whole) {
                    ++at;
                    continue;
                }
                A8Task& t = slot[args.count++] = tasks[at];
                t.w += static_cast<int64_t>(col) * t.K;
                if (t.w_scale) t.w_scale += col;
                if (t.bias) t.bias += col;
                t.y = static_cast<uint8_t*>(t.y) + static_cast<int64_t>(col) * (t.y_dtype == RTQ_F32 ? 4 : 2);
                t.N = t.N - col < kMaxCols ? t.N - col : kMaxCols;
                col += t.N;
                if (col >= tasks[at].N) {
                    ++at;
                    col = 0;
                }
                blocks_n += (t.N + 15) / 16;
            }
            if (!args.count) break;
            const int64_t most = kMaxBlocks / blocks_n * 16;   // rows of a launch
            for (int64_t m = 0; m < M; m += most) {
                args.M = M - m < most ? M - m : most;
                for (int j = 0; j < args.count; ++j) {
                    A8Task& t = args.task[j] = slot[j];
                    t.x += m * t.K;
                    t.x_scale += m;
                    t.y = static_cast<uint8_t*>(t.y) + m * t.ldy * (t.y_dtype == RTQ_F32 ? 4 : 2);
                }
                auto run = [&](auto k) {
                    constexpr int KIND = decltype(k)::value;
                    return whole ? launch_kind<KIND, true>(args, stream) : launch_kind<KIND, false>(args, stream);
                };
                const int mark = timing_begin(stream);
                const hipError_t e = kind == kA8Int       ? run(std::integral_constant<int, kA8Int>())
                                     : kind == kA8IntWide ? run(std::integral_constant<int, kA8IntWide>())
                                     : kind == kA8F8      ? run(std::integral_constant<int, kA8F8>())
                                                          : run(std::integral_constant<int, kA8F8Wide>());
                timing_end(mark, stream);
                if (e != hipSuccess) return e;
            }
        }
    }
    return hipSuccess;
}

}  // namespace rtq
