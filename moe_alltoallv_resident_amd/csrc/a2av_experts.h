// What the kernels of the experts' products share: the call's arguments, a group's rows, the
// list of row tiles that every block makes from the group starts, and the activation.
#pragma once

#include "../../include/a2av.h"
#include "a2av_internal.h"
#include "a2av_mx.h"

#include <algorithm>
#include <type_traits>

namespace a2av {

constexpr int kWave = 64;
constexpr int kTileRows = 256;           // input rows and weight rows of a tile of the matrix-unit kernel
constexpr uint32_t kStOffsets = 8u;
static_assert(kStOffsets == A2AV_ST_OFFSETS, "status bit");

struct ExpertArgs {
    const uint8_t* in;
    const int32_t* off;      // [R][epr + 1]
    const uint8_t* weight;
    const uint8_t* scales;
    uint8_t* out;
    uint32_t* status;
    int64_t cap;
    int64_t in_row;          // bytes of a row of in, weight and out
    int64_t w_row;
    int64_t out_row;
    int32_t R, epr, G;       // G = R * epr groups
    int32_t K, N;
    int32_t width;           // columns that come out
    int32_t in_dtype, w_dtype, out_dtype;
    int32_t swiglu;
    int32_t few;             // groups of at most so many rows are the few-rows kernel's
    int32_t tile_least;      // fewer tiles than this of larger groups are too
};

struct Group {
    int64_t row;             // first row, counted over all slices
    int32_t rows;
};

// Group g's rows: starts past the capacity are cut to it (a receive overflow), a start out
// of order leaves the group empty.
__device__ inline Group group_of(const ExpertArgs& a, int g, bool* bad) {
    const int d = g / a.epr, le = g - d * a.epr;
    const int32_t* p = a.off + (int64_t)d * (a.epr + 1) + le;
    int32_t b = p[0], e = p[1];
    if (b < 0 || e < b) {
        *bad = true;
        b = e = 0;
    }
    const int32_t cap = (int32_t)a.cap;
    b = min(b, cap);
    e = min(e, cap);
    return Group{(int64_t)d * a.cap + b, e - b};
}

__host__ __device__ inline int pieces_of(int rows, int each) { return rows / each + (rows % each != 0); }

// Sums of four counts over all groups, `counts(rows)` each; every thread of the block calls it and
// has them afterwards.
struct Four {
    int v[4];
};
template <int THREADS, typename F>
__device__ Four count_groups(const ExpertArgs& a, int* wave_sum, F&& counts) {
    Four sum = {{0, 0, 0, 0}};
    bool bad = false;
    for (int g = threadIdx.x; g < a.G; g += THREADS) {
        const Four c = counts(group_of(a, g, &bad).rows);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum.v[k] += c.v[k];
    }
    if (bad && blockIdx.x == 0) atomicOr(a.status, kStOffsets);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) sum.v[k] += __shfl_xor(sum.v[k], m);
        if (threadIdx.x % kWave == 0) wave_sum[threadIdx.x / kWave * 4 + k] = sum.v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < THREADS / kWave; ++w) v += wave_sum[w * 4 + k];
        sum.v[k] = v;
    }
    __syncthreads();
    return sum;
}

// Row tiles of every `each` groups, as ends[i] = tiles of groups 0 .. each * (i + 1) - 1; returns how
// many there are.  Every thread of the block calls it; `tiles(rows)` says how many tiles a group has.
template <int THREADS, typename F>
__device__ int count_tiles(const ExpertArgs& a, int* ends, int* wave_sum, F&& tiles, int each = 1) {
    const int n = (a.G + each - 1) / each;
    const int per = (n + THREADS - 1) / THREADS;
    const int g0 = threadIdx.x * per;
    int sum = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        if (g0 + i >= n) break;
        for (int k = 0; k < each; ++k) {
            const int g = (g0 + i) * each + k;
            if (g < a.G) sum += tiles(group_of(a, g, &bad).rows);
        }
        ends[g0 + i] = sum;
    }
    if (bad && blockIdx.x == 0) atomicOr(a.status, kStOffsets);
    int scan = sum;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        const int up = __shfl_up(scan, m);
        if ((int)(threadIdx.x % kWave) >= m) scan += up;
    }
    if (threadIdx.x % kWave == kWave - 1) wave_sum[threadIdx.x / kWave] = scan;
    __syncthreads();
    int before = scan - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) {
        const int v = wave_sum[w];
        if (w < (int)threadIdx.x / kWave) before += v;
        total += v;
    }
    for (int i = 0; i < per; ++i) {
        if (g0 + i >= n) break;
        ends[g0 + i] += before;
    }
    __syncthreads();
    return total;
}

// Tiles of the groups of more than a.few rows, over the output's width.
__device__ inline int64_t large_tiles(const ExpertArgs& a, int row_tiles) {
    const int cols = a.swiglu ? kTileRows / 2 : kTileRows;
    return (int64_t)row_tiles * ((a.width + cols - 1) / cols);
}

// The list of row tiles has an entry for every group, or for every kCoarse of more than kEntries.
constexpr int kCoarse = 8, kEntries = kMaxExperts / kCoarse;
__device__ inline int groups_an_entry(const ExpertArgs& a) { return a.G > kEntries ? kCoarse : 1; }

struct Piece {
    int group;
    Group rows;
    int n;                   // which of the group's row tiles
};

// Row tile t of the list that count_tiles made with the same `tiles`.  All in scalar registers.
template <typename F>
__device__ inline Piece find_piece(const ExpertArgs& a, const int* ends, int each, int t, F&& tiles) {
    int lo = 0, hi = (a.G + each - 1) / each - 1;            // the first entry whose end is past t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    int left = t - (lo ? __builtin_amdgcn_readfirstlane(ends[lo - 1]) : 0), grp = lo * each;
    bool bad = false;
    Group gr = group_of(a, grp, &bad);
    // no round unless an entry has several groups
    for (int p; each > 1 && grp + 1 < a.G && left >= (p = tiles(gr.rows)); gr = group_of(a, ++grp, &bad)) left -= p;
    return Piece{__builtin_amdgcn_readfirstlane(grp), gr, __builtin_amdgcn_readfirstlane(left)};
}

// silu(g) * u.  The reciprocal is the hardware's (one step in the last place), an exact division
// takes ten instructions for nothing that survives the output's rounding.
__device__ inline float silu_mul(float g, float u) {
#ifdef A2AV_DEVICE_CODE
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
#else
    return 0.0f;
#endif
}

// ---- what the matrix-unit kernels share ----------------------------------------------

enum Kind { kF32, kBf16, kBf16Mx4, kMx8, kMx8Mx4 };      // rows and weights

inline Kind kind_of(const ExpertArgs& a) {
    if (a.in_dtype == A2AV_F32) return kF32;
    if (a.in_dtype == A2AV_BF16) return a.w_dtype == A2AV_MX4 ? kBf16Mx4 : kBf16;
    return a.w_dtype == A2AV_MX4 ? kMx8Mx4 : kMx8;
}

__host__ __device__ constexpr bool weight_scaled(int kind) { return kind >= kBf16Mx4; }
__host__ __device__ constexpr bool rows_scaled(int kind) { return kind >= kMx8; }

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

[[maybe_unused]] constexpr uint32_t kOutside = 0x80000000u;   // an offset that every buffer check refuses: reads zero

#ifdef A2AV_DEVICE_CODE
__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// acc += w . x^T for 32 weight rows and 32 input rows: lane (l32, h) gives 32 bytes, w0 and w1, of
// weight row l32 and the same elements of input row l32, and holds columns 8q + 4h .. 8q + 4h + 3 of
// row l32 in acc[4q] .. acc[4q + 3].  64 bytes of each row: 16 float32, 32 bfloat16 or 64 8-bit
// elements, of which w0 and x0 are the 16-byte piece h, w1 and x1 the piece 2 + h (4-bit weights: w0
// alone, elements 32h .. 32h + 31); byte BYTE of ws and xs is the scale of elements 32h .. 32h + 31.
template <int KIND, int BYTE>
__device__ inline f32x16 multiply32(u32x4 w0, u32x4 w1, int ws, u32x4 x0, u32x4 x1, int xs, f32x16 acc) {
    if constexpr (KIND == kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w0[e]), __uint_as_float(x0[e]), acc, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w1[e]), __uint_as_float(x1[e]), acc, 0, 0, 0);
        return acc;
    } else if constexpr (KIND == kBf16 || KIND == kBf16Mx4) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w0), __builtin_bit_cast(bf16x8, x0), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w1), __builtin_bit_cast(bf16x8, x1), acc, 0, 0, 0);
    } else {
        const i32x8 w = {(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]};
        const i32x8 x = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, KIND == kMx8 ? 0 : 4, 0, BYTE, ws, BYTE, xs);
    }
}

// The LDS address of a shared array: what the loads below take.
__device__ inline uint32_t lds_address(const void* shared) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)shared);
}

// 16 bytes a lane, from each lane's offset straight to 1024 neighbouring bytes of LDS.  Written as
// an instruction without outputs: with the builtin the compiler waits for every such load before
// the next read of any LDS, so that nothing could be loaded while a step is multiplied.  Whoever
// reads the bytes calls wait_for_loads first, and a barrier where other wavefronts loaded them.
__device__ inline void load_to_lds(u32x4 buf, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    u32x4 b;                                             // scalar registers, whatever the compiler thinks of it
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_readfirstlane(buf[i]);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voffset), "s"(b), "s"(__builtin_amdgcn_readfirstlane(soffset))
                 : "memory");
}

// The same with 4 bytes a lane and 256 of LDS.
__device__ inline void load_word_to_lds(u32x4 buf, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    u32x4 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_readfirstlane(buf[i]);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voffset), "s"(b), "s"(__builtin_amdgcn_readfirstlane(soffset))
                 : "memory");
}

// Waits until at most N of this wavefront's loads are on their way (they arrive in order).
template <int N>
__device__ inline void wait_for_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// A barrier that waits for this wavefront's LDS reads and writes alone, not for its loads and stores.
__device__ inline void block_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// Sixteen scale bytes from p on, of which `valid` belong to the row (the others become zero: what
// they scale is zero, but a NaN byte would make it NaN) and `readable` may be read.  For rows of
// scales that are not whole words, which cannot be loaded straight to LDS.
__device__ inline u32x4 scale_bytes(const uint8_t* p, int valid, int64_t readable) {
    u32x4 v = {0, 0, 0, 0};
    if (valid <= 0) return v;
    if (readable >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < valid) v[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) v[w] &= valid >= 4 * w + 4 ? ~0u : valid <= 4 * w ? 0u : (1u << (8 * (valid - 4 * w))) - 1u;
    return v;
}

// Lanes of this wavefront hand each other values through LDS: what was written before it is read
// after it (LDS instructions of a wavefront are carried out in order).
__device__ inline void wave_sync() {
    asm volatile("" : : : "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" : : : "memory");
}

// The buffer of `bytes` bytes at p as the four words that the instruction takes.
__device__ inline u32x4 buffer_words(const uint8_t* p, uint32_t bytes) {
    const uint64_t at = (uint64_t)(uintptr_t)p;
    u32x4 w;
    w[0] = __builtin_amdgcn_readfirstlane((uint32_t)at);
    w[1] = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) & 0xFFFFu;
    w[2] = __builtin_amdgcn_readfirstlane(bytes);
    w[3] = 0x00020000u;
    return w;
}

// Eight E2M1 elements and the bits of their scale's power of two as eight bfloat16, exactly.
__device__ inline u32x4 widen_e2m1(uint32_t q, float scale) {
    u32x4 v;
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
    return v;
}

// acc += w . x^T for 16 weight rows and 16 input rows: lane (l16, g) gives 16 bytes of weight row
// l16 and of input row l16, the same elements of both, and holds columns 4g .. 4g + 3 of row l16.
template <int KIND>
__device__ inline f32x4 multiply16(u32x4 w, u32x4 x, f32x4 acc) {
    if constexpr (KIND == kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]), __uint_as_float(x[e]), acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    }
}

// The same for 128 elements in 8 (rows) and 8 or 4 bits (weights) with their scale bytes.  8-bit
// operands: lane group g gives elements 16g .. 16g + 15 (lo) and 64 + 16g .. 64 + 16g + 15 (hi) of
// its row; 4-bit ones: 32g .. 32g + 31 (lo); the scale byte of elements 32g .. 32g + 31 is lane
// group g's in both.
template <int KIND>
__device__ inline f32x4 multiply_scaled(u32x4 wlo, u32x4 whi, int ws, u32x4 xlo, u32x4 xhi, int xs, f32x4 acc) {
    const i32x8 w = {(int)wlo[0], (int)wlo[1], (int)wlo[2], (int)wlo[3], (int)whi[0], (int)whi[1], (int)whi[2], (int)whi[3]};
    const i32x8 x = {(int)xlo[0], (int)xlo[1], (int)xlo[2], (int)xlo[3], (int)xhi[0], (int)xhi[1], (int)xhi[2], (int)xhi[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, KIND == kMx8 ? 0 : 4, 0, 0, ws, 0, xs);
}
#endif

// Whether rows and weights are whole 16-byte pieces, which the stream and tile kernels need.
inline bool experts_whole_pieces(const ExpertArgs& a) {
    return a.in_row % 16 == 0 && a.w_row % 16 == 0 && (uintptr_t)a.in % 16 == 0 && (uintptr_t)a.weight % 16 == 0;
}

// Rows that are not (float32 and bfloat16 only: the others always are).
hipError_t launch_experts_general(const ExpertArgs& a, int num_cu, hipStream_t st);
// Groups of 1 .. a.few rows; of more as well, in pieces of a.few, where they would make tiles for
// fewer than half of the CUs (a.tile_least).
int few_rows(const ExpertArgs& a);
hipError_t launch_experts_few(const ExpertArgs& a, int num_cu, hipStream_t st);
// Groups of more rows.
hipError_t launch_experts_tile(const ExpertArgs& a, int num_cu, hipStream_t st);

}  // namespace a2av
