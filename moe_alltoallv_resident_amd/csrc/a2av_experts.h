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

// Row tiles of every group, as ends[g] = tiles of groups 0 .. g; returns how many there are.
// Every thread of the block calls it; `tiles(rows)` says how many tiles a group has.
template <int THREADS, typename F>
__device__ int count_tiles(const ExpertArgs& a, int* ends, int* wave_sum, F&& tiles) {
    const int per = (a.G + THREADS - 1) / THREADS;
    const int g0 = threadIdx.x * per;
    int sum = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        if (g0 + i >= a.G) break;
        sum += tiles(group_of(a, g0 + i, &bad).rows);
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
        if (g0 + i >= a.G) break;
        ends[g0 + i] += before;
    }
    __syncthreads();
    return total;
}

// The group of row tile t: the first whose end is past t.
__device__ inline int find_group(const int* ends, int G, int t) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ inline float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// The general kernel, for whatever the others do not take.
hipError_t launch_experts_general(const ExpertArgs& a, int num_cu, hipStream_t st);
// The matrix-unit tiles.
bool experts_tile_takes(const ExpertArgs& a);
hipError_t launch_experts_tile(const ExpertArgs& a, int num_cu, hipStream_t st);

}  // namespace a2av
