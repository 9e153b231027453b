// Root-mean-square norm of token rows with the residual's addition, output in the rows'
// type and / or as 8-bit rows (declared in include/a2av.h).
//
// s = x + residual;  v = s / sqrt(mean(s^2) + eps) * weight.  About five operations an
// element against 4 to 14 bytes: bound by memory, so every array is read or written once.
// A row's threads keep the whole row in registers (float32) between the sum of squares and
// the outputs, and the 8-bit scales need no pass of their own: the 32 elements of a scale
// sit in neighbouring lanes of one wavefront.  65,536 bfloat16 rows of 5120 with the residual to
// 8-bit rows: 408 us, 5.8 TB/s read and written, as fast as a copy; one row: 3.8 us.
#include "../../include/a2av.h"
#include "a2av_mx.h"

#include <type_traits>

namespace a2av {
namespace {

constexpr int kWave = 64;
constexpr int kMaxHidden = 65536;

// N elements of the row type as one load or store.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T e[N];
};

__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(u16 v) { return bf16_to_f32(v); }
template <typename T>
__device__ inline T from_f32(float v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else return (u16)f32_to_bf16(v);
}

struct NormArgs {
    const void* x;
    const void* residual;
    const void* weight;
    void* residual_out;
    void* y;
    uint8_t* y8;
    int64_t rows;
    int32_t hidden;
    int32_t row8;      // bytes of an 8-bit row
    float eps;
};

// TPR threads hold a row, VPT vectors of VEC elements each (vector i of the row is thread
// i % TPR's).  Inactive vectors are zeros, which neither the sum nor a maximum sees.
template <typename T, int VEC, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rmsnorm_kernel(NormArgs a) {
    constexpr int kRows = (TPR < 256 ? 256 : TPR) / TPR;   // rows of a block
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (kRows > 1 && row >= a.rows) return;                // whole wavefronts: no barrier below when kRows > 1
    const int nvec = a.hidden / VEC;
    const P* x = (const P*)((const T*)a.x + row * a.hidden);
    const P* res = a.residual ? (const P*)((const T*)a.residual + row * a.hidden) : nullptr;
    float s[VPT][VEC];
    {
        P px[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = lane + v * TPR;
            px[v] = x[i < nvec ? i : 0];
        }
        if (res) {
            P pr[VPT];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int i = lane + v * TPR;
                pr[v] = res[i < nvec ? i : 0];
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[v][e] = to_f32(px[v].e[e]) + to_f32(pr[v].e[e]);
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[v][e] = to_f32(px[v].e[e]);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const bool on = lane + v * TPR < nvec;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[v][e] = on ? s[v][e] : 0.0f;
            sum = fmaf(s[v][e], s[v][e], sum);
        }
    }
#pragma unroll
    for (int m = kWave / 2; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if constexpr (TPR > kWave) {
        __shared__ float part[TPR / kWave];
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / kWave; ++w) sum += part[w];
    }
    const float inv = 1.0f / sqrtf(sum / (float)a.hidden + a.eps);
    if (a.residual_out) {
        P* out = (P*)((T*)a.residual_out + row * a.hidden);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = lane + v * TPR;
            P p;
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.e[e] = from_f32<T>(s[v][e]);
            if (i < nvec) out[i] = p;
        }
    }
    if (!a.y && !a.y8) return;
    const P* weight = (const P*)a.weight;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = lane + v * TPR;
        if (weight) {
            const P p = weight[i < nvec ? i : 0];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[v][e] = s[v][e] * inv * to_f32(p.e[e]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[v][e] *= inv;
        }
    }
    if (a.y) {
        P* out = (P*)((T*)a.y + row * a.hidden);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = lane + v * TPR;
            P p;
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.e[e] = from_f32<T>(s[v][e]);
            if (i < nvec) out[i] = p;
        }
    }
    if (a.y8) {
        uint8_t* out = a.y8 + row * a.row8;
        constexpr int kLanes = kMxGroup / VEC;             // neighbouring lanes that share a scale
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = lane + v * TPR;                  // hidden % 32 == 0: a group is all on or all off
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) m = max(m, abs_bits(s[v][e]));
#pragma unroll
            for (int k = 1; k < kLanes; k <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, k));
            const uint32_t sb = mx_scale_byte(m);
            const float f = mx_inverse(sb);
            const bool bad = sb == 255u;
            if (i < nvec) {
                if constexpr (VEC == 1) {
                    out[i] = (uint8_t)mx8_pack(s[v][0] * f, 0.0f, 0.0f, 0.0f, bad);
                } else {
                    uint32_t q[VEC / 4];
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        q[e / 4] = mx8_pack(s[v][e] * f, s[v][e + 1] * f, s[v][e + 2] * f, s[v][e + 3] * f, bad);
                    if constexpr (VEC == 8) ((u32x2*)out)[i] = u32x2{q[0], q[1]};
                    else ((uint32_t*)out)[i] = q[0];
                }
                if (i % kLanes == 0) out[a.hidden + i / kLanes] = (uint8_t)sb;
            }
        }
        const int used = a.hidden + a.hidden / kMxGroup;
        if (lane < a.row8 - used) out[used + lane] = 0;
    }
}

template <typename T, int VEC, int TPR, int VPT>
hipError_t launch(const NormArgs& a, hipStream_t st) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
    hipLaunchKernelGGL((rmsnorm_kernel<T, VEC, TPR, VPT>), dim3((unsigned)((a.rows + kRows - 1) / kRows)), dim3(kThreads),
                       0, st, a);
    return hipGetLastError();
}

template <typename T, int VEC, int TPR>
hipError_t launch_vpt(const NormArgs& a, hipStream_t st) {
    const int v = (a.hidden / VEC + TPR - 1) / TPR;
    if (v <= 1) return launch<T, VEC, TPR, 1>(a, st);
    if (v <= 2) return launch<T, VEC, TPR, 2>(a, st);
    if (v <= 4) return launch<T, VEC, TPR, 4>(a, st);
    if (v <= 8) return launch<T, VEC, TPR, 8>(a, st);
    if (v <= 16) return launch<T, VEC, TPR, 16>(a, st);
    if constexpr (TPR == 1024 && VEC < 8) {
        if (v <= 32) return launch<T, VEC, TPR, 32>(a, st);
        if (v <= 64) return launch<T, VEC, TPR, 64>(a, st);
    }
    return hipErrorInvalidValue;
}

template <typename T, int VEC>
hipError_t launch_vec(const NormArgs& a, hipStream_t st) {
    const int nvec = a.hidden / VEC;
    if (nvec <= 64 * 8) return launch_vpt<T, VEC, 64>(a, st);
    if (nvec <= 256 * 8) return launch_vpt<T, VEC, 256>(a, st);
    return launch_vpt<T, VEC, 1024>(a, st);
}

bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

}  // namespace
}  // namespace a2av

extern "C" {

int64_t a2av_row_bytes(int32_t dtype, int64_t n) {
    if (n < 1 || n > INT32_MAX) return -1;
    switch (dtype) {
        case A2AV_F32: return 4 * n;
        case A2AV_BF16: return 2 * n;
        case A2AV_MX8: return n % a2av::kMxGroup == 0 ? a2av::mx8_row_bytes(n) : -1;
        default: return -1;
    }
}

int a2av_rmsnorm(const void* x, const void* residual, const void* weight, void* residual_out, void* y, void* y8,
                 int64_t rows, int32_t hidden, int32_t dtype, float eps, void* stream) {
    using namespace a2av;
    if (dtype != A2AV_F32 && dtype != A2AV_BF16) return A2AV_ERR_INVALID;
    if (rows < 0 || rows > INT32_MAX || hidden < 1 || hidden > kMaxHidden || !(eps >= 0.0f)) return A2AV_ERR_INVALID;
    // arrays of no rows may be null
    if (rows > 0 && (!x || (!residual_out && !y && !y8) || (residual_out && !residual))) return A2AV_ERR_INVALID;
    if (y8 && (hidden % kMxGroup != 0 || !aligned16(y8))) return A2AV_ERR_INVALID;
    const size_t es = dtype == A2AV_F32 ? 4 : 2;
    const size_t bytes = es * (size_t)hidden;
    const void* rp[] = {x, residual, weight, residual_out, y};
    bool wide = bytes % 16 == 0;
    for (const void* p : rp) {
        if ((uintptr_t)p % es != 0) return A2AV_ERR_INVALID;
        wide = wide && aligned16(p);
    }
    if (rows == 0) return A2AV_OK;
    // Outputs: apart from each other and from the inputs, but for a row array written in place.
    struct Range {
        uintptr_t at, end;
    };
    auto range = [](const void* p, size_t n) { return Range{(uintptr_t)p, p ? (uintptr_t)p + n : (uintptr_t)p}; };
    auto meet = [](Range a, Range b) { return a.at < b.end && b.at < a.end; };
    const size_t all = bytes * (size_t)rows, all8 = (size_t)rows * (size_t)mx8_row_bytes(hidden);
    const Range ins[] = {range(x, all), range(residual, all), range(weight, bytes)};
    const Range outs[] = {range(residual_out, all), range(y, all), range(y8, all8)};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 3; ++i)
            if (meet(outs[o], ins[i]) && !(o < 2 && i < 2 && outs[o].at == ins[i].at)) return A2AV_ERR_INVALID;
        for (int p = 0; p < o; ++p)
            if (meet(outs[o], outs[p])) return A2AV_ERR_INVALID;
    }
    const NormArgs a{x, residual, weight, residual_out, y, (uint8_t*)y8, rows, hidden, (int32_t)mx8_row_bytes(hidden), eps};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (dtype == A2AV_F32) e = wide ? launch_vec<float, 4>(a, st) : launch_vec<float, 1>(a, st);
    else e = wide ? launch_vec<u16, 8>(a, st) : launch_vec<u16, 1>(a, st);
    return e == hipSuccess ? A2AV_OK : A2AV_ERR_HIP;
}

}  // extern "C"
