// The experts' products for experts with at most 16 rows: a decode step's case, bound by
// reading the weights, each of which meets 16 rows at most.
//
// A wavefront takes 16 or 32 weight rows and a part of their length, loads them straight into
// registers in the matrix instruction's layout (nothing is shared, so nothing goes through
// LDS) and multiplies them with all the rows at once; rows that are not there read zeros and
// cost no memory.  The parts of a weight row's length are added through LDS.
#include "a2av_experts.h"

namespace a2av {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kBlocksPerCu = 2;

// Elements of a unit, the step of the walk along a row: 16 bytes of a weight row for each lane
// (32 with 8-bit weights).
[[maybe_unused]] __host__ __device__ constexpr int unit_elems(int kind) { return kind == kF32 ? 16 : kind == kBf16 ? 32 : 128; }
// 16-byte pieces of a unit in a lane's registers.
[[maybe_unused]] __host__ __device__ constexpr int w_pieces(int kind) { return kind == kMx8 ? 2 : 1; }
[[maybe_unused]] __host__ __device__ constexpr int x_pieces(int kind) { return kind == kBf16Mx4 ? 4 : kind >= kMx8 ? 2 : 1; }
// Units loaded before the first of them is used.
[[maybe_unused]] __host__ __device__ constexpr int batch_units(int kind) { return kind == kF32 || kind == kBf16 ? 4 : kind == kMx8 ? 1 : 2; }

#ifdef A2AV_DEVICE_CODE
__device__ inline u32x4 load16(__amdgpu_buffer_rsrc_t buf, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, (int)off, 0, 0));
}

template <int KIND, int NT>
struct Batch {
    u32x4 w[batch_units(KIND)][NT][w_pieces(KIND)];
    u32x4 x[batch_units(KIND)][x_pieces(KIND)];
    uint8_t ws[batch_units(KIND)][NT], xs[batch_units(KIND)];
};
#endif

struct Job {
    const uint8_t* in;       // the group's first row
    const uint8_t* weight;   // its expert's
    const uint8_t* scales;
    uint8_t* out;
    int rows;                // 1 .. 16
    int col0;                // the tile's first output column
};

// NT: 16-row pieces of a wavefront.  A tile is kWaves / parts times 16 * NT weight rows.
// With SwiGLU the two pieces are 16 columns' gate and up rows, one piece 8 columns' both.
template <int KIND, int NT>
__device__ __forceinline__ void run_job(const ExpertArgs& a, const Job& t, int parts, f32x4* part) {
#ifdef A2AV_DEVICE_CODE
    constexpr int kUnit = unit_elems(KIND), kBatch = batch_units(KIND);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane % 16, g = lane / 16;
    const int wrow = wave / parts, wpart = wave % parts;     // this wavefront's weight rows and part
    const int units = (a.K + kUnit - 1) / kUnit;
    const int blocks = a.K / kMxGroup;

    const __amdgpu_buffer_rsrc_t xbuf = buffer_of(t.in, (uint32_t)(t.rows * a.in_row));
    const __amdgpu_buffer_rsrc_t wbuf = buffer_of(t.weight, (uint32_t)(a.N * a.w_row));
    __amdgpu_buffer_rsrc_t sbuf = wbuf;
    if constexpr (weight_scaled(KIND)) sbuf = buffer_of(t.scales, (uint32_t)a.N * (uint32_t)blocks);
    int wr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        int c, up = 0;
        if (!a.swiglu) {
            c = t.col0 + (wrow * NT + j) * 16 + l16;
        } else if (NT == 2) {
            c = t.col0 + wrow * 16 + l16;
            up = j;
        } else {
            c = t.col0 + wrow * 8 + l16 % 8;
            up = l16 / 8;
        }
        wr[j] = c < a.width ? c + up * a.width : -1;
    }
    // Lane (l16, g)'s elements of unit u, as byte offsets; outside a row they read zeros.
    auto load = [&](Batch<KIND, NT>& b, int at) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int unit = at + u;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int p = 0; p < w_pieces(KIND); ++p) {
                    const uint32_t o = (KIND == kMx8 ? unit * 128 + p * 64 : unit * 64) + g * 16;
                    const bool on = unit < units && o < (uint32_t)a.w_row && wr[j] >= 0;
                    b.w[u][j][p] = load16(wbuf, on ? (uint32_t)(wr[j] * a.w_row) + o : kOutside);
                }
#pragma unroll
            for (int p = 0; p < x_pieces(KIND); ++p) {
                uint32_t o, end;
                if constexpr (KIND == kBf16Mx4) {
                    o = unit * 256 + g * 64 + p * 16;        // the elements of the lane's 16 bytes of 4-bit weights
                    end = a.K * 2;
                } else if constexpr (KIND >= kMx8) {
                    o = unit * 128 + p * 64 + g * 16;
                    end = a.K;
                } else {
                    o = unit * 64 + g * 16;
                    end = (uint32_t)a.in_row;
                }
                const bool on = unit < units && o < end;        // rows past the last are past the buffer's end
                b.x[u][p] = load16(xbuf, on ? (uint32_t)(l16 * a.in_row) + o : kOutside);
            }
            if constexpr (weight_scaled(KIND)) {
                const int blk = unit * 4 + g;
                const bool on = unit < units && blk < blocks;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b.ws[u][j] = __builtin_amdgcn_raw_buffer_load_b8(sbuf, on && wr[j] >= 0 ? (int)((uint32_t)(wr[j] * blocks) + blk) : (int)kOutside,
                                                                     0, 0);
                if constexpr (rows_scaled(KIND))
                    b.xs[u] = __builtin_amdgcn_raw_buffer_load_b8(xbuf, on ? (int)(l16 * a.in_row + a.K + blk) : (int)kOutside, 0, 0);
            }
        }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0, 0, 0, 0};
    auto use = [&](const Batch<KIND, NT>& b) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (KIND == kF32 || KIND == kBf16) {
                    acc[j] = multiply16<KIND>(b.w[u][j][0], b.x[u][0], acc[j]);
                } else if constexpr (KIND == kBf16Mx4) {
                    const float f = __uint_as_float((uint32_t)b.ws[u][j] << 23);
#pragma unroll
                    for (int p = 0; p < 4; ++p) acc[j] = multiply16<KIND>(widen_e2m1(b.w[u][j][0][p], f), b.x[u][p], acc[j]);
                } else {
                    const u32x4 none = {0, 0, 0, 0};
                    acc[j] = multiply_scaled<KIND>(b.w[u][j][0], KIND == kMx8 ? b.w[u][j][w_pieces(KIND) - 1] : none, b.ws[u][j],
                                                   b.x[u][0], b.x[u][x_pieces(KIND) - 1], b.xs[u], acc[j]);
                }
            }
    };
    // The parts take batches in turn, so that together they sweep along their rows.
    {
        const int step = parts * kBatch;
        Batch<KIND, NT> b0, b1;
        load(b0, wpart * kBatch);
        for (int at = wpart * kBatch; at < units; at += 2 * step) {
            load(b1, at + step);
            use(b0);
            load(b0, at + 2 * step);
            use(b1);
        }
    }

    // part[wave][j][lane]: the parts of a row are neighbours
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(wave * NT + j) * kWave + lane] = acc[j];
    __syncthreads();
    const int groups = kWaves / parts;
    const int cols = groups * 16 * NT / (a.swiglu ? 2 : 1);
    const int quads = cols / 4;                              // four neighbouring columns: one lane's result
    auto sum = [&](int row, int j, int ln) {
        f32x4 v = part[(row * parts * NT + j) * kWave + ln];
        for (int p = 1; p < parts; ++p) v += part[((row * parts + p) * NT + j) * kWave + ln];
        return v;
    };
    for (int i = threadIdx.x; i < 16 * quads; i += kThreads) {
        const int m = i / quads, q = i % quads;
        f32x4 v;
        if (!a.swiglu) {
            v = sum(q / 4 / NT, q / 4 % NT, m + 16 * (q % 4));
        } else {
            f32x4 up;
            if (NT == 2) {
                v = sum(q / 4, 0, m + 16 * (q % 4));
                up = sum(q / 4, NT - 1, m + 16 * (q % 4));
            } else {
                v = sum(q / 2, 0, m + 16 * (q % 2));
                up = sum(q / 2, 0, m + 16 * (q % 2 + 2));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], up[e]);
        }
        const int c = t.col0 + 4 * q;
        const bool on = m < t.rows && c < a.width;
        uint8_t* out = t.out + m * a.out_row;
        if (rows_scaled(KIND) && a.out_dtype == A2AV_MX8) {
            // a scale's 32 columns are eight neighbouring threads' (the tile has a multiple of 32)
            uint32_t mx = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = max(mx, abs_bits(v[e]));
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, s));
            const uint32_t sb = mx_scale_byte(mx);
            const float f = mx_inverse(sb);
            if (on) {
                *(uint32_t*)(out + c) = mx8_pack(v[0] * f, v[1] * f, v[2] * f, v[3] * f, sb == 255u);
                if (c % kMxGroup == 0) out[a.width + c / kMxGroup] = (uint8_t)sb;
                if (c + 4 == a.width)
                    for (int b = a.width + a.width / kMxGroup; b < a.out_row; ++b) out[b] = 0;
            }
        } else if (on) {
            if constexpr (KIND == kF32) {
                float* p = (float*)out + c;
                if (a.width % 4 == 0 && (uintptr_t)a.out % 16 == 0) *(f32x4*)p = v;
                else
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.width) p[e] = v[e];
            } else {
                u16* p = (u16*)out + c;
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = f32_to_bf16(v[e]);
                if (a.width % 4 == 0 && (uintptr_t)a.out % 8 == 0) *(u32x2*)p = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
                else
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.width) p[e] = (u16)b[e];
            }
        }
    }
    __syncthreads();                                         // `part` is free again
#endif
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 2 * kBlocksPerCu) expert_few_kernel(ExpertArgs a) {
    __shared__ int ends[kMaxExperts];
    __shared__ int wave_sum[kWaves];
    __shared__ f32x4 part[kWaves * 2 * kWave];
    const int n = count_tiles<kThreads>(a, ends, wave_sum, [](int rows) { return rows > 0 && rows <= kFewRows ? 1 : 0; });
    if (n == 0) return;
    const int64_t pieces = (int64_t)n * ((a.N + 15) / 16);   // of 16 weight rows
    const int batches = (a.K + unit_elems(KIND) * batch_units(KIND) - 1) / (unit_elems(KIND) * batch_units(KIND));
    const bool two = pieces >= 4 * (int64_t)gridDim.x;
    const int wide = two ? 2 : 1;
    const int most = a.out_dtype != A2AV_MX8 ? 8 : a.swiglu ? 2 * wide : 4 * wide;   // a tile of 8-bit rows has 32 columns at least
    int parts = 1;
    while (parts < most && parts < batches) parts *= 2;
    const int cols = kWaves / parts * 16 * wide / (a.swiglu ? 2 : 1);
    const int nt = (a.width + cols - 1) / cols;
    const int64_t total = (int64_t)n * nt;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
        const int i = __builtin_amdgcn_readfirstlane((int)(t / nt)), tn = __builtin_amdgcn_readfirstlane((int)(t % nt));
        const int grp = __builtin_amdgcn_readfirstlane(find_group(ends, a.G, i));
        bool bad = false;
        const Group gr = group_of(a, grp, &bad);
        const int64_t w0 = (int64_t)grp * a.N;
        const Job job{a.in + gr.row * a.in_row, a.weight + w0 * a.w_row, a.scales + w0 * (a.K / kMxGroup),
                      a.out + gr.row * a.out_row, __builtin_amdgcn_readfirstlane(gr.rows), tn * cols};
        if (two) run_job<KIND, 2>(a, job, parts, part);
        else run_job<KIND, 1>(a, job, parts, part);
    }
}

template <int KIND>
hipError_t launch(const ExpertArgs& a, int num_cu, hipStream_t st) {
    hipLaunchKernelGGL((expert_few_kernel<KIND>), dim3((unsigned)(num_cu * kBlocksPerCu)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_few(const ExpertArgs& a, int num_cu, hipStream_t st) {
    switch (kind_of(a)) {
        case kF32: return launch<kF32>(a, num_cu, st);
        case kBf16: return launch<kBf16>(a, num_cu, st);
        case kBf16Mx4: return launch<kBf16Mx4>(a, num_cu, st);
        case kMx8: return launch<kMx8>(a, num_cu, st);
        default: return launch<kMx8Mx4>(a, num_cu, st);
    }
}

}  // namespace a2av
