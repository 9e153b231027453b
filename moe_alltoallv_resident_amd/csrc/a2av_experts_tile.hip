// The experts' products on the matrix units.
//
// A tile is up to 256 rows of one expert by 256 rows of its weight.  Both are staged through
// LDS in steps of 128 bytes of a row (64 bfloat16, 128 e4m3, 32 float32 elements; 4-bit weights
// take 32 or 64 bytes for the same elements), loaded straight from memory into LDS while the
// step before is multiplied.  Eight wavefronts, two along the rows and four along the weight,
// hold 128 x 64 results each in registers.  The weight is the matrix instruction's first
// operand, so a lane ends up with four neighbouring columns of one output row.
//
// Matrix instructions: 16x16x32 (bfloat16), 16x16x4 (float32), 16x16x128 with a scale for every
// 32 elements (e4m3 and E2M1 as they are stored).  4-bit weights with bfloat16 rows are widened
// in registers, exactly: an E2M1 element times a power of two is a bfloat16.
#include "a2av_experts.h"

namespace a2av {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Kind { kF32, kBf16, kBf16Mx4, kMx8, kMx8Mx4 };

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kTileN = 256;              // weight rows of a tile
constexpr int kMaxM = 256;               // input rows of the largest tile
constexpr int kRowStep = 128;            // bytes of an input row in a step
constexpr int kSuper = 8;                // row tiles that are walked together
[[maybe_unused]] constexpr uint32_t kOutside = 0x80000000u;   // an offset that every buffer check refuses: reads zero

__host__ __device__ constexpr int weight_step(int kind) {        // bytes of a weight row in a step
    return kind == kBf16Mx4 ? 32 : kind == kMx8Mx4 ? 64 : 128;
}
[[maybe_unused]] __host__ __device__ constexpr int step_elems(int kind) {   // elements of a step
    return kind == kF32 ? 32 : kind == kBf16 || kind == kBf16Mx4 ? 64 : 128; }
__host__ __device__ constexpr bool weight_scaled(int kind) { return kind >= kBf16Mx4; }
__host__ __device__ constexpr bool rows_scaled(int kind) { return kind >= kMx8; }

template <int KIND>
struct Stage {
    alignas(1024) uint8_t x[kMaxM * kRowStep];
    alignas(1024) uint8_t w[kTileN * weight_step(KIND)];
    uint32_t xs[rows_scaled(KIND) ? kMaxM : 1];         // a step's scale bytes of each row
    uint32_t ws[weight_scaled(KIND) ? kTileN : 1];
};

// Where 16-byte piece c of row r stands in its LDS row: eight neighbouring rows' same pieces, read
// by eight neighbouring lanes, fall into different banks.
template <int STEP>
__device__ inline int place(int r, int c) {
    if constexpr (STEP == 128) return r * 128 + ((c ^ (r & 7)) << 4);
    else if constexpr (STEP == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else return r * 32 + (c << 4);
}

// The piece that belongs at place p of row r.
template <int STEP>
__device__ inline int piece_at(int r, int p) {
    if constexpr (STEP == 128) return p ^ (r & 7);
    else if constexpr (STEP == 64) return p ^ ((r >> 1) & 3);
    else return p;
}

#ifdef A2AV_DEVICE_CODE
__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}

// 16 bytes a lane, from each lane's offset to 1024 neighbouring bytes of LDS.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t buf, uint8_t* lds, uint32_t voffset, uint32_t soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (__attribute__((address_space(3))) void*)lds, 16, (int)voffset, (int)soffset,
                                             0, 0);
}
#endif

// Up to four scale bytes from `at` on, of which the first `n` are the row's.
[[maybe_unused]] __device__ inline uint32_t load_scales(const uint8_t* at, int n, bool whole) {
    if (whole) return *(const uint32_t*)at;
    uint32_t v = 0;
    for (int i = 0; i < 4; ++i)
        if (i < n) v |= (uint32_t)at[i] << (8 * i);
    return v;
}

// Everything of a tile that does not depend on its height.
struct Tile {
    const uint8_t* in;       // its first row
    const uint8_t* weight;   // its expert's
    const uint8_t* scales;
    uint8_t* out;
    int rows;                // 1 .. 256
    int col0;                // its first output column
};

// MT: 16-row pieces of a wavefront; the tile has 32 * MT rows.
template <int KIND, int MT>
__device__ __forceinline__ void run_tile(const ExpertArgs& a, const Tile& t, Stage<KIND>* stage) {
#ifdef A2AV_DEVICE_CODE
    constexpr int kWStep = weight_step(KIND), kWPieces = kWStep / 16, kWRows = kWave / kWPieces;
    constexpr int kXLoads = (32 * MT / 8 + kWaves - 1) / kWaves, kWLoads = kTileN / kWRows / kWaves;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4, l16 = lane % 16, g = lane / 16;
    const int steps = (a.K + step_elems(KIND) - 1) / step_elems(KIND);
    const int x_bytes = KIND == kF32 ? a.K * 4 : KIND == kBf16 || KIND == kBf16Mx4 ? a.K * 2 : a.K;
    const int x_tail = x_bytes - (steps - 1) * kRowStep, w_tail = (int)a.w_row - (steps - 1) * kWStep;

    const __amdgpu_buffer_rsrc_t xbuf = buffer_of(t.in, (uint32_t)(t.rows * a.in_row));
    const __amdgpu_buffer_rsrc_t wbuf = buffer_of(t.weight, (uint32_t)(a.N * a.w_row));
    // Byte offsets of this lane's pieces; rows past the tile's, columns past the last one and, in
    // the last step, pieces past the row's end read zeros.
    uint32_t xo[kXLoads], wo[kWLoads];
    bool xt[kXLoads], wt[kWLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
        const int r = (i * kWaves + wave) * 8 + lane / 8, c = piece_at<128>(r, lane % 8);
        xo[i] = (uint32_t)(r * a.in_row + c * 16);          // past the last row: past the buffer's end
        xt[i] = c * 16 < x_tail;
    }
    // weight row of tile row r: with SwiGLU 16 gate rows and the 16 up rows of the same columns in turn
    auto weight_row = [&](int r) {
        if (!a.swiglu) return t.col0 + r < a.width ? t.col0 + r : -1;
        const int c = t.col0 + (r / 32) * 16 + r % 16;
        return c < a.width ? c + (r / 16 % 2 ? a.width : 0) : -1;
    };
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
        const int r = (i * kWaves + wave) * kWRows + lane / kWPieces, c = piece_at<kWStep>(r, lane % kWPieces);
        const int wr = weight_row(r);
        wo[i] = wr < 0 ? kOutside : (uint32_t)(wr * a.w_row + c * 16);
        wt[i] = c * 16 < w_tail;
    }
    auto load = [&](int s) {
        Stage<KIND>& st = stage[s & 1];
        const bool last = s == steps - 1;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            if (32 * MT / 8 % kWaves == 0 || i * kWaves + wave < 32 * MT / 8)
                load_to_lds(xbuf, st.x + (i * kWaves + wave) * 1024, last && !xt[i] ? kOutside : xo[i], s * kRowStep);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
            load_to_lds(wbuf, st.w + (i * kWaves + wave) * 1024, last && !wt[i] ? kOutside : wo[i], s * kWStep);
    };
    // Scale bytes go through a register: thread i holds weight row i's, thread 256 + i input row i's.
    constexpr int kSteps = step_elems(KIND) / kMxGroup;     // scale bytes of a step
    const int blocks = a.K / kMxGroup;
    const uint8_t* sp = nullptr;
    bool whole = false;
    if constexpr (weight_scaled(KIND)) {
        if (threadIdx.x < kTileN) {
            const int wr = weight_row(threadIdx.x);
            if (wr >= 0) sp = t.scales + (int64_t)wr * blocks;
            whole = kSteps == 4 && blocks % 4 == 0 && (uintptr_t)t.scales % 4 == 0;
        } else if (rows_scaled(KIND)) {
            const int r = threadIdx.x - kTileN;
            if (r < t.rows) sp = t.in + (int64_t)r * a.in_row + a.K;
            whole = blocks % 4 == 0;
        }
    }
    auto scales_of = [&](int s) -> uint32_t {
        return sp ? load_scales(sp + s * kSteps, min(kSteps, blocks - s * kSteps), whole) : 0u;
    };
    auto put_scales = [&](int s, uint32_t v) {
        Stage<KIND>& st = stage[s & 1];
        if (threadIdx.x < kTileN) st.ws[threadIdx.x] = v;
        else if (rows_scaled(KIND)) st.xs[threadIdx.x - kTileN] = v;
    };

    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    __syncthreads();                                        // the tile before has been read
    load(0);
    if constexpr (weight_scaled(KIND)) put_scales(0, scales_of(0));
    for (int s = 0; s < steps; ++s) {
        __syncthreads();                                    // step s is in LDS, step s - 1 has been read
        uint32_t next = 0;
        if (s + 1 < steps) {
            load(s + 1);
            if constexpr (weight_scaled(KIND)) next = scales_of(s + 1);
        }
        const Stage<KIND>& st = stage[s & 1];
        if constexpr (KIND == kF32 || KIND == kBf16 || KIND == kBf16Mx4) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                u32x4 x[MT], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = wn * 64 + j * 16 + l16;
                    if constexpr (KIND == kBf16Mx4) {
                        const uint32_t q = *(const uint32_t*)(st.w + r * kWStep + k * 16 + g * 4);
                        const float f = __uint_as_float((st.ws[r] >> (8 * k) & 255u) << 23);
                        w[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 0));
                        w[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 1));
                        w[j][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 2));
                        w[j][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 3));
                    } else {
                        w[j] = *(const u32x4*)(st.w + place<128>(r, k * 4 + g));
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) x[i] = *(const u32x4*)(st.x + place<128>((wm * MT + i) * 16 + l16, k * 4 + g));
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (KIND == kF32) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[j][e]), __uint_as_float(x[i][e]),
                                                                                 acc[i][j], 0, 0, 0);
                        } else {
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j]),
                                                                                __builtin_bit_cast(bf16x8, x[i]), acc[i][j], 0, 0, 0);
                        }
                    }
            }
        } else {
            // The 8-bit operand of 128 elements: lane group g holds elements 16g .. 16g + 15 and
            // 64 + 16g .. 64 + 16g + 15 of its row; the 4-bit one 32g .. 32g + 31; the scale byte of
            // elements 32g .. 32g + 31 is lane group g's in both.
            i32x8 w[4];
            int sw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wn * 64 + j * 16 + l16;
                u32x4 lo, hi = {0, 0, 0, 0};
                if constexpr (KIND == kMx8) {
                    lo = *(const u32x4*)(st.w + place<128>(r, g));
                    hi = *(const u32x4*)(st.w + place<128>(r, 4 + g));
                } else {
                    lo = *(const u32x4*)(st.w + place<64>(r, g));
                }
                w[j] = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
                sw[j] = ((const uint8_t*)&st.ws[r])[g];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = (wm * MT + i) * 16 + l16;
                const u32x4 lo = *(const u32x4*)(st.x + place<128>(r, g)), hi = *(const u32x4*)(st.x + place<128>(r, 4 + g));
                const i32x8 x = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
                const int sx = ((const uint8_t*)&st.xs[r])[g];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j], x, acc[i][j], KIND == kMx8 ? 0 : 4, 0, 0,
                                                                                 sw[j], 0, sx);
            }
        }
        if constexpr (weight_scaled(KIND))
            if (s + 1 < steps) put_scales(s + 1, next);
    }

    // Results: lane (l16, g) has columns 4g .. 4g + 3 of a 16 x 16 piece, of input row l16.
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = (wm * MT + i) * 16 + l16;
        const bool on = r < t.rows;
        uint8_t* out = t.out + r * a.out_row;
        f32x4 v[4];
        int n = 4;                                          // 16-column pieces
        int col = t.col0 + wn * 64;
        if (a.swiglu) {
            n = 2;
            col = t.col0 + wn * 32;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[p][e] = silu_mul(acc[i][2 * p][e], acc[i][2 * p + 1][e]);
            v[2] = v[3] = f32x4{0, 0, 0, 0};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[i][j];
        }
        if (rows_scaled(KIND) && a.out_dtype == A2AV_MX8) {
            // 32 columns: two pieces of the four lanes that share a row
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * h >= n) break;
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max(m, max(abs_bits(v[2 * h][e]), abs_bits(v[2 * h + 1][e])));
                m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32));
                const uint32_t sb = mx_scale_byte(m);
                const float f = mx_inverse(sb);
                const int c = col + 32 * h;                 // the width is a multiple of 32
                if (on && c < a.width) {
                    *(uint32_t*)(out + c + 4 * g) = mx8_pack(v[2 * h][0] * f, v[2 * h][1] * f, v[2 * h][2] * f, v[2 * h][3] * f,
                                                             sb == 255u);
                    *(uint32_t*)(out + c + 16 + 4 * g) = mx8_pack(v[2 * h + 1][0] * f, v[2 * h + 1][1] * f, v[2 * h + 1][2] * f,
                                                                  v[2 * h + 1][3] * f, sb == 255u);
                    if (g == 0) out[a.width + c / kMxGroup] = (uint8_t)sb;
                    const int used = a.width + a.width / kMxGroup;
                    if (c + 32 == a.width)
                        for (int b = used + g; b < a.out_row; b += 4) out[b] = 0;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = col + 16 * j + 4 * g;
                if (j >= n || !on || c >= a.width) continue;
                if constexpr (KIND == kF32) {
                    float* p = (float*)out + c;
                    if (a.width % 4 == 0 && (uintptr_t)a.out % 16 == 0) *(f32x4*)p = v[j];
                    else
                        for (int e = 0; e < 4; ++e)
                            if (c + e < a.width) p[e] = v[j][e];
                } else {
                    u16* p = (u16*)out + c;
                    uint32_t b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = f32_to_bf16(v[j][e]);
                    if (a.width % 4 == 0 && (uintptr_t)a.out % 8 == 0) *(u32x2*)p = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
                    else
                        for (int e = 0; e < 4; ++e)
                            if (c + e < a.width) p[e] = (u16)b[e];
                }
            }
        }
    }
#endif
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) expert_tile_kernel(ExpertArgs a) {
    __shared__ Stage<KIND> stage[2];
    __shared__ int ends[kMaxExperts];
    __shared__ int wave_sum[kWaves];
    const int mt = count_tiles<kThreads>(a, ends, wave_sum, [](int rows) { return (rows + kMaxM - 1) / kMaxM; });
    const int cols = a.swiglu ? kTileN / 2 : kTileN;
    const int nt = (a.width + cols - 1) / cols;
    const int64_t total = (int64_t)mt * nt;
    // Blocks go to the eight dies in turn.  Of every gridDim.x tiles a die gets one run of
    // neighbours, whose rows and weights its L2 then holds once.
    const int run = gridDim.x / 8;
    const int pos = (blockIdx.x % 8) * run + blockIdx.x / 8;
    for (int64_t t = pos; t < total; t += gridDim.x) {
        const int64_t sup = t / ((int64_t)kSuper * nt);
        const int in_sup = (int)(t - sup * kSuper * nt), high = min(kSuper, mt - (int)sup * kSuper);
        const int tm = __builtin_amdgcn_readfirstlane((int)sup * kSuper + in_sup % high);
        const int tn = __builtin_amdgcn_readfirstlane(in_sup / high);
        const int grp = __builtin_amdgcn_readfirstlane(find_group(ends, a.G, tm));
        bool bad = false;
        const Group gr = group_of(a, grp, &bad);
        const int m0 = (tm - (grp ? ends[grp - 1] : 0)) * kMaxM;
        const int64_t row = gr.row + m0;
        const int64_t w0 = (int64_t)grp * a.N;
        const Tile tile{a.in + row * a.in_row, a.weight + w0 * a.w_row, a.scales + w0 * (a.K / kMxGroup), a.out + row * a.out_row,
                        __builtin_amdgcn_readfirstlane(min(kMaxM, gr.rows - m0)), tn * cols};
        if (tile.rows > 128) run_tile<KIND, 8>(a, tile, stage);
        else if (tile.rows > 64) run_tile<KIND, 4>(a, tile, stage);
        else if (tile.rows > 32) run_tile<KIND, 2>(a, tile, stage);
        else run_tile<KIND, 1>(a, tile, stage);
    }
}

template <int KIND>
hipError_t launch(const ExpertArgs& a, int num_cu, hipStream_t st) {
    // a multiple of the eight dies; one block a CU (its LDS allows no second)
    hipLaunchKernelGGL((expert_tile_kernel<KIND>), dim3((unsigned)std::max(8, num_cu / 8 * 8)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

Kind kind_of(const ExpertArgs& a) {
    if (a.in_dtype == A2AV_F32) return kF32;
    if (a.in_dtype == A2AV_BF16) return a.w_dtype == A2AV_MX4 ? kBf16Mx4 : kBf16;
    return a.w_dtype == A2AV_MX4 ? kMx8Mx4 : kMx8;
}

}  // namespace

// Rows and weights in whole 16-byte pieces, an expert's weight within a 32-bit offset.
bool experts_tile_takes(const ExpertArgs& a) {
    return a.in_row % 16 == 0 && a.w_row % 16 == 0 && (uintptr_t)a.in % 16 == 0 && (uintptr_t)a.weight % 16 == 0 &&
           a.N * a.w_row <= INT32_MAX && kMaxM * a.in_row <= INT32_MAX;
}

hipError_t launch_experts_tile(const ExpertArgs& a, int num_cu, hipStream_t st) {
    switch (kind_of(a)) {
        case kF32: return launch<kF32>(a, num_cu, st);
        case kBf16: return launch<kBf16>(a, num_cu, st);
        case kBf16Mx4: return launch<kBf16Mx4>(a, num_cu, st);
        case kMx8: return launch<kMx8>(a, num_cu, st);
        default: return launch<kMx8Mx4>(a, num_cu, st);
    }
}

}  // namespace a2av
