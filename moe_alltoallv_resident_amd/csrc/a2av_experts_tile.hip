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

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kTileN = 256;              // weight rows of a tile
constexpr int kMaxM = 256;               // input rows of the largest tile
constexpr int kRowStep = 128;            // bytes of an input row in a step
constexpr int kSuper = 8;                // row tiles that are walked together

__host__ __device__ constexpr int weight_step(int kind) {        // bytes of a weight row in a step
    return kind == kBf16Mx4 ? 32 : kind == kMx8Mx4 ? 64 : 128;
}
[[maybe_unused]] __host__ __device__ constexpr int step_elems(int kind) {   // elements of a step
    return kind == kF32 ? 32 : kind == kBf16 || kind == kBf16Mx4 ? 64 : 128; }

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

    const u32x4 xbuf = buffer_words(t.in, (uint32_t)(t.rows * a.in_row));
    const u32x4 wbuf = buffer_words(t.weight, (uint32_t)(a.N * a.w_row));
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
    auto load = [&](int s, Stage<KIND>* st) __attribute__((always_inline)) {
        const bool last = s == steps - 1;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            if (32 * MT / 8 % kWaves == 0 || i * kWaves + wave < 32 * MT / 8)
                load_to_lds(xbuf, st->x + (i * kWaves + wave) * 1024, last && !xt[i] ? kOutside : xo[i], s * kRowStep);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
            load_to_lds(wbuf, st->w + (i * kWaves + wave) * 1024, last && !wt[i] ? kOutside : wo[i], s * kWStep);
    };
    // Scale bytes, a 32-bit word of four a row: wavefronts 0 .. 3 load the weight's, 4 .. 7 the input
    // rows'.  Rows of scales that are not whole words (a width that is no multiple of 128) are
    // read byte by byte instead, without a step's head start.
    const int blocks = a.K / kMxGroup;
    const bool whole = blocks % 4 == 0 && (uintptr_t)t.scales % 4 == 0;
    const u32x4 sbuf = buffer_words(wave < 4 ? t.scales : t.in,
                                    wave < 4 ? (uint32_t)a.N * (uint32_t)blocks : (uint32_t)(t.rows * a.in_row));
    uint32_t so = kOutside;
    if constexpr (weight_scaled(KIND)) {
        if (wave < 4) {
            const int wr = weight_row(threadIdx.x);
            if (wr >= 0) so = (uint32_t)(wr * blocks);
        } else if (rows_scaled(KIND) && (int)threadIdx.x - kTileN < t.rows) {
            so = (uint32_t)((threadIdx.x - kTileN) * a.in_row + a.K);
        }
    }
    auto load_scales = [&](int s, Stage<KIND>* st) __attribute__((always_inline)) {
        if (!rows_scaled(KIND) && wave >= 4) return;
        uint32_t* to = wave < 4 ? st->ws : st->xs;
        const int first = s * step_elems(KIND) / kMxGroup / 4 * 4;      // the word's first block
        if (whole) {
            load_word_to_lds(sbuf, to + wave % 4 * kWave, so, first);
        } else {
            const uint8_t* p = wave < 4 ? t.scales : t.in;
            uint32_t v = 0;
            for (int i = 0; i < 4; ++i)
                if (so != kOutside && first + i < blocks) v |= (uint32_t)p[so + first + i] << (8 * i);
            to[wave % 4 * kWave + lane] = v;
        }
    };

    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // One step: the next one's loads begin, then this one's pieces are multiplied.
    auto step = [&](int s, Stage<KIND>* into, const Stage<KIND>* from) __attribute__((always_inline)) {
        const Stage<KIND>& st = *from;
        if (s + 1 < steps) {
            load(s + 1, into);
            if constexpr (weight_scaled(KIND)) load_scales(s + 1, into);
        }
        if constexpr (KIND == kF32 || KIND == kBf16 || KIND == kBf16Mx4) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                u32x4 x[MT], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = wn * 64 + j * 16 + l16;
                    if constexpr (KIND == kBf16Mx4) {
                        const uint32_t q = *(const uint32_t*)(st.w + r * kWStep + k * 16 + g * 4);
                        w[j] = widen_e2m1(q, __uint_as_float((uint32_t)((const uint8_t*)&st.ws[r])[s % 2 * 2 + k] << 23));
                    } else {
                        w[j] = *(const u32x4*)(st.w + place<128>(r, k * 4 + g));
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) x[i] = *(const u32x4*)(st.x + place<128>((wm * MT + i) * 16 + l16, k * 4 + g));
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = multiply16<KIND>(w[j], x[i], acc[i][j]);
            }
        } else {
            u32x4 lo[4], hi[4];
            int sw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wn * 64 + j * 16 + l16;
                lo[j] = *(const u32x4*)(st.w + place<kWStep>(r, g));
                if constexpr (KIND == kMx8) hi[j] = *(const u32x4*)(st.w + place<kWStep>(r, 4 + g));
                else hi[j] = u32x4{0, 0, 0, 0};
                sw[j] = ((const uint8_t*)&st.ws[r])[g];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = (wm * MT + i) * 16 + l16;
                const u32x4 xlo = *(const u32x4*)(st.x + place<128>(r, g)), xhi = *(const u32x4*)(st.x + place<128>(r, 4 + g));
                const int sx = ((const uint8_t*)&st.xs[r])[g];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = multiply_scaled<KIND>(lo[j], hi[j], sw[j], xlo, xhi, sx, acc[i][j]);
            }
        }
    };
    __syncthreads();                                        // the tile before has been read
    load(0, &stage[0]);
    if constexpr (weight_scaled(KIND)) load_scales(0, &stage[0]);
    for (int s = 0; s < steps; ++s) {
        wait_for_loads<0>();
        __syncthreads();                                    // step s is in LDS, step s - 1 has been read
        step(s, &stage[(s + 1) & 1], &stage[s & 1]);
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
    const int mt = count_tiles<kThreads>(a, ends, wave_sum, [](int rows) { return rows > kFewRows ? (rows + kMaxM - 1) / kMaxM : 0; });
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

}  // namespace

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
