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

[[maybe_unused]] constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kTileN = kTileRows;        // weight rows of a tile
constexpr int kMaxM = kTileRows;         // input rows of the largest tile
constexpr int kRowStep = 128;            // bytes of an input row in a step
[[maybe_unused]] constexpr int kSuper = 8;                // row tiles that are walked together

[[maybe_unused]] __host__ __device__ constexpr int weight_step(int kind) {        // bytes of a weight row in a step
    return kind == kBf16Mx4 ? 32 : kind == kMx8Mx4 ? 64 : 128;
}
[[maybe_unused]] __host__ __device__ constexpr int step_elems(int kind) {   // elements of a step
    return kind == kF32 ? 32 : kind == kBf16 || kind == kBf16Mx4 ? 64 : 128; }

template <int KIND>
struct Stage {
    alignas(1024) uint8_t x[kMaxM * kRowStep];
    alignas(1024) uint8_t w[kTileN * weight_step(KIND)];
};

// Scale bytes of sixteen blocks of 32 elements for each weight row and, behind them, each input row.
constexpr int kQuad = 16;
struct Scales {
    alignas(1024) uint8_t of[kTileN + kMaxM][kQuad];
};

// A wavefront's place to put output rows together, in the second half of the scales: that is free
// while the next tile's first steps are loaded.
[[maybe_unused]] constexpr int kOutStage = sizeof(Scales) / kWaves;
static_assert(kOutStage == 1024, "eight rows of 128 bytes");

template <int KIND>
struct Shared {
    Stage<KIND> stage[2];
    Scales scales[2];
    int ends[kMaxExperts];
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

// Row pieces of 16 for each of the two wavefronts along the rows: a tile has 32 * 8, 4, 2 or 1 rows.
[[maybe_unused]] __device__ inline int height_of(int rows) { return rows > 128 ? 8 : rows > 64 ? 4 : rows > 32 ? 2 : 1; }

struct Tile {
    const uint8_t* in;       // its first row
    const uint8_t* weight;   // its expert's
    const uint8_t* scales;
    uint8_t* out;
    int rows;                // 1 .. 256; 0: there is no tile
    int col0;                // its first output column
};

#ifdef A2AV_DEVICE_CODE
// Brings a tile's steps to LDS.  A lane's pieces keep their place in a row from step to step.
template <int KIND>
struct Loader {
    static constexpr int kWStep = weight_step(KIND), kWPieces = kWStep / 16, kWRows = kWave / kWPieces;
    static constexpr int kWLoads = kTileN / kWRows / kWaves;     // of a wavefront for a step
    static constexpr int kXLoads = kMaxM / 8 / kWaves;           // load i: the tile's rows 64 i .. 64 i + 63
    static constexpr int kBlocks = step_elems(KIND) / kMxGroup;  // scale bytes of a step

    Shared<KIND>& sh;
    int lane, wave, steps, blocks;
    u32x4 xbuf, wbuf, sbuf;
    uint32_t xo[kXLoads], wo[kWLoads], so;
    bool x_over, w_over;     // the lane's pieces are past the row's end in the last step
    const uint8_t* sp;       // scales that are read byte by byte

    // weight row of tile row r: with SwiGLU 16 gate rows and the 16 up rows of the same columns in turn
    static __device__ int weight_row(const ExpertArgs& a, const Tile& t, int r) {
        if (!a.swiglu) return t.col0 + r < a.width ? t.col0 + r : -1;
        const int c = t.col0 + (r / 32) * 16 + r % 16;
        return c < a.width ? c + (r / 16 % 2 ? a.width : 0) : -1;
    }

    __device__ __forceinline__ Loader(const ExpertArgs& a, Shared<KIND>& s) : sh(s) {
        lane = threadIdx.x % kWave;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        steps = (a.K + step_elems(KIND) - 1) / step_elems(KIND);
        blocks = a.K / kMxGroup;
    }

    // Byte offsets of this lane's pieces; rows past the tile's and columns past the last one read
    // zeros, and so do in the last step pieces past the row's end.
    __device__ __forceinline__ void begin(const ExpertArgs& a, const Tile& t) {
        xbuf = buffer_words(t.in, (uint32_t)(t.rows * a.in_row));
        wbuf = buffer_words(t.weight, (uint32_t)(a.N * a.w_row));
        const int x_bytes = KIND == kF32 ? a.K * 4 : KIND == kBf16 || KIND == kBf16Mx4 ? a.K * 2 : a.K;
        // row 8 n + lane / 8: its swizzle, and so its piece, is the same for every n
        const int xc = piece_at<128>(lane / 8, lane % 8) * 16;
        x_over = xc >= x_bytes - (steps - 1) * kRowStep;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) xo[i] = (uint32_t)(((i * kWaves + wave) * 8 + lane / 8) * a.in_row + xc);
        const int wc = piece_at<kWStep>(lane / kWPieces, lane % kWPieces) * 16;
        w_over = wc >= (int)a.w_row - (steps - 1) * kWStep;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
            const int wr = weight_row(a, t, (i * kWaves + wave) * kWRows + lane / kWPieces);
            wo[i] = wr < 0 ? kOutside : (uint32_t)(wr * a.w_row + wc);
        }
        if constexpr (weight_scaled(KIND)) {
            // wavefronts 0 .. 3 load the weight rows' scales, 4 .. 7 the input rows'
            sbuf = buffer_words(wave < 4 ? t.scales : t.in,
                                wave < 4 ? (uint32_t)a.N * (uint32_t)blocks : (uint32_t)(t.rows * a.in_row));
            sp = wave < 4 ? t.scales : t.in;
            so = kOutside;
            if (wave < 4) {
                const int wr = weight_row(a, t, threadIdx.x);
                if (wr >= 0) so = (uint32_t)(wr * blocks);
            } else if (rows_scaled(KIND) && (int)threadIdx.x - kTileN < t.rows) {
                so = (uint32_t)((threadIdx.x - kTileN) * a.in_row + a.K);
            }
        }
    }
    // Loads past the last step read zeros too: the counts that the waits go by stay the same.
    __device__ __forceinline__ void rows(int s, int i) {
        const bool on = s < steps - 1 || (s == steps - 1 && !x_over);
        load_to_lds(xbuf, sh.stage[s & 1].x + (i * kWaves + wave) * 1024, on ? xo[i] : kOutside, s * kRowStep);
    }
    __device__ __forceinline__ void weights(int s) {
        const bool on = s < steps - 1 || (s == steps - 1 && !w_over);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
            load_to_lds(wbuf, sh.stage[s & 1].w + (i * kWaves + wave) * 1024, on ? wo[i] : kOutside, s * kWStep);
    }
    // Scale bytes, sixteen blocks at a time.  Rows of scales that are not whole words (a width that
    // is no multiple of 128) are read byte by byte.
    __device__ __forceinline__ void scales(const ExpertArgs& a, int quad) {
        if (!weight_scaled(KIND) || (wave >= 4 && !rows_scaled(KIND)) || quad * kQuad >= blocks) return;
        uint8_t* to = sh.scales[quad & 1].of[wave * kWave];
        if (blocks % 4 == 0 && (uintptr_t)a.scales % 4 == 0) {
            load_to_lds(sbuf, to, so, quad * kQuad);
        } else {
#pragma unroll 1
            for (int w = 0; w < kQuad; w += 4) {
                uint32_t v = 0;
                for (int i = 0; i < 4; ++i)
                    if (so != kOutside && quad * kQuad + w + i < blocks) v |= (uint32_t)sp[so + quad * kQuad + w + i] << (8 * i);
                *(uint32_t*)(to + lane * kQuad + w) = v;
            }
        }
    }
    // What the first steps wait for, in the order of the steps that follow.
    template <int LO, int HI>
    __device__ __forceinline__ void first(const ExpertArgs& a) {
        scales(a, 0);
        weights(0);
#pragma unroll
        for (int i = 0; i < LO + HI; ++i) rows(0, i);
        weights(1);
#pragma unroll
        for (int i = 0; i < LO; ++i) rows(1, i);
    }
};

// All steps of a tile, then its output.  A wavefront goes on to the next tile's loads as soon as its
// own stores are on their way.
// MT: the tile's height.  The wavefront along the rows wm has the 16-row pieces 2 i + wm.
//
// A step has two phases: the first multiplies the pieces 0 .. kLo - 1 of a wavefront's rows, the
// second the others.  After the first phase nobody reads the step's weight rows (they stay in
// registers) and first input rows again, so their places take those of the step after the next;
// the other input rows' places are free after the second phase.  So every load has one and a
// half steps' time with two stages of LDS.
template <int KIND, int MT>
__device__ __forceinline__ void run_tile(const ExpertArgs& a, const Tile& t, Shared<KIND>& sh) {
    constexpr int kLo = MT > 2 ? MT / 2 : MT;
    constexpr int kXLo = MT == 8 ? 2 : 1, kXHi = MT == 8 ? 2 : MT == 4 ? 1 : 0;   // loads of the two phases' rows
    constexpr int kAhead = Loader<KIND>::kWLoads + kXLo + kXHi;
    constexpr int kWStep = weight_step(KIND), kBlocks = Loader<KIND>::kBlocks;
    Loader<KIND> ld(a, sh);
    ld.begin(a, t);
    ld.template first<kXLo, kXHi>(a);
    const int lane = ld.lane, wave = ld.wave, steps = ld.steps;
    const int wm = wave / 4, wn = wave % 4, l16 = lane % 16, g = lane / 16;

    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    for (int s = 0; s < steps; ++s) {
        const Stage<KIND>& st = sh.stage[s & 1];
        const uint8_t* sc = sh.scales[s * kBlocks / kQuad & 1].of[0] + s * kBlocks % kQuad;
        wait_for_loads<kAhead>();                           // the first phase's rows of step s
        block_barrier();                                    // the second phase of step s - 1 has been read
#pragma unroll
        for (int i = 0; i < kXHi; ++i) ld.rows(s + 1, kXLo + i);
        // 16-bit and 32-bit elements: two times 64 bytes of each row; 8 and 4 bits: 128 elements at once
        constexpr bool kScaledForm = KIND == kMx8 || KIND == kMx8Mx4;
        u32x4 w[2][4];
        int sw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = wn * 64 + j * 16 + l16;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if constexpr (KIND == kBf16Mx4) {
                    const uint32_t q = *(const uint32_t*)(st.w + r * kWStep + k * 16 + g * 4);
                    w[k][j] = widen_e2m1(q, __uint_as_float((uint32_t)sc[r * kQuad + k] << 23));
                } else if constexpr (KIND == kMx8Mx4) {
                    w[k][j] = k ? u32x4{0, 0, 0, 0} : *(const u32x4*)(st.w + place<kWStep>(r, g));
                } else {
                    w[k][j] = *(const u32x4*)(st.w + place<kWStep>(r, k * 4 + g));
                }
            }
            if constexpr (kScaledForm) sw[j] = sc[r * kQuad + g];
        }
        auto multiply = [&](int i) __attribute__((always_inline)) {
            const int r = (2 * i + wm) * 16 + l16;
            const u32x4 x0 = *(const u32x4*)(st.x + place<128>(r, g)), x1 = *(const u32x4*)(st.x + place<128>(r, 4 + g));
            if constexpr (kScaledForm) {
                const int sx = sc[(kTileN + r) * kQuad + g];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = multiply_scaled<KIND>(w[0][j], w[1][j], sw[j], x0, x1, sx, acc[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = multiply16<KIND>(w[0][j], x0, acc[i][j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = multiply16<KIND>(w[1][j], x1, acc[i][j]);
            }
        };
#pragma unroll
        for (int i = 0; i < kLo; ++i) multiply(i);
        wait_for_loads<kAhead>();                           // the second phase's rows of step s
        block_barrier();                                    // the first phase's have been read
        ld.weights(s + 2);
#pragma unroll
        for (int i = 0; i < kXLo; ++i) ld.rows(s + 2, i);
        if (s * kBlocks % kQuad == 0) ld.scales(a, s * kBlocks / kQuad + 1);
#pragma unroll
        for (int i = kLo; i < MT; ++i) multiply(i);
    }
    block_barrier();                                        // the last step has been read

    // Results: lane (l16, g) has columns 4g .. 4g + 3 of a 16 x 16 piece, of input row l16.  Stored
    // as they are, every row would go out in pieces of 32 bytes; so a wavefront puts up to 128 bytes
    // of 8 or 16 rows together in LDS first.
    uint8_t* stage = (uint8_t*)&sh.scales[1] + wave * kOutStage;
    const bool mx_out = rows_scaled(KIND) && a.out_dtype == A2AV_MX8;
    const bool runs = mx_out || (a.out_row % 16 == 0 && (uintptr_t)a.out % 16 == 0);
    const int c0 = t.col0 + wn * (a.swiglu ? 32 : 64);      // the wavefront's first column
    // Writes `rows` staged rows of `bytes` bytes, the first of them the tile's row r0, to column c.
    auto write = [&](int r0, int rows, int bytes, int c, int elem) __attribute__((always_inline)) {
        const int pieces = bytes / 16;
        const int r = lane / pieces, p = lane % pieces;
        wave_sync();
        const u32x4 v = r < rows ? *(const u32x4*)(stage + r * bytes + p * 16) : u32x4{0, 0, 0, 0};
        wave_sync();
        const int left = (a.width - c) * elem - p * 16;     // bytes from the piece to the row's end
        if (r < rows && r0 + r < t.rows && left > 0) {
            uint8_t* to = t.out + (r0 + r) * a.out_row + (int64_t)c * elem + p * 16;
            if (runs && left >= 16) {
                *(u32x4*)to = v;
            } else if constexpr (KIND == kF32) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * e < left) ((uint32_t*)to)[e] = v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (2 * e < left) ((u16*)to)[e] = (u16)(v[e / 2] >> (16 * (e % 2)));
            }
        }
    };
    auto pair = [](float lo, float hi) { return f32_to_bf16(lo) | f32_to_bf16(hi) << 16; };
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r0 = (2 * i + wm) * 16;
        if (r0 >= t.rows) continue;
        f32x4 v[4];
        if (a.swiglu) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[p][e] = silu_mul(acc[i][2 * p][e], acc[i][2 * p + 1][e]);
            v[2] = v[3] = f32x4{0, 0, 0, 0};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[i][j];
        }
        if (rows_scaled(KIND) && mx_out) {
            const int bytes = a.swiglu ? 32 : 64;
            // 32 columns: two pieces of the four lanes that share a row
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && a.swiglu) continue;
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max(m, max(abs_bits(v[2 * h][e]), abs_bits(v[2 * h + 1][e])));
                m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32));
                const uint32_t sb = mx_scale_byte(m);
                const float f = mx_inverse(sb);
#pragma unroll
                for (int q = 2 * h; q < 2 * h + 2; ++q)
                    *(uint32_t*)(stage + l16 * bytes + 16 * q + 4 * g) = mx8_pack(v[q][0] * f, v[q][1] * f, v[q][2] * f,
                                                                                  v[q][3] * f, sb == 255u);
                const int c = c0 + 32 * h;                  // the width is a multiple of 32
                if (r0 + l16 < t.rows && c < a.width) {
                    uint8_t* row = t.out + (r0 + l16) * a.out_row;
                    if (g == 0) row[a.width + c / kMxGroup] = (uint8_t)sb;
                    if (c + 32 == a.width)
                        for (int b = a.width + a.width / kMxGroup + g; b < a.out_row; b += 4) row[b] = 0;
                }
            }
            write(r0, 16, bytes, c0, 1);
        } else if constexpr (KIND == kF32) {
#pragma unroll
            for (int q = 0; q < 4; q += 2) {                // 32 columns at a time, 8 rows at a time
                if (q == 2 && a.swiglu) continue;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (l16 / 8 == half) {
                        *(f32x4*)(stage + l16 % 8 * 128 + 16 * g) = v[q];
                        *(f32x4*)(stage + l16 % 8 * 128 + 64 + 16 * g) = v[q + 1];
                    }
                    write(r0 + 8 * half, 8, 128, c0 + 16 * q, 4);
                }
            }
        } else if (a.swiglu) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *(u32x2*)(stage + l16 * 64 + 32 * q + 8 * g) = u32x2{pair(v[q][0], v[q][1]), pair(v[q][2], v[q][3])};
            write(r0, 16, 64, c0, 2);
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (l16 / 8 == half) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *(u32x2*)(stage + l16 % 8 * 128 + 32 * q + 8 * g) = u32x2{pair(v[q][0], v[q][1]), pair(v[q][2], v[q][3])};
                }
                write(r0 + 8 * half, 8, 128, c0, 2);
            }
        }
    }
}
#endif

template <int KIND>
__global__ void __launch_bounds__(kThreads) expert_tile_kernel(ExpertArgs a) {
#ifdef A2AV_DEVICE_CODE
    __shared__ Shared<KIND> sh;
    int* ends = sh.ends;
    const int mt = __builtin_amdgcn_readfirstlane(count_tiles<kThreads>(
        a, ends, (int*)sh.stage[0].x, [&](int rows) { return rows > a.few ? pieces_of(rows, kMaxM) : 0; }));
    const int cols = a.swiglu ? kTileN / 2 : kTileN;
    const int nt = (a.width + cols - 1) / cols;
    const int64_t total = (int64_t)mt * nt;
    if (total < a.tile_least) return;                       // the few-rows kernel took them
    // Blocks go to the eight dies in turn.  Of every gridDim.x tiles a die gets one run of
    // neighbours, whose rows and weights its L2 then holds once.
    const int run = gridDim.x / 8;
    const int pos = (blockIdx.x % 8) * run + blockIdx.x / 8;
    auto tile_at = [&](int64_t t) {
        Tile tile{};
        if (t >= total) return tile;
        const int64_t sup = t / ((int64_t)kSuper * nt);
        const int in_sup = (int)(t - sup * kSuper * nt), high = min(kSuper, mt - (int)sup * kSuper);
        const int tm = __builtin_amdgcn_readfirstlane((int)sup * kSuper + in_sup % high);
        const int tn = __builtin_amdgcn_readfirstlane(in_sup / high);
        const int grp = __builtin_amdgcn_readfirstlane(find_group(ends, a.G, tm));
        bool bad = false;
        const Group gr = group_of(a, grp, &bad);
        const int m0 = (tm - (grp ? __builtin_amdgcn_readfirstlane(ends[grp - 1]) : 0)) * kMaxM;
        const int64_t row = gr.row + m0;
        const int64_t w0 = (int64_t)grp * a.N;
        tile.in = a.in + row * a.in_row;
        tile.weight = a.weight + w0 * a.w_row;
        tile.scales = a.scales + w0 * (a.K / kMxGroup);
        tile.out = a.out + row * a.out_row;
        tile.rows = __builtin_amdgcn_readfirstlane(min(kMaxM, gr.rows - m0));
        tile.col0 = tn * cols;
        return tile;
    };
    Tile tile = tile_at(pos);
    for (int64_t t = pos; tile.rows > 0; t += gridDim.x) {
        const Tile next = tile_at(t + gridDim.x);
        switch (height_of(tile.rows)) {
            case 8: run_tile<KIND, 8>(a, tile, sh); break;
            case 4: run_tile<KIND, 4>(a, tile, sh); break;
            case 2: run_tile<KIND, 2>(a, tile, sh); break;
            default: run_tile<KIND, 1>(a, tile, sh); break;
        }
        tile = next;
    }
#endif
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
