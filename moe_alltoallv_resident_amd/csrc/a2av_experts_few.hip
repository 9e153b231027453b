// The experts' products for experts with few rows: a decode step's case, bound by reading the
// weights.
//
// Many tiles (a whole batch's step): a block streams 128 weight rows through LDS, 128 bytes of
// each at a time in a ring of two to four stages that are loaded straight from memory, and
// multiplies them with up to 64 input rows.  Whole 128-byte pieces matter: read into registers in
// the matrix instruction's layout, 64 bytes of sixteen rows at a time, the weights came at 4.3
// TB/s only.
//
// Few tiles (one token): a wavefront takes 16 weight rows and a part of their length straight into
// registers, so that as many CUs as possible read; the parts are added through LDS.
//
// Measured: 1,024 bfloat16 rows over 128 experts, 5120 -> 2 x 2048: 0.80 ms, 5.9 TB/s of weights;
// 4-bit weights 0.27 ms, 4.7 TB/s (LDS reads of the input rows beside the weights); 2,048 8-bit
// rows over 256 experts with 4-bit weights, 7168 -> 2 x 2048: 0.70 ms, 5.7 TB/s; one token with
// 4-bit weights 13 to 15 us with the call.
#include "a2av_experts.h"

#include <type_traits>

namespace a2av {
namespace {

[[maybe_unused]] constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kBlocksPerCu = 2;
constexpr int kDirectRows = 16;          // rows that the direct form takes at most
[[maybe_unused]] constexpr int kStreamRows = 128;     // weight rows of a stream tile
[[maybe_unused]] constexpr int kStreamLds = 79872;    // of a block: half of a CU's but for the list of groups

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

template <int KIND>
struct Batch {
    u32x4 w[batch_units(KIND)][w_pieces(KIND)];
    u32x4 x[batch_units(KIND)][x_pieces(KIND)];
    uint8_t ws[batch_units(KIND)], xs[batch_units(KIND)];
};
#endif

struct Job {
    const uint8_t* in;       // the group's first row
    const uint8_t* weight;   // its expert's
    const uint8_t* scales;
    uint8_t* out;
    int rows;                // 1 .. few
    int col0;                // the tile's first output column
};

#ifdef A2AV_DEVICE_CODE
// Writes four neighbouring columns of a row, in float32, as the output type.  With 8-bit rows the
// eight lanes of a scale's 32 columns call it together.
template <int KIND>
__device__ __forceinline__ void write_four(const ExpertArgs& a, uint8_t* row, int c, f32x4 v, bool on) {
    on = on && c < a.width;
    if (rows_scaled(KIND) && a.out_dtype == A2AV_MX8) {
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = max(mx, abs_bits(v[e]));
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, s));
        const uint32_t sb = mx_scale_byte(mx);
        const float f = mx_inverse(sb);
        if (on) {
            *(uint32_t*)(row + c) = mx8_pack(v[0] * f, v[1] * f, v[2] * f, v[3] * f, sb == 255u);
            if (c % kMxGroup == 0) row[a.width + c / kMxGroup] = (uint8_t)sb;
            if (c + 4 == a.width)
                for (int b = a.width + a.width / kMxGroup; b < a.out_row; ++b) row[b] = 0;
        }
    } else if (on) {
        if constexpr (KIND == kF32) {
            float* p = (float*)row + c;
            if (a.width % 4 == 0 && (uintptr_t)a.out % 16 == 0) *(f32x4*)p = v;
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.width) p[e] = v[e];
        } else {
            u16* p = (u16*)row + c;
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = f32_to_bf16(v[e]);
            if (a.width % 4 == 0 && (uintptr_t)a.out % 8 == 0) *(u32x2*)p = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.width) p[e] = (u16)b[e];
        }
    }
}

// ---- few tiles: straight into registers ----------------------------------------------

// A tile is kWaves / parts times 16 weight rows.  With SwiGLU a wavefront's 16 are 8 columns'
// gate rows and their up rows.
template <int KIND>
__device__ __forceinline__ void run_direct(const ExpertArgs& a, const Job& t, int parts, f32x4* part) {
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
    const int c = a.swiglu ? t.col0 + wrow * 8 + l16 % 8 : t.col0 + wrow * 16 + l16;
    const int wr = c < a.width ? (a.swiglu ? c + l16 / 8 * a.width : c) : -1;
    // Lane (l16, g)'s elements of unit u, as byte offsets; outside a row they read zeros.
    auto load = [&](Batch<KIND>& b, int at) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int unit = at + u;
#pragma unroll
            for (int p = 0; p < w_pieces(KIND); ++p) {
                const uint32_t o = (KIND == kMx8 ? unit * 128 + p * 64 : unit * 64) + g * 16;
                const bool on = unit < units && o < (uint32_t)a.w_row && wr >= 0;
                b.w[u][p] = load16(wbuf, on ? (uint32_t)(wr * a.w_row) + o : kOutside);
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
                const bool on = unit < units && o < end;     // rows past the last are past the buffer's end
                b.x[u][p] = load16(xbuf, on ? (uint32_t)(l16 * a.in_row) + o : kOutside);
            }
            if constexpr (weight_scaled(KIND)) {
                const int blk = unit * 4 + g;
                const bool on = unit < units && blk < blocks;
                b.ws[u] = __builtin_amdgcn_raw_buffer_load_b8(sbuf, on && wr >= 0 ? (int)((uint32_t)(wr * blocks) + blk) : (int)kOutside, 0, 0);
                if constexpr (rows_scaled(KIND))
                    b.xs[u] = __builtin_amdgcn_raw_buffer_load_b8(xbuf, on ? (int)(l16 * a.in_row + a.K + blk) : (int)kOutside, 0, 0);
            }
        }
    };
    f32x4 acc = {0, 0, 0, 0};
    auto use = [&](const Batch<KIND>& b) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if constexpr (KIND == kF32 || KIND == kBf16) {
                acc = multiply16<KIND>(b.w[u][0], b.x[u][0], acc);
            } else if constexpr (KIND == kBf16Mx4) {
                const float f = __uint_as_float((uint32_t)b.ws[u] << 23);
#pragma unroll
                for (int p = 0; p < 4; ++p) acc = multiply16<KIND>(widen_e2m1(b.w[u][0][p], f), b.x[u][p], acc);
            } else {
                const u32x4 none = {0, 0, 0, 0};
                acc = multiply_scaled<KIND>(b.w[u][0], KIND == kMx8 ? b.w[u][w_pieces(KIND) - 1] : none, b.ws[u], b.x[u][0],
                                            b.x[u][x_pieces(KIND) - 1], b.xs[u], acc);
            }
        }
    };
    // The parts take batches in turn, so that together they sweep along their rows.
    {
        const int step = parts * kBatch;
        Batch<KIND> b0, b1;
        load(b0, wpart * kBatch);
        for (int at = wpart * kBatch; at < units; at += 2 * step) {
            load(b1, at + step);
            use(b0);
            load(b0, at + 2 * step);
            use(b1);
        }
    }

    part[wave * kWave + lane] = acc;                         // the parts of a row are neighbours
    __syncthreads();
    const int cols = kWaves / parts * 16 / (a.swiglu ? 2 : 1);
    const int quads = cols / 4;                              // four neighbouring columns: one lane's result
    auto sum = [&](int row, int ln) {
        f32x4 v = part[row * parts * kWave + ln];
        for (int p = 1; p < parts; ++p) v += part[(row * parts + p) * kWave + ln];
        return v;
    };
    for (int i = threadIdx.x; i < 16 * quads; i += kThreads) {
        const int m = i / quads, q = i % quads;
        f32x4 v;
        if (!a.swiglu) {
            v = sum(q / 4, m + 16 * (q % 4));
        } else {
            v = sum(q / 2, m + 16 * (q % 2));
            const f32x4 up = sum(q / 2, m + 16 * (q % 2 + 2));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], up[e]);
        }
        write_four<KIND>(a, t.out + m * a.out_row, t.col0 + 4 * q, v, m < t.rows);
    }
    __syncthreads();                                         // `part` is free again
}

// ---- many tiles: a stream through LDS ------------------------------------------------

// A stage: 128 bytes of each of 128 weight rows, and the same elements of 16 * MT input rows.
template <int KIND, int MT>
struct Ring {
    static constexpr int kElems = KIND == kF32 ? 32 : KIND == kBf16 ? 64 : KIND == kMx8 ? 128 : 256;
    static constexpr int kXRow = KIND == kMx8Mx4 ? 256 : KIND == kBf16Mx4 ? 512 : 128;   // bytes of an input row
    static constexpr int kXBytes = 16 * MT * kXRow;
    static constexpr int kStage = kStreamRows * 128 + kXBytes;
    static constexpr int kScales = weight_scaled(KIND) ? 2 * (kStreamRows + 64) * 16 : 0;   // bytes behind the stages
    // as many stages as fit half of a CU's LDS, four at most
    static constexpr int kFit = (kStreamLds - kScales) / kStage;
    static constexpr int kDepth = kFit > 4 ? 4 : kFit > 3 && weight_scaled(KIND) ? 3 : kFit;
    static_assert(kDepth >= 2, "two stages at least");
    static constexpr int kXLoads = kXBytes / 1024;           // of all wavefronts for a stage
    static constexpr int kXPer = (kXLoads + kWaves - 1) / kWaves;
    static constexpr int kResult = 16 * MT * (kStreamRows + 4) * 4;
    static_assert(kResult <= kDepth * kStage, "results fit the ring");
};

// Place of 16-byte piece c of row r in LDS rows of ROW bytes: the same pieces of sixteen rows fall
// into different banks.
template <int ROW>
__device__ inline int moved(int r) {
    return ROW == 128 ? r & 7 : r & 15;
}
template <int ROW>
__device__ inline int place_of(int r, int c) {
    return r * ROW + ((c ^ moved<ROW>(r)) << 4);
}

// WHOLE: rows of scales are whole words; else (a width that is no multiple of 128) they go through
// registers.
template <int KIND, int MT, bool WHOLE>
__device__ __forceinline__ void run_stream(const ExpertArgs& a, const Job& t, uint8_t* lds) {
    using R = Ring<KIND, MT>;
    constexpr int kXRow = R::kXRow, kXPieces = kXRow / 16, kDepth = R::kDepth;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane % 16, g = lane / 16;
    const int steps = (a.K + R::kElems - 1) / R::kElems;
    const int x_bytes = KIND == kF32 ? a.K * 4 : KIND == kBf16 || KIND == kBf16Mx4 ? a.K * 2 : a.K;
    const int blocks = a.K / kMxGroup;
    const uint32_t lds_at = lds_address(lds);
    uint8_t* scales = lds + kDepth * R::kStage;              // two times sixteen blocks' bytes of the weight and input rows

    const u32x4 xbuf = buffer_words(t.in, (uint32_t)(t.rows * a.in_row));
    const u32x4 wbuf = buffer_words(t.weight, (uint32_t)(a.N * a.w_row));
    // wavefront w's 16 rows of the tile; with SwiGLU 8 columns' gate rows and their up rows
    auto weight_row = [&](int r) {
        const int c = a.swiglu ? t.col0 + r / 16 * 8 + r % 8 : t.col0 + r;
        return c < a.width ? (a.swiglu ? c + r / 8 % 2 * a.width : c) : -1;
    };
    uint32_t wo[2], xo[R::kXPer];
    const int wc = ((lane % 8) ^ (lane / 8)) * 16;           // load i: tile rows 16 * wave + 8 i ..
    const bool w_over = wc >= (int)a.w_row - (steps - 1) * 128;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int wr = weight_row(wave * 16 + i * 8 + lane / 8);
        wo[i] = wr < 0 ? kOutside : (uint32_t)(wr * a.w_row + wc);
    }
    bool x_over[R::kXPer];
#pragma unroll
    for (int i = 0; i < R::kXPer; ++i) {
        const int r = (i * kWaves + wave) * (1024 / kXRow) + lane / kXPieces, c = ((lane % kXPieces) ^ moved<kXRow>(r)) * 16;
        xo[i] = (uint32_t)(r * a.in_row + c);                // rows past the last: past the buffer's end
        x_over[i] = c >= x_bytes - (steps - 1) * kXRow;
    }
    // Wavefronts 0 and 1 load the weight rows' scale bytes, 2 the input rows', sixteen blocks at once.
    const bool scale_wave = weight_scaled(KIND) && wave < (rows_scaled(KIND) ? 3 : 2);
    const u32x4 sbuf = buffer_words(wave < 2 ? t.scales : t.in, wave < 2 ? (uint32_t)a.N * (uint32_t)blocks : (uint32_t)(t.rows * a.in_row));
    uint32_t so = kOutside;
    if (weight_scaled(KIND) && wave < 2) {
        const int wr = weight_row(wave * 64 + lane);
        if (wr >= 0) so = (uint32_t)(wr * blocks);
    } else if (rows_scaled(KIND) && wave == 2 && lane < t.rows) {
        so = (uint32_t)(lane * a.in_row + a.K);
    }
    constexpr int kBlocks = R::kElems / kMxGroup;            // of a stage
    const bool x_wave = R::kXLoads % kWaves == 0 || (R::kXPer - 1) * kWaves + wave < R::kXLoads;   // makes all kXPer loads
    // Past the last stage everything reads zeros: the counts that the waits go by stay the same.
    auto load = [&](int s) __attribute__((always_inline)) {
        const uint32_t st = lds_at + s % kDepth * R::kStage;
        if (weight_scaled(KIND) && scale_wave && s * kBlocks % 16 == 0 && s < steps) {
            if (WHOLE)
                load_to_lds(sbuf, lds_at + kDepth * R::kStage + (s * kBlocks / 16 % 2) * ((kStreamRows + 64) * 16) + wave * 1024, so, s * kBlocks);
            else
                *(u32x4*)(scales + (s * kBlocks / 16 % 2) * ((kStreamRows + 64) * 16) + wave * 1024 + lane * 16) =
                    so == kOutside ? u32x4{0, 0, 0, 0}
                                   : scale_bytes((wave < 2 ? t.scales : t.in) + so + s * kBlocks, blocks - s * kBlocks,
                                                 wave < 2 ? (int64_t)a.N * blocks - so - s * kBlocks : a.in_row - a.K - s * kBlocks);
        }
        const bool in = s < steps, last = s == steps - 1;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_to_lds(wbuf, st + wave * 2048 + i * 1024, in && !(last && w_over) ? wo[i] : kOutside, s * 128);
#pragma unroll
        for (int i = 0; i < R::kXPer; ++i)
            if (i + 1 < R::kXPer || x_wave)
                load_to_lds(xbuf, st + kStreamRows * 128 + (i * kWaves + wave) * 1024, in && !(last && x_over[i]) ? xo[i] : kOutside,
                            s * kXRow);
    };
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) load(s);
    for (int s = 0; s < steps; ++s) {
        // stage s has landed when only the later stages' loads are on their way
        if (x_wave) wait_for_loads<(kDepth - 2) * (2 + R::kXPer)>();
        else wait_for_loads<(kDepth - 2) * (1 + R::kXPer)>();
        block_barrier();                                     // for everyone, and stage s - 1 has been read
        load(s + kDepth - 1);
        const uint8_t* wst = lds + s % kDepth * R::kStage + wave * 2048;
        const uint8_t* xst = lds + s % kDepth * R::kStage + kStreamRows * 128;
        const uint8_t* sc = scales + (s * kBlocks / 16 % 2) * ((kStreamRows + 64) * 16) + s * kBlocks % 16;
        const u32x4 w0 = *(const u32x4*)(wst + place_of<128>(l16, g)), w1 = *(const u32x4*)(wst + place_of<128>(l16, 4 + g));
        if constexpr (KIND == kF32 || KIND == kBf16) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = i * 16 + l16;
                acc[i] = multiply16<KIND>(w0, *(const u32x4*)(xst + place_of<kXRow>(r, g)), acc[i]);
                acc[i] = multiply16<KIND>(w1, *(const u32x4*)(xst + place_of<kXRow>(r, 4 + g)), acc[i]);
            }
        } else if constexpr (KIND == kBf16Mx4) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u && s * kBlocks + 4 >= blocks) break;   // the row has ended: no scales here
                // a lane's 16 bytes are 32 elements, a scale's
                const float f = __uint_as_float((uint32_t)sc[(wave * 16 + l16) * 16 + u * 4 + g] << 23);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const u32x4 w = widen_e2m1(u ? w1[p] : w0[p], f);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[i] = multiply16<KIND>(w, *(const u32x4*)(xst + place_of<kXRow>(i * 16 + l16, (u * 4 + g) * 4 + p)), acc[i]);
                }
            }
        } else {
            constexpr int kUnits = KIND == kMx8 ? 1 : 2;     // of 128 elements
            const u32x4 none = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                if (u && s * kBlocks + 4 >= blocks) break;
                const int ws = sc[(wave * 16 + l16) * 16 + u * 4 + g];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int r = i * 16 + l16;
                    const int xs = sc[(kStreamRows + r) * 16 + u * 4 + g];
                    acc[i] = multiply_scaled<KIND>(u ? w1 : w0, KIND == kMx8 ? w1 : none, ws,
                                                   *(const u32x4*)(xst + place_of<kXRow>(r, u * 8 + g)),
                                                   *(const u32x4*)(xst + place_of<kXRow>(r, u * 8 + 4 + g)), xs, acc[i]);
                }
            }
        }
    }
    wait_for_loads<0>();
    block_barrier();                                         // LDS is free
    float* res = (float*)lds;                                // [16 * MT][kStreamRows + 4]
    constexpr int kPitch = kStreamRows + 4;
#pragma unroll
    for (int i = 0; i < MT; ++i) *(f32x4*)(res + (i * 16 + l16) * kPitch + wave * 16 + 4 * g) = acc[i];
    __syncthreads();
    const int quads = kStreamRows / (a.swiglu ? 8 : 4);
    for (int i = threadIdx.x; i < 16 * MT * quads; i += kThreads) {
        const int m = i / quads, q = i % quads;
        const float* row = res + m * kPitch;
        f32x4 v;
        if (!a.swiglu) {
            v = *(const f32x4*)(row + 4 * q);
        } else {
            v = *(const f32x4*)(row + q / 2 * 16 + q % 2 * 4);
            const f32x4 up = *(const f32x4*)(row + q / 2 * 16 + 8 + q % 2 * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], up[e]);
        }
        write_four<KIND>(a, t.out + m * a.out_row, t.col0 + 4 * q, v, m < t.rows);
    }
    block_barrier();                                         // LDS is free again
}
#endif

template <int KIND>
__global__ void __launch_bounds__(kThreads, 2 * kBlocksPerCu) expert_few_kernel(ExpertArgs a) {
#ifdef A2AV_DEVICE_CODE
    __shared__ __align__(1024) uint8_t lds[kStreamLds];
    __shared__ int ends[kEntries];
    const int per = groups_an_entry(a);
    const int cols_stream = a.swiglu ? kStreamRows / 2 : kStreamRows;
    const int nt_stream = (a.width + cols_stream - 1) / cols_stream;
    const int chunk = a.few;                                 // rows of a stream tile
    // The groups of more than `lo` and at most `hi` rows, in pieces of `chunk` rows.
    int lo = 0, hi = a.few;
    auto pieces = [&](int rows) { return rows > lo && rows <= hi ? pieces_of(rows, chunk) : 0; };
    auto list = [&] { return __builtin_amdgcn_readfirstlane(count_tiles<kThreads>(a, ends, (int*)lds, pieces, per)); };
    auto job_at = [&](int i, int col0) {
        const Piece p = find_piece(a, ends, per, i, pieces);
        const int64_t w0 = (int64_t)p.group * a.N, row = p.rows.row + (int64_t)p.n * chunk;
        return Job{a.in + row * a.in_row, a.weight + w0 * a.w_row, a.scales + w0 * (a.K / kMxGroup), a.out + row * a.out_row,
                   __builtin_amdgcn_readfirstlane(min(chunk, p.rows.rows - p.n * chunk)), col0};
    };
    // stream tiles of the small groups and of all, row tiles of the large ones, groups for the direct form
    const Four n4 = count_groups<kThreads>(a, (int*)lds, [&](int rows) {
        return Four{{rows <= chunk && rows > 0, pieces_of(rows, chunk), rows > chunk ? pieces_of(rows, kTileRows) : 0,
                     rows > 0 && rows <= kDirectRows}};
    });
    const bool all = large_tiles(a, n4.v[2]) < a.tile_least;
    if (all) hi = INT32_MAX;
    int n = __builtin_amdgcn_readfirstlane(all ? n4.v[1] : n4.v[0]);
    if (n == 0) return;
    const bool direct = __builtin_amdgcn_readfirstlane(n4.v[3]) > 0 &&
                        (int64_t)n * nt_stream < gridDim.x / kBlocksPerCu;
    if (direct) {
        // Not a stream tile for every CU: groups of up to 16 rows go by smaller pieces.  Every row's
        // length is cut into as many parts as a block has wavefronts.
        const int limit = hi;
        hi = kDirectRows;
        n = list();
        const int batches = (a.K + unit_elems(KIND) * batch_units(KIND) - 1) / (unit_elems(KIND) * batch_units(KIND));
        const int most = a.out_dtype != A2AV_MX8 ? 8 : a.swiglu ? 2 : 4;   // a tile of 8-bit rows has 32 columns at least
        int parts = 1;
        while (parts < most && parts < batches) parts *= 2;
        const int cols = kWaves / parts * 16 / (a.swiglu ? 2 : 1);
        const int nt = (a.width + cols - 1) / cols;
        for (int64_t t = blockIdx.x; t < (int64_t)n * nt; t += gridDim.x)
            run_direct<KIND>(a, job_at((int)(t / nt), (int)(t % nt) * cols), parts, (f32x4*)lds);
        lo = kDirectRows;
        hi = limit;
    }
    n = list();
    auto stream = [&](auto whole) __attribute__((always_inline)) {
        for (int64_t t = blockIdx.x; t < (int64_t)n * nt_stream; t += gridDim.x) {
            const Job job = job_at((int)(t / nt_stream), (int)(t % nt_stream) * cols_stream);
            if (job.rows <= 16) run_stream<KIND, 1, whole.value>(a, job, lds);
            else if (KIND == kBf16Mx4 || job.rows <= 32) run_stream<KIND, 2, whole.value>(a, job, lds);
            else if constexpr (KIND != kBf16Mx4) run_stream<KIND, 4, whole.value>(a, job, lds);
        }
    };
    if (!weight_scaled(KIND) || (a.K / kMxGroup % 4 == 0 && (uintptr_t)a.scales % 4 == 0)) stream(std::true_type());
    else if constexpr (weight_scaled(KIND)) stream(std::false_type());
#endif
}

template <int KIND>
hipError_t launch(const ExpertArgs& a, int num_cu, hipStream_t st) {
    hipLaunchKernelGGL((expert_few_kernel<KIND>), dim3((unsigned)(num_cu * kBlocksPerCu)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

// The stream takes up to 64 input rows, 32 of bfloat16 with 4-bit weights (their 256 elements of a
// stage are 512 bytes).
int few_rows(const ExpertArgs& a) { return kind_of(a) == kBf16Mx4 ? 32 : 64; }

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
