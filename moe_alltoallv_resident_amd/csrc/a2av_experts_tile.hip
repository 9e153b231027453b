// The experts' products on the matrix units.
//
// A tile is up to 256 rows of one expert by 256 rows of its weight.  Both are staged through
// LDS in steps of 128 bytes of a row (64 bfloat16, 128 e4m3, 32 float32 elements; 4-bit weights
// take 32 or 64 bytes for the same elements), loaded straight from memory into LDS while the
// steps before are multiplied.  Four wavefronts, one on each SIMD, hold 128 x 128 results each:
// that takes 128 KB of LDS reads a step where eight wavefronts of 128 x 64 take 192 KB, which
// with the 64 KB that arrive kept LDS busy for as long as the matrix units.  The weight is the
// matrix instruction's first operand, so a lane ends up with four neighbouring columns of one
// output row.
//
// Matrix instructions: 32x32x16 (bfloat16), 32x32x2 (float32), 32x32x64 with a scale for every
// 32 elements (e4m3 and E2M1 as they are stored).  4-bit weights with bfloat16 rows are widened
// in registers, exactly: an E2M1 element times a power of two is a bfloat16.
//
// Measured: 65,536 rows over 128 experts, 5120 -> 2 x 2048: bfloat16 2.83 ms (0.97 PFLOP/s; a
// library product of this size 1.43 at the same power limit), 8-bit rows and weights 1.83 ms; 262,144
// 8-bit rows over 256 experts with 4-bit weights, 2048 -> 7168: 4.3 ms (1.8 PFLOP/s).
#include "a2av_experts.h"

namespace a2av {
namespace {

[[maybe_unused]] constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kTileN = kTileRows;        // weight rows of a tile
constexpr int kMaxM = kTileRows;         // input rows of the largest tile
constexpr int kRowStep = 128;            // bytes of an input row in a step
[[maybe_unused]] constexpr int kSuper = 4;                // row tiles that are walked together

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

template <int KIND>
struct Shared {
    Stage<KIND> stage[2];
    Scales scales[2];
    int ends[kEntries];
    uint32_t ahead[kWaves][kWave];   // what is loaded only to have it in the L2 goes here
};

// Where 16-byte piece c of row r stands in its LDS row: the same pieces of any sixteen rows that
// differ modulo 16 fall into different banks (with the pieces moved by the row modulo 8 instead, half
// of the LDS cycles were conflicts).
[[maybe_unused]] __host__ __device__ constexpr int moved(int step, int r) { return step == 128 ? r >> 1 & 7 : step == 64 ? r >> 2 & 3 : r >> 3 & 1; }
template <int STEP>
__device__ inline int place(int r, int c) {
    return r * STEP + ((c ^ moved(STEP, r)) << 4);
}

// The piece that belongs at place p of row r.
template <int STEP>
__device__ inline int piece_at(int r, int p) {
    return p ^ moved(STEP, r);
}

// Row pieces of 32 for each of the two wavefronts along the rows: a tile has 64 * 4, 2 or 1 rows.
[[maybe_unused]] __device__ inline int height_of(int rows) { return rows > 128 ? 4 : rows > 64 ? 2 : 1; }

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
    static constexpr int kXLoads = kMaxM / 8 / kWaves;           // load i: the tile's rows 32 i .. 32 i + 31
    static constexpr int kBlocks = step_elems(KIND) / kMxGroup;  // scale bytes of a step

    Shared<KIND>& sh;
    uint32_t lds;            // its address
    int lane, wave, steps, blocks;
    u32x4 xbuf, wbuf, sbuf;
    uint32_t xo[kXLoads], wo[kWLoads], wso, xso, xrow;
    bool x_over, w_over;     // the lane's pieces are past the row's end in the last step
    const uint8_t *wsp, *xsp;   // for scales that go through registers

    // weight row of tile row r: with SwiGLU 32 gate rows and the 32 up rows of the same columns in turn
    static __device__ int weight_row(const ExpertArgs& a, const Tile& t, int r) {
        if (!a.swiglu) return t.col0 + r < a.width ? t.col0 + r : -1;
        const int c = t.col0 + (r / 64) * 32 + r % 32;
        return c < a.width ? c + (r / 32 % 2 ? a.width : 0) : -1;
    }

    __device__ __forceinline__ Loader(const ExpertArgs& a, Shared<KIND>& s) : sh(s) {
        lane = threadIdx.x % kWave;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        steps = (a.K + step_elems(KIND) - 1) / step_elems(KIND);
        blocks = a.K / kMxGroup;
        lds = lds_address(&sh);
    }

    // Byte offsets of this lane's pieces; rows past the tile's and columns past the last one read
    // zeros, and so do in the last step pieces past the row's end.
    __device__ __forceinline__ void begin(const ExpertArgs& a, const Tile& t) {
        xbuf = buffer_words(t.in, (uint32_t)(t.rows * a.in_row));
        wbuf = buffer_words(t.weight, (uint32_t)(a.N * a.w_row));
        const int x_bytes = KIND == kF32 ? a.K * 4 : KIND == kBf16 || KIND == kBf16Mx4 ? a.K * 2 : a.K;
        // load i has row 8 (4 i + wave) + lane / 8: its piece's move is the same for every i
        const int xc = piece_at<128>(wave * 8 + lane / 8, lane % 8) * 16;
        x_over = xc >= x_bytes - (steps - 1) * kRowStep;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) xo[i] = (uint32_t)(((i * kWaves + wave) * 8 + lane / 8) * a.in_row + xc);
        const int wc = piece_at<kWStep>(wave * kWRows + lane / kWPieces, lane % kWPieces) * 16;
        w_over = wc >= (int)a.w_row - (steps - 1) * kWStep;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
            const int wr = weight_row(a, t, (i * kWaves + wave) * kWRows + lane / kWPieces);
            wo[i] = wr < 0 ? kOutside : (uint32_t)(wr * a.w_row + wc);
        }
        xrow = (uint32_t)(threadIdx.x * a.in_row);
        if constexpr (weight_scaled(KIND)) {
            const int wr = weight_row(a, t, threadIdx.x);
            // each wavefront loads the scales of 64 weight rows and of 64 input rows
            sbuf = buffer_words(t.scales, (uint32_t)a.N * (uint32_t)blocks);
            wsp = t.scales;
            xsp = t.in;
            wso = wr >= 0 ? (uint32_t)(wr * blocks) : kOutside;
            xso = (int)threadIdx.x < t.rows ? (uint32_t)(threadIdx.x * a.in_row + a.K) : kOutside;
        }
    }
    __device__ __forceinline__ uint32_t stage_at(int s) { return lds + offsetof(Shared<KIND>, stage) + (s & 1) * sizeof(Stage<KIND>); }
    // Loads past the last step read zeros too: the counts that the waits go by stay the same.
    __device__ __forceinline__ void rows(int s, int i) {
        const bool on = s < steps - 1 || (s == steps - 1 && !x_over);
        load_to_lds(xbuf, stage_at(s) + offsetof(Stage<KIND>, x) + (i * kWaves + wave) * 1024, on ? xo[i] : kOutside, s * kRowStep);
    }
    __device__ __forceinline__ void weights(int s, int i) {
        const bool on = s < steps - 1 || (s == steps - 1 && !w_over);
        load_to_lds(wbuf, stage_at(s) + offsetof(Stage<KIND>, w) + (i * kWaves + wave) * 1024, on ? wo[i] : kOutside, s * kWStep);
    }
    // The memory lines of a step's input rows, into the L2 alone: a word of each of the wavefront's 64
    // rows.  8-bit rows are not whole lines long, so most of their 128-byte pieces lie in two lines and
    // come later than the weights' (185 -> 165 thousand cycles a tile of 40 steps).  Rows and weights
    // in whole lines lost by it (220 -> 258 thousand a tile of 80 steps in bfloat16).
    static constexpr int kLookAhead = rows_scaled(KIND) ? 4 : 0;   // steps
    __device__ __forceinline__ void look_ahead(int s) {
        if constexpr (kLookAhead > 0) load_word_to_lds(xbuf, lds + offsetof(Shared<KIND>, ahead) + wave * sizeof(sh.ahead[0]), s < steps ? xrow : kOutside, s * kRowStep);
    }
    // load n of a step's
    __device__ __forceinline__ void load(int s, int n) {
        if (n < kWLoads) weights(s, n);
        else rows(s, n - kWLoads);
    }
    // Scale bytes, sixteen blocks at a time; rows of scales that are not whole words (a width that is
    // no multiple of 128) go through registers.
    __device__ __forceinline__ void scales(const ExpertArgs& a, int quad) {
        if (!weight_scaled(KIND) || quad * kQuad >= blocks) return;
        if (blocks % 4 == 0 && (uintptr_t)a.scales % 4 == 0) {
            const uint32_t to = lds + offsetof(Shared<KIND>, scales) + (quad & 1) * sizeof(Scales) + wave * kWave * kQuad;
            load_to_lds(sbuf, to, wso, quad * kQuad);
            if (rows_scaled(KIND)) load_to_lds(xbuf, to + kTileN * kQuad, xso, quad * kQuad);
        } else {
            const int valid = blocks - quad * kQuad;
            u32x4 w = {0, 0, 0, 0}, x = w;
            if (wso != kOutside)
                w = scale_bytes(wsp + wso + quad * kQuad, valid, (int64_t)a.N * blocks - wso - quad * kQuad);
            if (rows_scaled(KIND) && xso != kOutside)
                x = scale_bytes(xsp + xso + quad * kQuad, valid, a.in_row - a.K - quad * kQuad);
            *(u32x4*)sh.scales[quad & 1].of[wave * kWave + lane] = w;
            if (rows_scaled(KIND)) *(u32x4*)sh.scales[quad & 1].of[kTileN + wave * kWave + lane] = x;
        }
    }
};

// A wavefront's operands of half a step: 64 bytes of 128 weight rows and of its input rows.
template <int HT>
struct Half {
    u32x4 w[4][2], x[HT][2];
};

// A step's scale words of the same rows, so shifted that byte 2k is the lane's of half k.
template <int HT>
struct Words {
    int w[4], x[HT];
};

// All steps of a tile, then its output.  A wavefront goes on to the next tile's loads as soon as its
// own stores are on their way.  HT: the tile's height; the wavefront along the rows wm has the 32-row
// pieces 2 i + wm.
//
// A step's first half is in registers when the step begins.  While it is multiplied the second half
// is read; as soon as everyone has read it the step's place in LDS takes the step after the next,
// and while the second half is multiplied the next step's first half is read.
//
// Measured at 65,536 bfloat16 rows, 5120 -> 2 x 2048 over 128 experts (a tile: 80 steps of 2,048
// cycles of matrix work): 192 thousand cycles a tile in the steps (219 with one barrier a step, when
// the next step's loads begin half a step later; 178 with the memory taken out), 14 for the output,
// 6 for the start.  By then the card lowers its clock under the load (to about 1.4 GHz), so that 12 %
// fewer cycles took 3 % off the time.
template <int KIND, int HT>
__device__ __forceinline__ void run_tile(const ExpertArgs& a, const Tile& t, Shared<KIND>& sh) {
    constexpr int kLoads = Loader<KIND>::kWLoads + 2 * HT;  // of a wavefront for a step
    constexpr int kWStep = weight_step(KIND), kBlocks = Loader<KIND>::kBlocks;
    Loader<KIND> ld(a, sh);
    ld.begin(a, t);
    ld.scales(a, 0);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) ld.load(0, n);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) ld.load(1, n);
#pragma unroll
    for (int s = 2; s < Loader<KIND>::kLookAhead; ++s) ld.look_ahead(s);
    const int lane = ld.lane, wave = ld.wave, steps = ld.steps;
    const int wm = wave / 2, wn = wave % 2, l32 = lane % 32, h = lane / 32;

    // Read n of the kReads that bring half k of step s to registers.
    constexpr int kReads = 4 + HT;
    auto read = [&](Half<HT>& f, Words<HT>& words, int s, int k, int n) __attribute__((always_inline)) {
        const Stage<KIND>& st = sh.stage[s & 1];
        const uint8_t* sc = sh.scales[s * kBlocks / kQuad & 1].of[0] + s * kBlocks % kQuad;
        if (n < 4) {
            const int r = wn * 128 + n * 32 + l32;
            if constexpr (KIND == kBf16Mx4) {
                const float scale = __uint_as_float((uint32_t)sc[r * kQuad + k] << 23);
                f.w[n][0] = widen_e2m1(*(const uint32_t*)(st.w + place<kWStep>(r, k) + h * 4), scale);
                f.w[n][1] = widen_e2m1(*(const uint32_t*)(st.w + place<kWStep>(r, k) + 8 + h * 4), scale);
            } else if constexpr (KIND == kMx8Mx4) {
                f.w[n][0] = *(const u32x4*)(st.w + place<kWStep>(r, k * 2 + h));
                f.w[n][1] = u32x4{0, 0, 0, 0};
            } else {
                f.w[n][0] = *(const u32x4*)(st.w + place<kWStep>(r, k * 4 + h));
                f.w[n][1] = *(const u32x4*)(st.w + place<kWStep>(r, k * 4 + 2 + h));
            }
            if (k == 0) words.w[n] = rows_scaled(KIND) ? *(const uint32_t*)(sc + r * kQuad) >> (8 * h) : 0;
        } else {
            const int i = n - 4, r = (2 * i + wm) * 32 + l32;
            f.x[i][0] = *(const u32x4*)(st.x + place<128>(r, k * 4 + h));
            f.x[i][1] = *(const u32x4*)(st.x + place<128>(r, k * 4 + 2 + h));
            if (k == 0) words.x[i] = rows_scaled(KIND) ? *(const uint32_t*)(sc + (kTileN + r) * kQuad) >> (8 * h) : 0;
        }
    };
    f32x16 acc[HT][4];
#pragma unroll
    for (int i = 0; i < HT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    // Product n of a half.  The order of reads, loads and products is fixed piece by piece: left to
    // itself the compiler puts every read right before its use, and with one wavefront on a SIMD
    // nothing else runs while it waits.
    constexpr int kProducts = 4 * HT;
    auto multiply = [&](const Half<HT>& f, const Words<HT>& words, auto half, int n) __attribute__((always_inline)) {
        const int i = n / 4, j = n % 4;
        acc[i][j] = multiply32<KIND, 2 * decltype(half)::value>(f.w[j][0], f.w[j][1], words.w[j], f.x[i][0], f.x[i][1], words.x[i],
                                                                acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 0> kFirst{};
    constexpr std::integral_constant<int, 1> kSecond{};

    Half<HT> f0, f1;
    Words<HT> words, next;
    wait_for_loads<kLoads + (Loader<KIND>::kLookAhead ? Loader<KIND>::kLookAhead - 2 : 0)>();   // step 0; step 1 is on its way
    block_barrier();
#pragma unroll
    for (int n = 0; n < kReads; ++n) read(f0, next, 0, 0, n);
    // Loads of a step that begin before the step ahead of it is needed, and those that begin after.
    constexpr int kEarly = kLoads / 2, kAhead = Loader<KIND>::kLookAhead ? 1 : 0, kMid = kProducts / 2;
    for (int s = 0; s < steps; ++s) {
        words = next;
#pragma unroll
        for (int n = 0; n < kMid; ++n) {
#pragma unroll
            for (int q = n * kReads / kMid; q < (n + 1) * kReads / kMid; ++q) read(f1, words, s, 1, q);
            multiply(f0, words, kFirst, n);
        }
        block_barrier();                                    // step s has been read
#pragma unroll
        for (int n = kMid; n < kProducts; ++n) {
#pragma unroll
            for (int q = (n - kMid) * kEarly / kMid; q < (n - kMid + 1) * kEarly / kMid; ++q) ld.load(s + 2, q);
            multiply(f0, words, kFirst, n);
        }
        wait_for_loads<kEarly + kAhead>();                  // step s + 1; what is looked ahead for may be on its way
        block_barrier();                                    // for everyone
        if (s * kBlocks % kQuad == 0) ld.scales(a, s * kBlocks / kQuad + 1);
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
#pragma unroll
            for (int q = kEarly + n * (kLoads - kEarly) / kProducts; q < kEarly + (n + 1) * (kLoads - kEarly) / kProducts; ++q) ld.load(s + 2, q);
            if (n == kProducts - 1) ld.look_ahead(s + Loader<KIND>::kLookAhead);
#pragma unroll
            for (int q = n * kReads / kProducts; q < (n + 1) * kReads / kProducts; ++q) read(f0, next, s + 1, 0, q);   // zeros after the last step
            multiply(f1, words, kSecond, n);
        }
    }
    wait_for_loads<0>();
    block_barrier();                                        // the last step has been read

    // Results: lane (l32, h) has columns 8q + 4h .. 8q + 4h + 3 of a 32 x 32 piece, of input row l32.
    // They go through the wavefront's quarter of the stages in float32, and a short loop makes eight
    // output columns a lane of them, in runs of up to 256 bytes a row.  (Done in registers instead, the
    // same work is unrolled for every piece and form of output: that code no longer fits the
    // instruction cache and took four times as long.)
    constexpr int kRoom = sizeof(sh.stage) / kWaves / 1024 * 1024;
    constexpr int kPitch = 128 * 4, kFit = kRoom / (32 * kPitch) < HT ? kRoom / (32 * kPitch) : HT;   // 32-row pieces at a time
    static_assert(kFit >= 1 && HT % kFit == 0, "whole passes");
    uint8_t* stage = (uint8_t*)&sh.stage[0] + wave * kRoom;
    auto at = [&](int r, int piece) { return (f32x4*)(stage + r * kPitch + ((piece ^ (r & 15)) << 4)); };   // four columns
    const bool mx_out = rows_scaled(KIND) && a.out_dtype == A2AV_MX8;
    const int elem = mx_out ? 1 : KIND == kF32 ? 4 : 2;
    const int shift = a.swiglu ? 3 : 4;                     // 8 or 16 times eight columns of the wavefront
    const int c0 = t.col0 + (wn << (shift + 3));
    const bool runs = mx_out || (a.out_row % 16 == 0 && (uintptr_t)a.out % 16 == 0);
#pragma unroll
    for (int i0 = 0; i0 < HT; i0 += kFit) {
#pragma unroll
        for (int i = i0; i < i0 + kFit; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *at((i - i0) * 32 + l32, j * 8 + 2 * q + h) = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                                                        acc[i][j][4 * q + 3]};
        wave_sync();
#pragma unroll 1
        for (int n = lane; n < kFit * 32 << shift; n += kWave) {
            const int r = n >> shift, u = n & ((1 << shift) - 1), row = (2 * (i0 + r / 32) + wm) * 32 + r % 32, c = c0 + 8 * u;
            f32x4 lo, hi;
            if (a.swiglu) {
                const int gate = u / 4 * 16 + u % 4 * 2;
                lo = *at(r, gate);
                hi = *at(r, gate + 1);
                const f32x4 ulo = *at(r, gate + 8), uhi = *at(r, gate + 9);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo[e] = silu_mul(lo[e], ulo[e]);
                    hi[e] = silu_mul(hi[e], uhi[e]);
                }
            } else {
                lo = *at(r, 2 * u);
                hi = *at(r, 2 * u + 1);
            }
            const int left = (a.width - c) * elem;          // bytes to the row's end
            const bool on = row < t.rows && left > 0;
            uint8_t* to = t.out + row * a.out_row + (int64_t)c * elem;
            if (rows_scaled(KIND) && mx_out) {
                // a scale's 32 columns are four neighbouring lanes' (the width is a multiple of 32)
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max(m, max(abs_bits(lo[e]), abs_bits(hi[e])));
                m = max(m, (uint32_t)__shfl_xor((int)m, 1));
                m = max(m, (uint32_t)__shfl_xor((int)m, 2));
                const uint32_t sb = mx_scale_byte(m);
                const float f = mx_inverse(sb);
                if (!on) continue;
                *(u32x2*)to = u32x2{mx8_pack(lo[0] * f, lo[1] * f, lo[2] * f, lo[3] * f, sb == 255u),
                                    mx8_pack(hi[0] * f, hi[1] * f, hi[2] * f, hi[3] * f, sb == 255u)};
                if (u % 4 == 0) t.out[row * a.out_row + a.width + c / kMxGroup] = (uint8_t)sb;
                if (c + 8 == a.width)
                    for (int b = a.width + a.width / kMxGroup; b < a.out_row; ++b) t.out[row * a.out_row + b] = 0;
            } else if constexpr (KIND == kF32) {
                if (!on) continue;
                if (runs && left >= 32) {
                    ((f32x4*)to)[0] = lo;
                    ((f32x4*)to)[1] = hi;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (4 * e < left) ((float*)to)[e] = e < 4 ? lo[e % 4] : hi[e % 4];
                }
            } else {
                if (!on) continue;
                const u32x4 v = {f32_to_bf16_pair(lo[0], lo[1]), f32_to_bf16_pair(lo[2], lo[3]), f32_to_bf16_pair(hi[0], hi[1]),
                                 f32_to_bf16_pair(hi[2], hi[3])};
                if (runs && left >= 16) {
                    *(u32x4*)to = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (2 * e < left) ((u16*)to)[e] = (u16)(v[e / 2] >> (16 * (e % 2)));
                }
            }
        }
        wave_sync();
    }
    block_barrier();                                        // the stages are free
}
#endif

template <int KIND>
__global__ void __launch_bounds__(kThreads) expert_tile_kernel(ExpertArgs a) {
#ifdef A2AV_DEVICE_CODE
    __shared__ Shared<KIND> sh;
    auto pieces = [&](int rows) { return rows > a.few ? pieces_of(rows, kMaxM) : 0; };
    const int each = groups_an_entry(a);
    const int mt = __builtin_amdgcn_readfirstlane(count_tiles<kThreads>(a, sh.ends, (int*)sh.stage[0].x, pieces, each));
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
        const Piece p = find_piece(a, sh.ends, each, tm, pieces);
        const int m0 = p.n * kMaxM;
        const int64_t row = p.rows.row + m0, w0 = (int64_t)p.group * a.N;
        tile.in = a.in + row * a.in_row;
        tile.weight = a.weight + w0 * a.w_row;
        tile.scales = a.scales + w0 * (a.K / kMxGroup);
        tile.out = a.out + row * a.out_row;
        tile.rows = __builtin_amdgcn_readfirstlane(min(kMaxM, p.rows.rows - m0));
        tile.col0 = tn * cols;
        return tile;
    };
    Tile tile = tile_at(pos);
    for (int64_t t = pos; tile.rows > 0; t += gridDim.x) {
        const Tile next = tile_at(t + gridDim.x);
        switch (height_of(tile.rows)) {
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
