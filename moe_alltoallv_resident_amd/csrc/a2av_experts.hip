// The experts' matrix products on expert-major receive rows (declared in include/a2av.h):
// out[r] = act(in[r] . weight_e^T) for every row r of every expert e, with the row counts
// read on the GPU.
//
// No host knows how many rows an expert got, so no grid can be cut to them: every block
// reads the group starts, counts the row tiles of every expert into LDS and walks the tile
// list (tile t, t + blocks, ...) until it ends.
// Here: the entry point and the general kernel.
#include "a2av_experts.h"

namespace a2av {
namespace {

constexpr int32_t kMaxDim = 1 << 20;

// ---- the general form ----------------------------------------------------------------
// Any width, stride and alignment that the call allows: elements are read one by one,
// widened to float32 and multiplied on the vector units.

__device__ inline float load_in(const ExpertArgs& a, const uint8_t* row, int k) {
    if (a.in_dtype == A2AV_F32) return ((const float*)row)[k];
    if (a.in_dtype == A2AV_BF16) return bf16_to_f32(((const u16*)row)[k]);
    return e4m3_to_f32(row[k]) * mx_scale(row[a.K + k / kMxGroup]);
}

__device__ inline float load_weight(const ExpertArgs& a, int64_t row, int k) {
    const uint8_t* p = a.weight + row * a.w_row;
    if (a.w_dtype == A2AV_F32) return ((const float*)p)[k];
    if (a.w_dtype == A2AV_BF16) return bf16_to_f32(((const u16*)p)[k]);
    const float s = mx_scale(a.scales[row * (a.K / kMxGroup) + k / kMxGroup]);
    if (a.w_dtype == A2AV_MX8) return e4m3_to_f32(p[k]) * s;
    return e2m1_to_f32((p[k / 2] >> (k % 2 * 4)) & 15u) * s;
}

constexpr int kGenThreads = 256;
constexpr int kGenM = 32, kGenN = 64, kGenK = 32;   // rows, weight rows and elements of a step

__global__ void __launch_bounds__(kGenThreads) expert_general_kernel(ExpertArgs a) {
    __shared__ int ends[kEntries];
    __shared__ int wave_sum[kGenThreads / kWave];
    __shared__ float xs[kGenM][kGenK + 1];
    __shared__ float ws[kGenN][kGenK + 1];
    __shared__ float res[kGenM][kGenN + 1];
    auto pieces = [](int rows) { return pieces_of(rows, kGenM); };
    const int each = groups_an_entry(a);
    const int mt = count_tiles<kGenThreads>(a, ends, wave_sum, pieces, each);
    const int cols = a.swiglu ? kGenN / 2 : kGenN;       // output columns of a tile
    const int nt = (a.width + cols - 1) / cols;
    const int tm = threadIdx.x / 16 * 2, tn = threadIdx.x % 16 * 4;
    for (int64_t t = blockIdx.x; t < (int64_t)mt * nt; t += gridDim.x) {
        const int col0 = (int)(t % nt) * cols;
        const Piece p = find_piece(a, ends, each, (int)(t / nt), pieces);
        const int g = p.group;
        const Group grp = p.rows;
        const int m0 = p.n * kGenM;
        const int rows = min(kGenM, grp.rows - m0);
        const uint8_t* in = a.in + (grp.row + m0) * a.in_row;
        uint8_t* out = a.out + (grp.row + m0) * a.out_row;
        const int width = min(cols, a.width - col0);
        float acc[2][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += kGenK) {
            for (int i = threadIdx.x; i < kGenM * kGenK; i += kGenThreads) {
                const int r = i / kGenK, k = k0 + i % kGenK;
                xs[r][i % kGenK] = r < rows && k < a.K ? load_in(a, in + r * a.in_row, k) : 0.0f;
            }
            for (int i = threadIdx.x; i < kGenN * kGenK; i += kGenThreads) {
                // with SwiGLU weight rows come in pairs: tile row 2c is column c's gate, 2c + 1 its up
                const int r = i / kGenK, k = k0 + i % kGenK;
                const int c = a.swiglu ? r / 2 : r;
                const int64_t wr = (int64_t)g * a.N + col0 + c + (a.swiglu && r % 2 ? a.width : 0);
                ws[r][i % kGenK] = c < width && k < a.K ? load_weight(a, wr, k) : 0.0f;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kGenK; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[tm + i][k], ws[tn + j][k], acc[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (a.swiglu) {
                    if (j % 2 == 0) res[tm + i][(tn + j) / 2] = silu_mul(acc[i][j], acc[i][j + 1]);
                } else {
                    res[tm + i][tn + j] = acc[i][j];
                }
            }
        __syncthreads();
        if (a.out_dtype != A2AV_MX8) {
            for (int i = threadIdx.x; i < kGenM * kGenN; i += kGenThreads) {
                const int r = i / kGenN, c = i % kGenN;
                if (r >= rows || c >= width) continue;
                uint8_t* p = out + r * a.out_row;
                if (a.out_dtype == A2AV_F32) ((float*)p)[col0 + c] = res[r][c];
                else ((u16*)p)[col0 + c] = (u16)f32_to_bf16(res[r][c]);
            }
        } else {
            // width is a multiple of 32, so is every tile's: one thread a scale
            const int groups = width / kMxGroup;
            for (int i = threadIdx.x; i < rows * groups; i += kGenThreads) {
                const int r = i / groups, c0 = i % groups * kMxGroup;
                uint32_t m = 0;
                for (int c = 0; c < kMxGroup; ++c) m = max(m, abs_bits(res[r][c0 + c]));
                const uint32_t sb = mx_scale_byte(m);
                const float f = mx_inverse(sb);
                uint8_t* p = out + r * a.out_row;
                for (int c = 0; c < kMxGroup; c += 4)
                    *(uint32_t*)(p + col0 + c0 + c) = mx8_pack(res[r][c0 + c] * f, res[r][c0 + c + 1] * f,
                                                               res[r][c0 + c + 2] * f, res[r][c0 + c + 3] * f, sb == 255u);
                p[a.width + (col0 + c0) / kMxGroup] = (uint8_t)sb;
            }
            const int used = a.width + a.width / kMxGroup, pad = (int)a.out_row - used;
            if (col0 + width == a.width)
                for (int i = threadIdx.x; i < rows * pad; i += kGenThreads) out[i / pad * a.out_row + used + i % pad] = 0;
        }
        __syncthreads();
    }
}

bool make_args(const a2av_matmul_t* c, ExpertArgs* a) {
    if (!c || c->num_ranks < 1 || c->experts_per_rank < 1) return false;
    if ((int64_t)c->num_ranks * c->experts_per_rank > kMaxExperts) return false;
    if (c->capacity_rows < 0 || c->capacity_rows > INT32_MAX / c->num_ranks) return false;   // rows are int32
    if (c->k < 1 || c->k > kMaxDim || c->n < 1 || c->n > kMaxDim) return false;
    const int32_t i = c->in_dtype, w = c->weight_dtype, o = c->out_dtype;
    const bool types = (i == A2AV_F32 && w == A2AV_F32 && o == A2AV_F32) ||
                       (i == A2AV_BF16 && (w == A2AV_BF16 || w == A2AV_MX4) && o == A2AV_BF16) ||
                       (i == A2AV_MX8 && (w == A2AV_MX8 || w == A2AV_MX4) && (o == A2AV_BF16 || o == A2AV_MX8));
    if (!types || (c->activation != A2AV_ACT_NONE && c->activation != A2AV_ACT_SWIGLU)) return false;
    const bool mx = w == A2AV_MX8 || w == A2AV_MX4;
    if (mx && c->k % kMxGroup != 0) return false;
    if (c->activation == A2AV_ACT_SWIGLU && c->n % 2 != 0) return false;
    const int32_t width = c->activation == A2AV_ACT_SWIGLU ? c->n / 2 : c->n;
    if (o == A2AV_MX8 && width % kMxGroup != 0) return false;
    a->cap = c->capacity_rows;
    a->in_row = a2av_row_bytes(i, c->k);
    a->w_row = w == A2AV_MX4 ? c->k / 2 : w == A2AV_MX8 ? c->k : a2av_row_bytes(w, c->k);
    a->out_row = a2av_row_bytes(o, width);
    a->R = c->num_ranks;
    a->epr = c->experts_per_rank;
    a->G = a->R * a->epr;
    a->K = c->k;
    a->N = c->n;
    a->width = width;
    a->in_dtype = i;
    a->w_dtype = w;
    a->out_dtype = o;
    a->swiglu = c->activation == A2AV_ACT_SWIGLU;
    return true;
}

size_t alignment_of(int32_t dtype) { return dtype == A2AV_F32 ? 4 : dtype == A2AV_BF16 ? 2 : 16; }

}  // namespace

hipError_t launch_experts_general(const ExpertArgs& a, int num_cu, hipStream_t st) {
    const int64_t mt = std::min<int64_t>((a.R * a.cap + kGenM - 1) / kGenM + a.G, INT32_MAX);
    const int cols = a.swiglu ? kGenN / 2 : kGenN;
    const int64_t tiles = mt * ((a.width + cols - 1) / cols);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, (int64_t)num_cu * 4);
    hipLaunchKernelGGL(expert_general_kernel, dim3(grid), dim3(kGenThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace a2av

extern "C" int a2av_expert_matmul(const a2av_matmul_t* cfg, const void* in, const int32_t* expert_offsets,
                                  const void* weight, const void* weight_scales, void* out, uint32_t* status,
                                  void* stream) {
    using namespace a2av;
    ExpertArgs a{};
    if (!make_args(cfg, &a) || !expert_offsets || !status) return A2AV_ERR_INVALID;
    if ((uintptr_t)status % 4 != 0 || (uintptr_t)expert_offsets % 4 != 0) return A2AV_ERR_INVALID;
    const bool mx = a.w_dtype == A2AV_MX8 || a.w_dtype == A2AV_MX4;
    if (!weight || mx != (weight_scales != nullptr)) return A2AV_ERR_INVALID;
    if (a.cap > 0 && (!in || !out)) return A2AV_ERR_INVALID;
    if ((uintptr_t)in % alignment_of(a.in_dtype) || (uintptr_t)weight % alignment_of(a.w_dtype) ||
        (uintptr_t)out % alignment_of(a.out_dtype))
        return A2AV_ERR_INVALID;
    // out apart from everything that is read
    const uintptr_t o = (uintptr_t)out, oe = o + (uintptr_t)(a.R * a.cap * a.out_row);
    auto meets = [&](const void* p, int64_t n) { return p && (uintptr_t)p < oe && o < (uintptr_t)p + (uintptr_t)n; };
    const int64_t wr = (int64_t)a.G * a.N;
    if (meets(in, a.R * a.cap * a.in_row) || meets(weight, wr * a.w_row) ||
        meets(weight_scales, wr * (a.K / kMxGroup)) || meets(expert_offsets, 4ll * a.R * (a.epr + 1)) || meets(status, 4))
        return A2AV_ERR_INVALID;
    if (a.cap == 0) return A2AV_OK;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return A2AV_ERR_HIP;
    a.in = (const uint8_t*)in;
    a.off = expert_offsets;
    a.weight = (const uint8_t*)weight;
    a.scales = (const uint8_t*)weight_scales;
    a.out = (uint8_t*)out;
    a.status = status;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (experts_mfma_takes(a)) {
        a.few = few_rows(a);
        a.tile_least = few_rows_all(a) ? cus / 2 : 0;
        e = launch_experts_few(a, cus, st);
        // a group of more rows needs a capacity of more, and a tile's worth of groups needs rows enough
        // (a group of r > few rows makes at most r / few row tiles)
        const int64_t most = a.cap > a.few ? a.R * a.cap / a.few : 0;
        const int cols = a.swiglu ? kTileRows / 2 : kTileRows;
        if (e == hipSuccess && most * ((a.width + cols - 1) / cols) >= std::max(a.tile_least, 1)) e = launch_experts_tile(a, cus, st);
    } else {
        e = launch_experts_general(a, cus, st);
    }
    return e == hipSuccess ? A2AV_OK : A2AV_ERR_HIP;
}
