// The experts' matrix products on expert-major receive rows (declared in include/a2av.h):
// out[r] = act(in[r] . weight_e^T) for every row r of every expert e, with the row counts
// read on the GPU.
//
// No host knows how many rows an expert got, so no grid can be cut to them: every block
// reads the group starts, counts the row tiles of every expert into LDS and walks the tile
// list (tile t, t + blocks, ...) until it ends.
// Here: the entry point, and the kernel for rows that are not whole 16-byte pieces.
#include "a2av_experts.h"

namespace a2av {
namespace {

constexpr int32_t kMaxDim = 1 << 20;

// ---- rows that are not whole 16-byte pieces ------------------------------------------
// float32 and bfloat16 rows of any length and address.  64 input rows by 64 weight rows a tile,
// 128 bytes of each a step: through registers into LDS, 16 bytes at a time wherever the row's
// elements lie (the memory takes such loads at any address).  What is left after a row's whole steps
// comes first.  The next two steps' loads run while a step is multiplied; 3, 4 and 6 in flight were no
// faster (8,192 bfloat16 rows x 4097 -> 2048 over 128 experts 0.84, 0.85, 0.84 and 0.87 ms, the
// whole-piece kernels 0.45 ms at 4096).
// With up to 16 rows a quarter of the products is made: 11 float32 rows x 1214 -> 104 take 21 us, all
// four 34.
[[maybe_unused]] constexpr int kGenThreads = 256;
[[maybe_unused]] constexpr int kGenRows = 64;             // input rows and weight rows of a tile
[[maybe_unused]] constexpr int kGenDepth = 2;             // steps whose loads are on their way

#ifdef A2AV_DEVICE_CODE
// The 16 bytes at `at` of a row of `bytes` bytes, zeros past its end: there the row's last 16 bytes,
// moved down.
template <typename T>
__device__ inline u32x4 row_piece(const uint8_t* row, int at, int bytes) {
    u32x4 v = {0, 0, 0, 0};
    if (at >= bytes) return v;
    if (bytes >= 16) {
        const int over = max(at + 16 - bytes, 0);
        uint64_t lo, hi;
        __builtin_memcpy(&lo, row + at - over, 8);
        __builtin_memcpy(&hi, row + at - over + 8, 8);
        const int by = 8 * (over % 8);
        if (over >= 8) lo = hi, hi = 0;
        if (by) lo = lo >> by | hi << (64 - by), hi >>= by;
        v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    } else if (at == 0) {
#pragma unroll 1
        for (int e = 0; e < bytes; e += sizeof(T)) {
            const uint32_t t = (uint32_t) * (const T*)(row + e) << (8 * (e % 4));
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] |= e / 4 == w ? t : 0;
        }
    }
    return v;
}
#endif

template <int KIND>
__global__ void __launch_bounds__(kGenThreads, 4) expert_general_kernel(ExpertArgs a) {
#ifdef A2AV_DEVICE_CODE
    using T = typename std::conditional<KIND == kF32, uint32_t, u16>::type;   // an element's bits
    __shared__ int ends[kEntries];
    __shared__ int wave_sum[kGenThreads / kWave];
    __shared__ __align__(16) uint8_t xs[kGenRows * 128], ws[kGenRows * 128];
    auto pieces = [](int rows) { return pieces_of(rows, kGenRows); };
    const int each = groups_an_entry(a);
    const int mt = count_tiles<kGenThreads>(a, ends, wave_sum, pieces, each);
    const int cols = a.swiglu ? kGenRows / 2 : kGenRows;     // output columns of a tile
    const int nt = (a.width + cols - 1) / cols;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, l16 = lane % 16, g = lane / 16;
    const int bytes = (int)a.in_row, whole = bytes / 128;
    // piece c of row r, so that eight rows' same pieces fall into different banks
    auto place = [](int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); };
    for (int64_t t = blockIdx.x; t < (int64_t)mt * nt; t += gridDim.x) {
        const int col0 = (int)(t % nt) * cols;
        const Piece p = find_piece(a, ends, each, (int)(t / nt), pieces);
        const int m0 = p.n * kGenRows, rows = min(kGenRows, p.rows.rows - m0);
        const uint8_t* in = a.in + (p.rows.row + m0) * a.in_row;
        uint8_t* out = a.out + (p.rows.row + m0) * a.out_row;
        const uint8_t* weight = a.weight + (int64_t)p.group * a.N * a.w_row;
        // this thread's pieces: rows threadIdx.x / 8 and 32 on.  With SwiGLU a wavefront's 16 weight
        // rows are 8 columns' gate rows and their up rows.
        const int c = threadIdx.x % 8;
        const uint8_t *xr[2], *wr[2];                        // past the last: the first, whose results are not written
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = threadIdx.x / 8 + 32 * i;
            xr[i] = in + (r < rows ? r : 0) * a.in_row;
            const int col = a.swiglu ? col0 + r / 16 * 8 + r % 8 : col0 + r;
            wr[i] = weight + (int64_t)(col >= a.width ? 0 : a.swiglu ? col + r / 8 % 2 * a.width : col) * a.w_row;
        }
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
        auto multiply = [&](const u32x4* xv, const u32x4* wv) __attribute__((always_inline)) {
            block_barrier();                                 // the step before has been read
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = threadIdx.x / 8 + 32 * i;
                *(u32x4*)(xs + place(r, c)) = xv[i];
                *(u32x4*)(ws + place(r, c)) = wv[i];
            }
            block_barrier();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4 w = *(const u32x4*)(ws + place(wave * 16 + l16, k * 4 + g));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i == 1 && rows <= 16) break;         // the other rows' results are not written
                    acc[i] = multiply16<KIND>(w, *(const u32x4*)(xs + place(i * 16 + l16, k * 4 + g)), acc[i]);
                }
            }
        };
        u32x4 xv[kGenDepth][2], wv[kGenDepth][2];
        // Past the last whole step the last one again: no condition, so that the waits for a step's
        // loads leave the later steps' loads on their way.
        auto load = [&](int s, int slot) __attribute__((always_inline)) {
            const int at = min(s, whole - 1) * 128 + c * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                __builtin_memcpy(&xv[slot][i], xr[i] + at, 16);
                __builtin_memcpy(&wv[slot][i], wr[i] + at, 16);
            }
        };
        u32x4 xt[2], wt[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {                        // what is left of the rows after the whole steps
            xt[i] = row_piece<T>(xr[i], whole * 128 + c * 16, bytes);
            wt[i] = row_piece<T>(wr[i], whole * 128 + c * 16, bytes);
        }
        if (whole > 0) {
#pragma unroll
            for (int j = 0; j < kGenDepth; ++j) load(j, j);
        }
        if (whole * 128 < bytes) multiply(xt, wt);
#pragma unroll 1
        for (int s = 0; s < whole; s += kGenDepth)
#pragma unroll
            for (int j = 0; j < kGenDepth; ++j) {
                if (s + j >= whole) {                        // zeros: no way out of the middle of the loop
#pragma unroll
                    for (int i = 0; i < 2; ++i) xv[j][i] = wv[j][i] = u32x4{0, 0, 0, 0};
                }
                multiply(xv[j], wv[j]);
                load(s + j + kGenDepth, j);
            }
        // lane (l16, g): columns 4g .. 4g + 3 of row l16; with SwiGLU lanes g >= 2 hold the ups
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 v = acc[i];
            int at = wave * 16 + 4 * g;
            bool on = true;
            if (a.swiglu) {
                at = wave * 8 + 4 * g;
                on = g < 2;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], __shfl_xor(acc[i][e], 32));
            }
            const int row = i * 16 + l16;
            uint8_t* to = out + row * a.out_row;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = col0 + at + e;
                if (!on || row >= rows || col >= a.width) continue;
                if constexpr (KIND == kF32) ((float*)to)[col] = v[e];
                else ((u16*)to)[col] = (u16)f32_to_bf16(v[e]);
            }
        }
    }
#endif
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
    if (c->n * (w == A2AV_MX4 ? c->k / 2 : w == A2AV_MX8 ? (int64_t)c->k : a2av_row_bytes(w, c->k)) > INT32_MAX) return false;
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
    const int64_t mt = std::min<int64_t>(a.R * a.cap / kGenRows + a.G, INT32_MAX);
    const int cols = a.swiglu ? kGenRows / 2 : kGenRows;
    const int64_t tiles = mt * ((a.width + cols - 1) / cols);
    const dim3 grid((unsigned)std::min<int64_t>(tiles, (int64_t)num_cu * 4));
    if (kind_of(a) == kF32) hipLaunchKernelGGL((expert_general_kernel<kF32>), grid, dim3(kGenThreads), 0, st, a);
    else hipLaunchKernelGGL((expert_general_kernel<kBf16>), grid, dim3(kGenThreads), 0, st, a);
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
    if (experts_whole_pieces(a)) {
        a.few = few_rows(a);
        a.tile_least = std::max(cus / 2, 1);
        e = launch_experts_few(a, cus, st);
        // a group of more rows needs a capacity of more, and a tile's worth of groups needs rows enough
        // (a group of r > few rows makes at most r / few row tiles)
        const int64_t most = a.cap > a.few ? a.R * a.cap / a.few : 0;
        const int cols = a.swiglu ? kTileRows / 2 : kTileRows;
        if (e == hipSuccess && most * ((a.width + cols - 1) / cols) >= a.tile_least) e = launch_experts_tile(a, cus, st);
    } else {
        e = launch_experts_general(a, cus, st);
    }
    return e == hipSuccess ? A2AV_OK : A2AV_ERR_HIP;
}
