// ep_expert.hip — the expert products between dispatch and combine, in 8 bits.
//
// Rows are 8-bit rows as the dispatch packs them (codes and a float scale per
// 128 of them), grouped by expert; an expert's weights are e4m3 codes [N, K]
// with a float scale per 128 x 128 block:
//   y[m,n] = sum over blocks b of K of
//              sx[m,b] * sw[n/128,b] * sum_{k in b} x[m,k] * w[n,k]
// ep_expert_product stores y in bf16.  ep_expert_gate_up has 2F columns, a
// gate and an up for each of F outputs, and stores silu(gate) * up as 8-bit
// rows, ready for the second product.
//
// One MFMA takes a whole block of K (16 x 16 x 128): its result, from a zero
// accumulator, is multiplied by the two scales and added in float.  The
// weights are its first operand and the rows its second, so a lane's four
// results are four neighbouring columns of one row: one row scale a lane, and
// stores of 8 bytes.  (The unit aligns each eight products to their largest
// and drops what falls 13 bits below it, 1.4e-5 of a random sum; between those
// eights and between blocks the sum is float.)

#include "ep_rows8.h"

namespace ep {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct ExpertArgs {
    const uint8_t* rows;
    const int32_t* group_offset;   // [G+1]
    const uint8_t* w;              // [G, N, K]
    const float* w_scale;          // [G, ceil(N/128), K/128]
    uint8_t* out;
    int32_t* st;
    int64_t M;                     // rows that `rows` and `out` hold
    int32_t G, N, K, row_bytes, out_bytes, n_tiles;
};

// The rows of tile `tile` of `bm` rows, tiles counted over the groups in order.
struct RowTile {
    int32_t g;        // group; -1: no such tile
    int64_t first;    // first row of the tile
    int32_t count;    // its rows, 1 .. bm
};

__device__ inline int64_t clamp_row(int64_t r, int64_t M) { return r < 0 ? 0 : r > M ? M : r; }

// Called by whole wavefronts: lane l looks at group g0 + l, 64 groups a step.
// Offsets outside [0, M] or decreasing are clamped, so that a tile's rows are
// always rows of the buffers (check_groups reports them).
__device__ inline RowTile find_tile(const int32_t* off, int G, int64_t M, int64_t tile, int bm) {
    RowTile r{-1, 0, 0};
    const int lane = lane_id();
    int64_t before = 0;   // tiles of the groups before g0
    for (int g0 = 0; g0 < G; g0 += kWave) {
        const int g = g0 + lane;
        int64_t lo = 0, n = 0;
        if (g < G) {
            lo = clamp_row(off[g], M);
            n = clamp_row(off[g + 1], M) - lo;
            n = n < 0 ? 0 : n;
        }
        const int t = (int)((n + bm - 1) / bm);
        int sum = t;   // inclusive scan: at most M < 2^31 tiles where the offsets are in order
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) {
            const int up = __shfl_up(sum, o);
            sum += lane >= o ? up : 0;
        }
        const uint64_t here = __ballot(tile < before + sum);
        if (here) {
            const int l = __builtin_ctzll(here);
            const int in = (int)(tile - before) - (bcast(sum, l) - bcast(t, l));
            // overlapping groups can wrap the sum: such a tile is left out
            if (in < 0 || in >= bcast(t, l)) return r;
            r.g = g0 + l;
            r.first = (int64_t)bcast((int32_t)lo, l) + (int64_t)in * bm;
            const int64_t left = (int64_t)bcast((int32_t)n, l) - (int64_t)in * bm;
            r.count = (int)(left < bm ? left : bm);
            return r;
        }
        before += bcast(sum, kWave - 1);
    }
    return r;
}

// Decreasing or negative offsets, and rows beyond M, by the first workgroup.
__device__ inline void check_groups(const ExpertArgs& a) {
    for (int g = (int)threadIdx.x; g <= a.G; g += (int)blockDim.x) {
        const int32_t o = a.group_offset[g];
        if (o < 0 || (g > 0 && o < a.group_offset[g - 1])) set_error(a.st, EP_ERR_INVALID_ARG);
        if (o > a.M) set_error(a.st, EP_ERR_CAPACITY);
    }
}

__device__ inline i32x8 join(i32x4 lo, i32x4 hi) {
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// D = A B of one 16 x 16 x 128 block, all block exponents one (127).  Lane l
// gives 32 codes of row l % 16 of A and of column l % 16 of B; which 32 of the
// 128 is the same for both.  D: rows 4 (l / 16) + i, column l % 16.
__device__ inline f32x4 mfma16(i32x8 a, i32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0,
                                                            0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}

__device__ inline f32x4 fma4(f32x4 v, float s, f32x4 acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(v[i], s, acc[i]);
    return acc;
}

__device__ inline i32x4 load16(const uint8_t* p) { return *reinterpret_cast<const i32x4*>(p); }

// Adds blocks [b0, b1) of 16 weight rows times MT x 16 rows to acc.  wrow: this
// lane's weight row; xrow[j]: its rows of the second operand; both in bounds.
template <int MT>
__device__ inline void stream_blocks(const uint8_t* wrow, const float* sw,
                                     const uint8_t* const* xrow, int K, int b0, int b1,
                                     f32x4* acc) {
    const int g = lane_id() / 16 * 16;
    for (int b = b0; b < b1; ++b) {
        const int k = b * kScaleBlock + g;
        const i32x8 w = join(load16(wrow + k), load16(wrow + k + 64));
        const float s = sw[b];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const i32x8 x = join(load16(xrow[j] + k), load16(xrow[j] + k + 64));
            const float sx = reinterpret_cast<const float*>(xrow[j] + K)[b];
            acc[j] = fma4(mfma16(w, x), s * sx, acc[j]);
        }
    }
}

// Few rows a group: the weights are read once, straight from memory to
// registers.  A workgroup has 16 weight rows and MT x 16 rows; its four
// wavefronts split K and join in LDS in their order.
template <int MT>
__global__ __launch_bounds__(256) void product_small_kernel(ExpertArgs a) {
    __shared__ f32x4 s_acc[4][MT][kWave];
    if (blockIdx.x == 0) check_groups(a);
    const int nt = (int)(blockIdx.x % (unsigned)a.n_tiles);
    const RowTile tile =
        find_tile(a.group_offset, a.G, a.M, blockIdx.x / (unsigned)a.n_tiles, 16 * MT);
    if (tile.g < 0) return;
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int n0 = nt * 16, nb = a.K / kScaleBlock;
    // rows behind the last weight row or the tile's last row repeat the last
    // one: their results are not stored
    const int n = n0 + lane % 16 < a.N ? n0 + lane % 16 : a.N - 1;
    const uint8_t* wrow = a.w + ((int64_t)tile.g * a.N + n) * a.K;
    const float* sw = a.w_scale + ((int64_t)tile.g * ((a.N + 127) / 128) + n0 / 128) * nb;
    const uint8_t* xrow[MT];
    f32x4 acc[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int m = j * 16 + lane % 16;
        xrow[j] = a.rows + (tile.first + (m < tile.count ? m : tile.count - 1)) * a.row_bytes;
        acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    stream_blocks<MT>(wrow, sw, xrow, a.K, nb * wave / 4, nb * (wave + 1) / 4, acc);
#pragma unroll
    for (int j = 0; j < MT; ++j) s_acc[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < MT; j += 4) {
        const f32x4 v =
            ((s_acc[0][j][lane] + s_acc[1][j][lane]) + s_acc[2][j][lane]) + s_acc[3][j][lane];
        const int m = j * 16 + lane % 16, c = n0 + lane / 16 * 4;
        if (m < tile.count && c < a.N)   // N is a multiple of 8: all four columns or none
            *reinterpret_cast<u32x2*>(a.out + (tile.first + m) * a.out_bytes + 2 * c) =
                u32x2{bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3])};
    }
}

__device__ inline float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// One thread's eight outputs of row `m`: quantised with the block's other
// lanes (16 neighbouring lanes hold a block of 128).
__device__ inline void store_block(const ExpertArgs& a, int64_t m, int fb, const float* h, bool on) {
    const int F = a.N / 2, sub = lane_id() % 16;
    const float am = fmaxf(group_max<16>(amax8(h)), kAmaxMin);
    if (!on) return;
    uint8_t* row = a.out + m * a.out_bytes;
    *reinterpret_cast<u32x2*>(row + fb * kScaleBlock + sub * 8) = fp8_pack8(h, kFp8Max / am);
    if (sub == 0) *reinterpret_cast<float*>(row + F + 4 * fb) = am / kFp8Max;
    if (fb == F / kScaleBlock - 1)   // the row's last block also writes the zero pad
        for (int o = F + F / 32 + 4 * sub; o < a.out_bytes; o += 64)
            *reinterpret_cast<uint32_t*>(row + o) = 0u;
}

// Few rows a group, with the gate: a workgroup has the 128 gates and 128 ups
// of one output block and MT x 16 rows; wavefront w has 16 of those weight
// rows over all of K.
template <int MT>
__global__ __launch_bounds__(1024) void gate_up_small_kernel(ExpertArgs a) {
    constexpr int kPitch = 2 * kScaleBlock + 4;
    __shared__ float s_y[16 * MT][kPitch];
    if (blockIdx.x == 0) check_groups(a);
    const int fb = (int)(blockIdx.x % (unsigned)a.n_tiles);
    const RowTile tile =
        find_tile(a.group_offset, a.G, a.M, blockIdx.x / (unsigned)a.n_tiles, 16 * MT);
    if (tile.g < 0) return;
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int F = a.N / 2, nb = a.K / kScaleBlock;
    const int n0 = (wave < 8 ? 0 : F) + fb * kScaleBlock + wave % 8 * 16;
    const uint8_t* wrow = a.w + ((int64_t)tile.g * a.N + n0 + lane % 16) * a.K;
    const float* sw = a.w_scale + ((int64_t)tile.g * (a.N / 128) + n0 / 128) * nb;
    const uint8_t* xrow[MT];
    f32x4 acc[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int m = j * 16 + lane % 16;
        xrow[j] = a.rows + (tile.first + (m < tile.count ? m : tile.count - 1)) * a.row_bytes;
        acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    stream_blocks<MT>(wrow, sw, xrow, a.K, 0, nb, acc);
#pragma unroll
    for (int j = 0; j < MT; ++j)
        *reinterpret_cast<f32x4*>(&s_y[j * 16 + lane % 16][wave * 16 + lane / 16 * 4]) = acc[j];
    __syncthreads();
    // 16 lanes a row, eight outputs each
    for (int m = (int)threadIdx.x / 16; m < 16 * MT; m += 64) {
        const float* y = &s_y[m][lane % 16 * 8];
        float h[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) h[q] = silu_mul(y[q], y[kScaleBlock + q]);
        store_block(a, tile.first + m, fb, h, m < tile.count);
    }
}

// Shared by both calls: shapes whose indexes the kernels hold in 32 bits.
int check_expert(int32_t G, int64_t M, int32_t N, int32_t K) {
    if (G < 1 || G > kMaxE || M < 0 || M >= ((int64_t)1 << 31)) return EP_ERR_INVALID_ARG;
    if (K < kScaleBlock || K % kScaleBlock != 0 || K > kMaxH) return EP_ERR_INVALID_ARG;
    if (N < 8 || N % 8 != 0 || N > kMaxH) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Row tiles of bm rows that M rows in G groups can need at most.
inline int64_t max_tiles(int64_t M, int32_t G, int bm) {
    return M / bm + (G < M ? (int64_t)G : M);
}

}  // namespace ep

using namespace ep;

namespace {
int expert_args(ExpertArgs& a, int32_t G, int64_t M, int32_t N, int32_t K, const void* rows,
                const int32_t* group_offset, const void* w, const float* w_scale, void* out,
                int32_t* dev_status) {
    if (!dev_status || !group_offset || !w || !w_scale) return EP_ERR_INVALID_ARG;
    if (M > 0 && (!rows || !out)) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)rows | (uintptr_t)w | (uintptr_t)out) & 15) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)w_scale | (uintptr_t)group_offset | (uintptr_t)dev_status) & 3)
        return EP_ERR_INVALID_ARG;
    a.rows = reinterpret_cast<const uint8_t*>(rows);
    a.group_offset = group_offset;
    a.w = reinterpret_cast<const uint8_t*>(w);
    a.w_scale = w_scale;
    a.out = reinterpret_cast<uint8_t*>(out);
    a.st = dev_status;
    a.M = M;
    a.G = G;
    a.N = N;
    a.K = K;
    a.row_bytes = (int32_t)row_bytes(K, EP_FMT_FP8_E4M3_B128);
    return EP_OK;
}

// Workgroups of a launch: column tiles x the row tiles that there can be.
int grid_of(const ExpertArgs& a, int bm, unsigned* blocks) {
    const int64_t n = max_tiles(a.M, a.G, bm) * a.n_tiles;
    if (n >= ((int64_t)1 << 31)) {
        record_error("expert product: more than 2^31 tiles");
        return EP_ERR_INVALID_ARG;
    }
    *blocks = (unsigned)n;
    return EP_OK;
}

#define EP_LAUNCH_TILES(KERNEL, BM, THREADS)                                               \
    do {                                                                                   \
        unsigned blocks = 0;                                                               \
        const int v_ = grid_of(a, BM, &blocks);                                            \
        if (v_ != EP_OK) return v_;                                                        \
        clear_hip_error();                                                                 \
        hipLaunchKernelGGL((KERNEL), dim3(blocks), dim3(THREADS), 0, stream, a);           \
        EP_HIP_CHECK(hipGetLastError());                                                   \
        return EP_OK;                                                                      \
    } while (0)
}  // namespace

extern "C" int ep_expert_product(int32_t G, int64_t M, int32_t N, int32_t K, const void* rows,
                                 const int32_t* group_offset, const void* w, const float* w_scale,
                                 void* out, int32_t* dev_status, hipStream_t stream) {
    int v = check_expert(G, M, N, K);
    if (v != EP_OK) return v;
    ExpertArgs a{};
    v = expert_args(a, G, M, N, K, rows, group_offset, w, w_scale, out, dev_status);
    if (v != EP_OK) return v;
    if (M == 0) return EP_OK;
    a.out_bytes = 2 * N;
    a.n_tiles = (int32_t)ceil_div(N, 16);
    const int64_t per = ceil_div(M, G);   // rows a group, were they even
    if (per <= 16) EP_LAUNCH_TILES(product_small_kernel<1>, 16, 256);
    if (per <= 32) EP_LAUNCH_TILES(product_small_kernel<2>, 32, 256);
    EP_LAUNCH_TILES(product_small_kernel<4>, 64, 256);
}

extern "C" int ep_expert_gate_up(int32_t G, int64_t M, int32_t F, int32_t K, const void* rows,
                                 const int32_t* group_offset, const void* w, const float* w_scale,
                                 void* out_rows, int32_t* dev_status, hipStream_t stream) {
    if (F < kScaleBlock || F % kScaleBlock != 0 || F > kMaxH / 2) return EP_ERR_INVALID_ARG;
    int v = check_expert(G, M, 2 * F, K);
    if (v != EP_OK) return v;
    ExpertArgs a{};
    v = expert_args(a, G, M, 2 * F, K, rows, group_offset, w, w_scale, out_rows, dev_status);
    if (v != EP_OK) return v;
    if (M == 0) return EP_OK;
    a.out_bytes = (int32_t)row_bytes(F, EP_FMT_FP8_E4M3_B128);
    a.n_tiles = F / kScaleBlock;
    const int64_t per = ceil_div(M, G);
    if (per <= 16) EP_LAUNCH_TILES(gate_up_small_kernel<1>, 16, 1024);
    if (per <= 32) EP_LAUNCH_TILES(gate_up_small_kernel<2>, 32, 1024);
    EP_LAUNCH_TILES(gate_up_small_kernel<4>, 64, 1024);
}
