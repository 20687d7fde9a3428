// ep_norm.hip — root-mean-square norm with the residual's addition, the output
// in bf16 and in 8-bit rows, and its backward.
//
// Forward, per row of H values:
//   r = bf16(x + residual)                      (r = x without a residual)
//   y = r * rsqrt(mean(r^2) + eps) * weight
// with y stored as bf16, as an 8-bit row (codes and per-128 scales, the form
// that the dispatch sends), or both.  y goes from float straight to each form:
// one rounding each.  The statistics are those of the stored r, so a backward
// that reads r sees what the forward normalised.
//
// Backward, with h = r * rstd and g = grad_y * weight:
//   grad_x = rstd * (g - h * mean(g * h)) + grad_residual
//   grad_weight = sum over rows of grad_y * h
//
// Both are bound by memory: a row is read once into registers, its sum taken
// across the row's threads, and written once.  16384 x 7168 with a residual,
// bf16 and 8-bit outputs (1.06 GB): 194 us, 5.5 TB/s; the backward of 4096 x 7168
// with a residual's gradient (235 MB): 49 us, 4.8 TB/s, and 5 us for the sum of
// the weight gradient's parts.

#include "ep_rows8.h"

namespace ep {

constexpr int kNormMaxH = 32768;        // 1024 threads x 4 vectors of 8
constexpr int kNormBackBlocks = 512;    // workgroups, and partial sums, of a backward

struct NormArgs {
    const u32x4* x;
    const u32x4* residual;
    const f32x4* weight;
    u32x4* residual_out;
    u32x4* y;
    uint8_t* rows;
    float* rstd;
    float eps, inv_h;
    int32_t T, H, nv, row_bytes;
};

// Sum over the threads of a row.  TPR threads hold it: within a wavefront
// (16 or 64), or, TPR = 0, all the workgroup's wavefronts, which meet in LDS.
// `turn` alternates between two LDS slots, so that one barrier a row suffices:
// a wavefront writes a slot again only after the barrier of the row between.
template <int TPR>
__device__ inline float row_sum(float v, int turn) {
    if constexpr (TPR != 0) {
        return group_sum<TPR>(v);
    } else {
        v = group_sum<64>(v);
        __shared__ float s_part[2][16];
        const int nw = (int)(blockDim.x / kWave);
        if (lane_id() == 0) s_part[turn][threadIdx.x / kWave] = v;
        __syncthreads();
        float s = 0.0f;
        for (int w = 0; w < nw; ++w) s += s_part[turn][w];
        return s;
    }
}

// V vectors of 8 values a thread, TPR threads a row (0: the workgroup).
template <int V, int TPR>
__global__ __launch_bounds__(TPR ? 256 : 1024) void norm_kernel(NormArgs a) {
    const int tpr = TPR ? TPR : (int)blockDim.x;
    const int rpb = TPR ? 256 / TPR : 1;
    const int tid = TPR ? (int)threadIdx.x % TPR : (int)threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + (TPR ? (int)threadIdx.x / TPR : 0);

    bool on[V];
    float w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vi = tid + i * tpr;
        on[i] = vi < a.nv;
#pragma unroll
        for (int q = 0; q < 8; ++q) w[i][q] = 0.0f;
        if (on[i]) {
            const f32x4 w0 = a.weight[2 * vi], w1 = a.weight[2 * vi + 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[i][q] = w0[q];
                w[i][4 + q] = w1[q];
            }
        }
    }

    // TPR = 0: every thread of the workgroup has the same row, so the loop and
    // its barriers are uniform; otherwise there is no barrier.
    int turn = 0;
    for (; row < a.T; row += step, turn ^= 1) {
        const int64_t base = row * a.nv;
        u32x4 r[V];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int vi = tid + i * tpr;
            r[i] = on[i] ? a.x[base + vi] : u32x4{0, 0, 0, 0};
        }
        if (a.residual) {
            u32x4 e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int vi = tid + i * tpr;
                e[i] = on[i] ? a.residual[base + vi] : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8], g[8];
                unpack8(r[i], f);
                unpack8(e[i], g);
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] += g[q];
                r[i] = pack8(f);
            }
            if (a.residual_out) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int vi = tid + i * tpr;
                    if (on[i]) a.residual_out[base + vi] = r[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            unpack8(r[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) ss = fmaf(f[q], f[q], ss);
        }
        ss = row_sum<TPR>(ss, turn);
        const float rstd = 1.0f / sqrtf(fmaf(ss, a.inv_h, a.eps));
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
        uint8_t* const out8 = a.rows + row * a.row_bytes;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int vi = tid + i * tpr;
            float f[8];
            unpack8(r[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = f[q] * rstd * w[i][q];
            if (a.y && on[i]) a.y[base + vi] = pack8(f);
            if (a.rows) {
                // a block is 16 neighbouring lanes: nv and tpr are multiples of 16
                const float am = fmaxf(group_max<16>(amax8(f)), kAmaxMin);
                if (on[i]) {
                    *reinterpret_cast<u32x2*>(out8 + vi * 8) = fp8_pack8(f, kFp8Max / am);
                    if ((vi & 15) == 0)
                        *reinterpret_cast<float*>(out8 + a.H + vi / 4) = am / kFp8Max;
                }
            }
        }
        if (a.rows)
            for (int o = a.H + a.H / 32 + 4 * tid; o < a.row_bytes; o += 4 * tpr)
                *reinterpret_cast<uint32_t*>(out8 + o) = 0u;
    }
}

struct NormBackArgs {
    const u32x4* r;
    const f32x4* weight;
    const float* rstd;
    const u32x4* grad_y;
    const u32x4* grad_residual;
    u32x4* grad_x;
    f32x4* part;     // [gridDim.x * rows per workgroup .. ] partial sums of grad_weight, [blocks, H]
    float inv_h;
    int32_t T, nv;
};

// Each workgroup takes every gridDim.x-th row and keeps its columns' sums of
// grad_y * h in registers; they leave as one row of `part` at the end.
template <int V>
__global__ __launch_bounds__(1024) void norm_back_kernel(NormBackArgs a) {
    const int tpr = (int)blockDim.x, tid = (int)threadIdx.x;
    bool on[V];
    float w[V][8], acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vi = tid + i * tpr;
        on[i] = vi < a.nv;
#pragma unroll
        for (int q = 0; q < 8; ++q) w[i][q] = acc[i][q] = 0.0f;
        if (on[i]) {
            const f32x4 w0 = a.weight[2 * vi], w1 = a.weight[2 * vi + 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[i][q] = w0[q];
                w[i][4 + q] = w1[q];
            }
        }
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const int64_t base = row * a.nv;
        const float rstd = a.rstd[row];
        u32x4 r[V], d[V], e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int vi = tid + i * tpr;
            r[i] = on[i] ? a.r[base + vi] : u32x4{0, 0, 0, 0};
            d[i] = on[i] ? a.grad_y[base + vi] : u32x4{0, 0, 0, 0};
            e[i] = (on[i] && a.grad_residual) ? a.grad_residual[base + vi] : u32x4{0, 0, 0, 0};
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8], g[8];
            unpack8(r[i], f);
            unpack8(d[i], g);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float h = f[q] * rstd;
                acc[i][q] = fmaf(g[q], h, acc[i][q]);
                s = fmaf(g[q] * w[i][q], h, s);
            }
        }
        const float mean = row_sum<0>(s, turn) * a.inv_h;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int vi = tid + i * tpr;
            float f[8], g[8], z[8];
            unpack8(r[i], f);
            unpack8(d[i], g);
            unpack8(e[i], z);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                z[q] = fmaf(rstd, fmaf(-f[q] * rstd, mean, g[q] * w[i][q]), z[q]);
            if (on[i]) a.grad_x[base + vi] = pack8(z);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int vi = tid + i * tpr;
        if (on[i]) {
            f32x4* p = a.part + ((int64_t)blockIdx.x * a.nv + vi) * 2;
            p[0] = f32x4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
            p[1] = f32x4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
        }
    }
}

// Column sums of `part` [n, H] in a fixed order: 16 threads of 4 columns, 64
// slices of the rows, joined in LDS.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const f32x4* part, int n, int H4,
                                                           f32x4* out) {
    __shared__ f32x4 s[64][16];
    const int c = (int)threadIdx.x % 16, g = (int)threadIdx.x / 16;
    const int col = (int)blockIdx.x * 16 + c;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < H4)
#pragma unroll 8
        for (int b = g; b < n; b += 64) v += part[(int64_t)b * H4 + col];
    s[g][c] = v;
    __syncthreads();
    if (g < 8) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[g + 8 * i][c];
        s[g][c] = v;
    }
    __syncthreads();
    if (g == 0 && col < H4) {
        for (int i = 1; i < 8; ++i) v += s[i][c];
        out[col] = v;
    }
}

int check_norm(int32_t T, int32_t H) {
    if (T < 0 || H < 8 || H % 8 != 0) return EP_ERR_INVALID_ARG;
    if (H > kNormMaxH) {
        record_error("ep_rmsnorm: H > 32768");
        return EP_ERR_INVALID_ARG;
    }
    return EP_OK;
}

inline int back_blocks(int32_t T) { return T < kNormBackBlocks ? T : kNormBackBlocks; }

// Threads of a row that a workgroup shares, V vectors each.
inline int row_threads(int nv, int V) { return (int)(ceil_div(ceil_div(nv, V), kWave) * kWave); }

}  // namespace ep

using namespace ep;

namespace {
template <int V, int TPR>
int launch_norm(const NormArgs& a, hipStream_t stream) {
    const int rpb = TPR ? 256 / TPR : 1;
    const int64_t blocks = ceil_div(a.T, rpb);
    const int threads = TPR ? 256 : row_threads(a.nv, V);
    clear_hip_error();
    hipLaunchKernelGGL((norm_kernel<V, TPR>), dim3(loop_grid(blocks, threads)),
                       dim3((unsigned)threads), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

template <int V>
int launch_norm_back(const NormBackArgs& a, int blocks, hipStream_t stream) {
    hipLaunchKernelGGL((norm_back_kernel<V>), dim3((unsigned)blocks),
                       dim3((unsigned)row_threads(a.nv, V)), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}
}  // namespace

extern "C" int ep_rmsnorm(int32_t T, int32_t H, const void* x, const void* residual,
                          const float* weight, float eps, void* residual_out, void* y, void* rows,
                          float* rstd, hipStream_t stream) {
    int v = check_norm(T, H);
    if (v != EP_OK) return v;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return EP_ERR_INVALID_ARG;
    if (rows && H % kScaleBlock != 0) return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (residual_out && !residual) return EP_ERR_INVALID_ARG;
    if (!y && !rows) return EP_ERR_INVALID_ARG;
    if (!x || !weight) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)residual_out |
         (uintptr_t)y | (uintptr_t)rows) & 15)
        return EP_ERR_INVALID_ARG;
    if ((uintptr_t)rstd & 3) return EP_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = reinterpret_cast<const u32x4*>(x);
    a.residual = reinterpret_cast<const u32x4*>(residual);
    a.weight = reinterpret_cast<const f32x4*>(weight);
    a.residual_out = reinterpret_cast<u32x4*>(residual_out);
    a.y = reinterpret_cast<u32x4*>(y);
    a.rows = reinterpret_cast<uint8_t*>(rows);
    a.rstd = rstd;
    a.eps = eps;
    a.inv_h = 1.0f / (float)H;
    a.T = T;
    a.H = H;
    a.nv = H / 8;
    a.row_bytes = rows ? (int32_t)row_bytes(H, EP_FMT_FP8_E4M3_B128) : 0;
    if (a.nv <= 16) return launch_norm<1, 16>(a, stream);
    if (a.nv <= 64) return launch_norm<1, 64>(a, stream);
    if (a.nv <= 1024) return launch_norm<1, 0>(a, stream);
    return a.nv <= 2048 ? launch_norm<2, 0>(a, stream) : launch_norm<4, 0>(a, stream);
}

extern "C" size_t ep_rmsnorm_workspace_bytes(int32_t T, int32_t H) {
    if (check_norm(T, H) != EP_OK) return 0;
    return (size_t)back_blocks(T) * H * sizeof(float);
}

extern "C" int ep_rmsnorm_backward(int32_t T, int32_t H, const void* r, const float* weight,
                                   const float* rstd, const void* grad_y,
                                   const void* grad_residual, void* grad_x, float* grad_weight,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int v = check_norm(T, H);
    if (v != EP_OK) return v;
    if (!grad_weight || ((uintptr_t)grad_weight & 15)) return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!r || !weight || !rstd || !grad_y || !grad_x || !workspace) return EP_ERR_INVALID_ARG;
        if (((uintptr_t)r | (uintptr_t)weight | (uintptr_t)grad_y | (uintptr_t)grad_residual |
             (uintptr_t)grad_x | (uintptr_t)workspace) & 15)
            return EP_ERR_INVALID_ARG;
        if ((uintptr_t)rstd & 3) return EP_ERR_INVALID_ARG;
        if (workspace_bytes < ep_rmsnorm_workspace_bytes(T, H)) return EP_ERR_INVALID_ARG;
    }
    const int blocks = back_blocks(T), H4 = H / 4;
    clear_hip_error();
    if (T > 0) {
        NormBackArgs a{};
        a.r = reinterpret_cast<const u32x4*>(r);
        a.weight = reinterpret_cast<const f32x4*>(weight);
        a.rstd = rstd;
        a.grad_y = reinterpret_cast<const u32x4*>(grad_y);
        a.grad_residual = reinterpret_cast<const u32x4*>(grad_residual);
        a.grad_x = reinterpret_cast<u32x4*>(grad_x);
        a.part = reinterpret_cast<f32x4*>(workspace);
        a.inv_h = 1.0f / (float)H;
        a.T = T;
        a.nv = H / 8;
        v = a.nv <= 1024   ? launch_norm_back<1>(a, blocks, stream)
            : a.nv <= 2048 ? launch_norm_back<2>(a, blocks, stream)
                           : launch_norm_back<4>(a, blocks, stream);
        if (v != EP_OK) return v;
    }
    hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)ceil_div(H4, 16)), dim3(1024), 0, stream,
                       reinterpret_cast<const f32x4*>(workspace), blocks, H4,
                       reinterpret_cast<f32x4*>(grad_weight));
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}
