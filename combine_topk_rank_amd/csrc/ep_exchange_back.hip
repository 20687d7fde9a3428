// ep_exchange_back.hip — the gradients of combine and dispatch, in both layouts
// (per rank and per expert).
//
// Combine: out[t] = sum over t's rows s of W_s y[s], W_s the sum of the gates of
// the choices that s serves (per expert: the one choice's gate).  So
//   grad_y[s]        = W_s * grad_out[t]
//   grad_topk_w[t,j] = <grad_out[t], y[s]>  for the row s that serves choice j
// Dispatch copies x[t] to each of t's rows and the gates beside them.  So
//   grad_x[t]        = grad_other[t] + sum over t's rows s of grad_rows[s]
//   grad_topk_w[t,j] = gradient of the gate that went with row s for choice j
// Sums are float; each output is rounded once.

#include "ep_rows8.h"

namespace ep {

struct ExchangeBackArgs {
    const int32_t* idx;       // [T, k]
    const float* w;           // [T, k]
    const int32_t* slot;      // [T, R], or, per expert, [T, k]
    const u32x4* y;           // combine: y; dispatch: grad_rows
    const u32x4* grad_out;    // combine: grad_out; dispatch: grad_other
    const float* grad_gates;  // dispatch: [rows, k], or, per expert, [rows]
    u32x4* out;               // combine: grad_y; dispatch: grad_x
    float* grad_w;            // [T, k]
    int32_t* st;
    int64_t rows;
    int32_t T, E, R, k, epr, nv, per;   // per: wavefronts a token
};

// The rows of a token: lane i has row i's slot (rank i's, or choice i's), or -1.
template <bool LL>
__device__ inline int32_t token_slot(const ExchangeBackArgs& a, int64_t t, int lane) {
    int32_t s = -1;
    if (LL) {
        if (lane < a.k) {
            const int e = a.idx[t * a.k + lane];
            if (e >= 0 && e < a.E) s = a.slot[t * a.k + lane];
        }
    } else if (lane < a.R) {
        s = a.slot[t * a.R + lane];
    }
    if (s >= a.rows) {
        set_error(a.st, EP_ERR_CAPACITY);   // beyond the rows of the buffers: skipped
        s = -1;
    }
    return s;
}

// Combine.  A wavefront has one row of one token (row i of the token's rows, in
// their order): it reads the row of y and the token's gradient (which the
// token's other wavefronts, its neighbours, read too: it stays in cache), and
// writes the row of grad_y.  V vectors of 8 a lane are under way at a time.  Bound by
// memory: 4096 tokens of 7168, 8 of 256 experts on 32 ranks (28 400 rows, 874 MB): 162 us,
// 5.4 TB/s (with plain loads and stores of the rows 179).
template <int V, bool LL, bool GY, bool GW>
__global__ __launch_bounds__(kBlock) void combine_back_kernel(ExchangeBackArgs a) {
    const int lane = lane_id();
    const int64_t waves = (int64_t)a.T * a.per;
    const int64_t step = (int64_t)gridDim.x * (kBlock / kWave);
    for (int64_t gw = (int64_t)blockIdx.x * (kBlock / kWave) +
                      __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
         gw < waves; gw += step) {
        const int64_t t = (uint32_t)gw / (uint32_t)a.per;   // T * max(k, R) < 2^31
        const int i = (int)(gw - t * a.per);
        int e = -1;
        float w = 0.0f;
        if (lane < a.k) {
            e = a.idx[t * a.k + lane];
            w = a.w[t * a.k + lane];
            if (e >= a.E) e = -1;
        }
        const int32_t s_lane = token_slot<LL>(a, t, lane);
        int32_t s = -1;
        float W = 0.0f;
        bool mine = false;      // this lane's choice is served by the wavefront's row
        if (LL) {
            s = bcast(s_lane, i);
            W = bcastf(w, i);
            mine = lane == i;
        } else {
            uint64_t m = __ballot(s_lane >= 0);
            for (int q = 0; q < i; ++q) m &= m - 1;
            if (m) {
                const int r = __builtin_ctzll(m);
                s = bcast(s_lane, r);
                mine = e >= 0 && (unsigned)(e - r * a.epr) < (unsigned)a.epr;
                for (uint64_t c = __ballot(mine); c; c &= c - 1)   // ascending choices
                    W += bcastf(w, __builtin_ctzll(c));
            }
            // choices without a row
            if (GW && i == 0) {
                const int32_t sr = __shfl(s_lane, e < 0 ? 0 : e / a.epr);
                if (lane < a.k && (e < 0 || sr < 0)) a.grad_w[t * a.k + lane] = 0.0f;
            }
        }
        if (s < 0) {
            if (GW && LL && lane == 0) a.grad_w[t * a.k + i] = 0.0f;
            continue;
        }
        const u32x4* y = a.y + (int64_t)s * a.nv;
        const u32x4* g = a.grad_out + t * a.nv;
        u32x4* out = a.out + (int64_t)s * a.nv;
        float dot[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) dot[q] = 0.0f;
        for (int v0 = lane; v0 < a.nv; v0 += V * kWave) {
            u32x4 gv[V], yv[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = v0 + v * kWave;
                gv[v] = at < a.nv ? g[at] : u32x4{0, 0, 0, 0};
                if (GW) yv[v] = at < a.nv ? __builtin_nontemporal_load(y + at) : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = v0 + v * kWave;
                float gf[8];
                unpack8(gv[v], gf);
                if (GW) {
                    float yf[8];
                    unpack8(yv[v], yf);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dot[q] = fmaf(gf[q], yf[q], dot[q]);
                }
                if (GY && at < a.nv) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) gf[q] *= W;
                    __builtin_nontemporal_store(pack8(gf), out + at);
                }
            }
        }
        if (GW) {
            const float d = group_sum<64>(((dot[0] + dot[1]) + (dot[2] + dot[3])) +
                                          ((dot[4] + dot[5]) + (dot[6] + dot[7])));
            if (mine && lane < a.k) a.grad_w[t * a.k + lane] = d;
        }
    }
}

// Dispatch.  A wavefront has V vectors of 8 a lane of one token's gradient and
// adds the token's rows in their order, B of them under way at a time.  Bound by memory:
// the same batch with grad_other (524 MB) 84 us, 6.2 TB/s.
template <int V, int B, bool LL>
__global__ __launch_bounds__(kBlock) void dispatch_back_kernel(ExchangeBackArgs a) {
    const int lane = lane_id();
    const int64_t waves = (int64_t)a.T * a.per;
    const int64_t step = (int64_t)gridDim.x * (kBlock / kWave);
    for (int64_t gw = (int64_t)blockIdx.x * (kBlock / kWave) +
                      __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
         gw < waves; gw += step) {
        const int64_t t = gw / a.per;
        const int chunk = (int)(gw - t * a.per);
        const int32_t s_lane = token_slot<LL>(a, t, lane);
        if (a.grad_w && chunk == 0) {
            int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
            if (e >= a.E) e = -1;
            const int32_t s = LL ? s_lane : __shfl(s_lane, e < 0 ? 0 : e / a.epr);
            if (lane < a.k)
                a.grad_w[t * a.k + lane] =
                    e < 0 || s < 0 ? 0.0f : a.grad_gates[LL ? (int64_t)s : (int64_t)s * a.k + lane];
        }
        const int v0 = chunk * V * kWave + lane;
        float acc[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = v0 + v * kWave;
            unpack8(a.grad_out && at < a.nv ? a.grad_out[t * a.nv + at] : u32x4{0, 0, 0, 0}, acc[v]);
        }
        for (uint64_t m = __ballot(s_lane >= 0); m;) {
            int32_t s[B];
            int n = 0;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                s[b] = 0;
                if (m) {
                    s[b] = bcast(s_lane, __builtin_ctzll(m));
                    m &= m - 1;
                    n = b + 1;
                }
            }
            u32x4 r[B][V];
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int at = v0 + v * kWave;
                    r[b][v] = b < n && at < a.nv
                                  ? __builtin_nontemporal_load(a.y + (int64_t)s[b] * a.nv + at)
                                  : u32x4{0, 0, 0, 0};
                }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (b >= n) break;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f[8];
                    unpack8(r[b][v], f);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[v][q] += f[q];
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = v0 + v * kWave;
            if (at < a.nv) __builtin_nontemporal_store(pack8(acc[v]), a.out + t * a.nv + at);
        }
    }
}

}  // namespace ep

using namespace ep;

namespace {

#define EP_LAUNCH_EXCHANGE(...)                                                                   \
    do {                                                                                          \
        clear_hip_error();                                                                        \
        hipLaunchKernelGGL((__VA_ARGS__),                                                         \
                           dim3(loop_grid(ceil_div((int64_t)a.T * a.per, kBlock / kWave), kBlock)), \
                           dim3(kBlock), 0, stream, a);                                           \
        EP_HIP_CHECK(hipGetLastError());                                                          \
        return EP_OK;                                                                             \
    } while (0)

// What both calls of a layout check; *done: there is nothing to launch.
int exchange_args(ExchangeBackArgs& a, const ep_shape_t* shape, int64_t rows,
                  const int32_t* topk_idx, const int32_t* slot, int32_t* dev_status, bool* done) {
    const int v = validate_shape(shape);
    if (v != EP_OK) return v;
    const ep_shape_t s = *shape;
    if (!dev_status || ((uintptr_t)dev_status & 3) || rows < 0) return EP_ERR_INVALID_ARG;
    *done = s.T == 0;
    if (*done) return EP_OK;
    if (!topk_idx || !slot || (((uintptr_t)topk_idx | (uintptr_t)slot) & 3)) return EP_ERR_INVALID_ARG;
    a.idx = topk_idx;
    a.slot = slot;
    a.st = dev_status;
    a.rows = rows;
    a.T = s.T;
    a.E = s.E;
    a.R = s.R;
    a.k = s.k;
    a.epr = s.E / s.R;
    a.nv = s.H / 8;
    return EP_OK;
}

template <bool LL, bool GY, bool GW>
int launch_combine_back(ExchangeBackArgs& a, hipStream_t stream) {
    if (a.nv <= 64) EP_LAUNCH_EXCHANGE(combine_back_kernel<1, LL, GY, GW>);
    if (a.nv <= 128) EP_LAUNCH_EXCHANGE(combine_back_kernel<2, LL, GY, GW>);
    if (a.nv <= 256) EP_LAUNCH_EXCHANGE(combine_back_kernel<4, LL, GY, GW>);
    // rows of 7168: 4 vectors under way 167 us, 7 166, 8 162, 14 160 (but rows of 2048 29 : 36)
    EP_LAUNCH_EXCHANGE(combine_back_kernel<8, LL, GY, GW>);
}

template <bool LL>
int combine_back(const ep_shape_t* shape, const void* y, int64_t y_rows, const int32_t* topk_idx,
                 const float* topk_w, const int32_t* slot, const void* grad_out, void* grad_y,
                 float* grad_topk_w, int32_t* dev_status, hipStream_t stream) {
    ExchangeBackArgs a{};
    bool done = false;
    const int v = exchange_args(a, shape, y_rows, topk_idx, slot, dev_status, &done);
    if (v != EP_OK || done) return v;
    if (!topk_w || !grad_out || (!grad_y && !grad_topk_w && y_rows > 0)) return EP_ERR_INVALID_ARG;
    if (grad_topk_w && !y && y_rows > 0) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)y | (uintptr_t)grad_out | (uintptr_t)grad_y) & 15) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)topk_w | (uintptr_t)grad_topk_w) & 3) return EP_ERR_INVALID_ARG;
    if (!grad_y && !grad_topk_w) return EP_OK;
    a.w = topk_w;
    a.y = reinterpret_cast<const u32x4*>(y);
    a.grad_out = reinterpret_cast<const u32x4*>(grad_out);
    a.out = reinterpret_cast<u32x4*>(grad_y);
    a.grad_w = grad_topk_w;
    a.per = LL || a.k < a.R ? a.k : a.R;
    if (!grad_topk_w) return launch_combine_back<LL, true, false>(a, stream);
    if (!grad_y) return launch_combine_back<LL, false, true>(a, stream);
    return launch_combine_back<LL, true, true>(a, stream);
}

template <bool LL>
int dispatch_back(const ep_shape_t* shape, const int32_t* topk_idx, const int32_t* slot,
                  const void* grad_rows, int64_t rows, const float* grad_gates,
                  const void* grad_other, void* grad_x, float* grad_topk_w, int32_t* dev_status,
                  hipStream_t stream) {
    ExchangeBackArgs a{};
    bool done = false;
    const int v = exchange_args(a, shape, rows, topk_idx, slot, dev_status, &done);
    if (v != EP_OK || done) return v;
    if (!grad_x || (rows > 0 && !grad_rows)) return EP_ERR_INVALID_ARG;
    if (grad_topk_w ? rows > 0 && !grad_gates : grad_gates != nullptr) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)grad_rows | (uintptr_t)grad_other | (uintptr_t)grad_x) & 15)
        return EP_ERR_INVALID_ARG;
    if (((uintptr_t)grad_gates | (uintptr_t)grad_topk_w) & 3) return EP_ERR_INVALID_ARG;
    a.y = reinterpret_cast<const u32x4*>(grad_rows);
    a.grad_gates = grad_gates;
    a.grad_out = reinterpret_cast<const u32x4*>(grad_other);
    a.out = reinterpret_cast<u32x4*>(grad_x);
    a.grad_w = grad_topk_w;
    const int vpl = a.nv <= 64 ? 1 : a.nv <= 128 ? 2 : 4;
    a.per = (int32_t)ceil_div(a.nv, (int64_t)vpl * kWave);
    if (vpl == 1) EP_LAUNCH_EXCHANGE(dispatch_back_kernel<1, 4, LL>);
    if (vpl == 2) EP_LAUNCH_EXCHANGE(dispatch_back_kernel<2, 4, LL>);
    EP_LAUNCH_EXCHANGE(dispatch_back_kernel<4, 4, LL>);
}
}  // namespace

extern "C" int ep_combine_backward(const ep_shape_t* shape, const void* y, int64_t y_rows,
                                   const int32_t* topk_idx, const float* topk_w,
                                   const int32_t* send_slot, const void* grad_out, void* grad_y,
                                   float* grad_topk_w, int32_t* dev_status, hipStream_t stream) {
    return combine_back<false>(shape, y, y_rows, topk_idx, topk_w, send_slot, grad_out, grad_y,
                               grad_topk_w, dev_status, stream);
}

extern "C" int ep_combine_ll_backward(const ep_shape_t* shape, const void* y, int64_t y_rows,
                                      const int32_t* topk_idx, const float* topk_w,
                                      const int32_t* expert_slot, const void* grad_out,
                                      void* grad_y, float* grad_topk_w, int32_t* dev_status,
                                      hipStream_t stream) {
    return combine_back<true>(shape, y, y_rows, topk_idx, topk_w, expert_slot, grad_out, grad_y,
                              grad_topk_w, dev_status, stream);
}

extern "C" int ep_dispatch_backward(const ep_shape_t* shape, const int32_t* topk_idx,
                                    const int32_t* send_slot, const void* grad_rows, int64_t rows,
                                    const float* grad_slot_local_w, const void* grad_other,
                                    void* grad_x, float* grad_topk_w, int32_t* dev_status,
                                    hipStream_t stream) {
    return dispatch_back<false>(shape, topk_idx, send_slot, grad_rows, rows, grad_slot_local_w,
                                grad_other, grad_x, grad_topk_w, dev_status, stream);
}

extern "C" int ep_dispatch_ll_backward(const ep_shape_t* shape, const int32_t* topk_idx,
                                       const int32_t* expert_slot, const void* grad_rows,
                                       int64_t rows, const float* grad_slot_w,
                                       const void* grad_other, void* grad_x, float* grad_topk_w,
                                       int32_t* dev_status, hipStream_t stream) {
    return dispatch_back<true>(shape, topk_idx, expert_slot, grad_rows, rows, grad_slot_w,
                               grad_other, grad_x, grad_topk_w, dev_status, stream);
}
