// ep_grad_norm.hip — the norm of all gradients together, and their clipping.
//
// The tensors of a call come as a host table, which goes to the kernels by value
// (kTable tensors a launch).  A tensor is cut into units of kUnit threads' loads;
// a workgroup takes one run of the launch's units and looks its first tensor up
// once.  Loads are 16 bytes from the first aligned element on; the elements
// before it belong to the first unit.
//
// The norm: squares and their sums in double (a float's square leaves float's
// range from 1.8e19 up and, towards zero, 1e-19 down); a partial sum a workgroup;
// the last workgroup of the last launch adds them in their order.
//
// The clip: v * m * 2^e with max_norm / norm = m * 2^e, so a ratio below float's
// range still scales what float holds.

#include "ep_rows8.h"

namespace ep {

constexpr int kGradThreads = 1024;
constexpr int kGradGrid = 512;            // two workgroups a CU
constexpr int kTable = 128;               // tensors of a launch: its table is 3.6 KB of arguments
constexpr int kUnitVecs = 2;              // groups of 8 elements a thread
constexpr int kUnit = kGradThreads * 8 * kUnitVecs;
constexpr int64_t kMaxTensor = (int64_t)1 << 38;   // elements: a launch's units fit 32 bits
static_assert((kMaxTensor / kUnit + 1) * kTable < ((int64_t)1 << 32), "units fit 32 bits");

struct GradTable {
    const void* src[kTable];    // bit 0: float (an address of either type has it clear)
    void* dst[kTable];          // clip only; bit 0 as src's
    int64_t n[kTable];
    uint32_t first[kTable + 1]; // first unit of each tensor
    int32_t count;
};

struct GradArgs {
    GradTable t;
    double* partial;            // norm: this launch's partial sums
    const double* partials;     // norm, last launch: all of them
    double* sum_squares;
    float* norm;
    uint32_t* ticket;           // norm, last launch: workgroups that are done
    double max_norm;            // clip
    uint32_t units;
    int32_t n_partials;         // norm: 0 in all launches but the last
    bool in_place;              // clip
};

// Elements before the first 16-byte boundary.
__host__ __device__ inline int64_t head_of(uintptr_t p, int64_t n, bool wide) {
    const int64_t h = (int64_t)((16 - (p & 15)) & 15) / (wide ? 4 : 2);
    return h < n ? h : n;
}

__device__ inline float load1(const void* p, int64_t i, bool wide) {
    return wide ? reinterpret_cast<const float*>(p)[i]
                : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// Eight elements from an aligned address.
__device__ inline void load8(const void* p, int64_t i, bool wide, float* f) {
    if (wide) {
        const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
        const f32x4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = a[j];
            f[4 + j] = b[j];
        }
    } else {
        unpack8(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
                    reinterpret_cast<const uint16_t*>(p) + i)),
                f);
    }
}

// Walks a workgroup's run of units.  `eight(tensor, i)` gets the first of eight
// aligned elements, `one(tensor, i)` a single one.
template <typename EIGHT, typename ONE>
__device__ inline void walk(const GradArgs& a, EIGHT eight, ONE one) {
    const uint32_t per = a.units / gridDim.x, extra = a.units % gridDim.x, b = blockIdx.x;
    uint32_t u = b * per + (b < extra ? b : extra);
    const uint32_t end = u + per + (b < extra);
    if (u == end) return;
    int lo = 0, hi = a.t.count - 1;     // the last tensor whose first unit is not behind u
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.t.first[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int tid = (int)threadIdx.x;
    for (int t = lo; u < end; ++u) {
        if (u >= a.t.first[t + 1]) ++t;     // every tensor of the table has a unit
        const uintptr_t p = (uintptr_t)a.t.src[t];
        const bool wide = p & 1;
        const int64_t n = a.t.n[t], head = head_of(p & ~(uintptr_t)1, n, wide);
        const uint32_t in = u - a.t.first[t];
        if (in == 0 && tid < head) one(t, (int64_t)tid);
        const int64_t at = head + (int64_t)in * kUnit;
#pragma unroll
        for (int v = 0; v < kUnitVecs; ++v) {
            const int64_t i = at + (int64_t)(v * kGradThreads + tid) * 8;
            if (i + 8 <= n)
                eight(t, i);
            else
                for (int64_t j = i; j < n; ++j) one(t, j);
        }
    }
}

__device__ inline double block_sum(double v) {
    __shared__ double s_part[kGradThreads / kWave];
#pragma unroll
    for (int o = kWave / 2; o; o /= 2) v += __shfl_xor(v, o);
    if (lane_id() == 0) s_part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = threadIdx.x < kGradThreads / kWave ? s_part[threadIdx.x] : 0.0;
    if (threadIdx.x < kWave) {
#pragma unroll
        for (int o = kWave / 2; o; o /= 2) v += __shfl_xor(v, o);
    }
    __syncthreads();
    return v;    // of the first wavefront
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(GradArgs a) {
    double sum = 0.0;
    const auto add = [&](float f) { sum = fma((double)f, (double)f, sum); };
    walk(
        a,
        [&](int t, int64_t i) {
            const uintptr_t p = (uintptr_t)a.t.src[t];
            float f[8];
            load8((const void*)(p & ~(uintptr_t)1), i, p & 1, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) add(f[q]);
        },
        [&](int t, int64_t i) {
            const uintptr_t p = (uintptr_t)a.t.src[t];
            add(load1((const void*)(p & ~(uintptr_t)1), i, p & 1));
        });
    sum = block_sum(sum);
    __shared__ bool s_last;
    if (threadIdx.x == 0) {
        __hip_atomic_store(a.partial + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = false;
        if (a.n_partials) {
            s_last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL,
                                            __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    sum = 0.0;
    for (int i = (int)threadIdx.x; i < a.n_partials; i += kGradThreads)
        sum += __hip_atomic_load(a.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        *a.sum_squares = sum;
        if (a.norm) *a.norm = (float)sqrt(sum);
        __hip_atomic_store(a.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(GradArgs a) {
    const double norm = sqrt(*a.sum_squares);
    const bool clip = norm > a.max_norm && norm < __builtin_huge_val();   // false for a NaN
    if (!clip && a.in_place) return;
    int e = 0;
    const float m = clip ? (float)frexp(a.max_norm / norm, &e) : 1.0f;
    walk(
        a,
        [&](int t, int64_t i) {
            const uintptr_t p = (uintptr_t)a.t.src[t], d = (uintptr_t)a.t.dst[t];
            float f[8];
            load8((const void*)(p & ~(uintptr_t)1), i, p & 1, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = ldexpf(f[q] * m, e);
            if (d & 1) {
                float* o = reinterpret_cast<float*>(d & ~(uintptr_t)1) + i;
                if (((uintptr_t)o & 15) == 0) {
                    __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]},
                                                reinterpret_cast<f32x4*>(o));
                    __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]},
                                                reinterpret_cast<f32x4*>(o) + 1);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = f[q];
                }
            } else {
                uint16_t* o = reinterpret_cast<uint16_t*>(d) + i;
                const u32x4 v = pack8(f);
                if (((uintptr_t)o & 15) == 0) {
                    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o));
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = (uint16_t)(v[q / 2] >> (q % 2 * 16));
                }
            }
        },
        [&](int t, int64_t i) {
            const uintptr_t p = (uintptr_t)a.t.src[t], d = (uintptr_t)a.t.dst[t];
            const float f = ldexpf(load1((const void*)(p & ~(uintptr_t)1), i, p & 1) * m, e);
            if (d & 1)
                reinterpret_cast<float*>(d & ~(uintptr_t)1)[i] = f;
            else
                reinterpret_cast<uint16_t*>(d)[i] = (uint16_t)bf16_pack(f, 0.0f);
        });
}

// A tensor of the table: its data may be NULL only where it has no elements.
int check_tensor(const ep_tensor_t& t) {
    if (t.n < 0 || t.n >= kMaxTensor) return EP_ERR_INVALID_ARG;
    if (t.dtype != EP_BF16 && t.dtype != EP_F32) return EP_ERR_INVALID_ARG;
    if (t.n > 0 && !t.data) return EP_ERR_INVALID_ARG;
    if ((uintptr_t)t.data & (t.dtype == EP_F32 ? 3 : 1)) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

int check_tensors(int32_t count, const ep_tensor_t* t) {
    if (count < 0 || (count > 0 && !t)) return EP_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i)
        if (check_tensor(t[i]) != EP_OK) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Fills a launch's table from tensor *at on, and moves *at behind its last.
void fill_table(GradArgs& a, int32_t count, const ep_tensor_t* src, const ep_tensor_t* dst,
                int32_t* at) {
    GradTable& t = a.t;
    t.count = 0;
    int64_t units = 0;
    for (; *at < count && t.count < kTable; ++*at) {
        const ep_tensor_t& s = src[*at];
        if (s.n == 0) continue;
        const bool wide = s.dtype == EP_F32;
        const int64_t rest = s.n - head_of((uintptr_t)s.data, s.n, wide);
        const int64_t mine = rest ? ceil_div(rest, kUnit) : 1;
        t.src[t.count] = (const void*)((uintptr_t)s.data | (wide ? 1 : 0));
        if (dst)
            t.dst[t.count] =
                (void*)((uintptr_t)dst[*at].data | (dst[*at].dtype == EP_F32 ? 1 : 0));
        t.n[t.count] = s.n;
        t.first[t.count++] = (uint32_t)units;
        units += mine;
    }
    t.first[t.count] = (uint32_t)units;
    a.units = (uint32_t)units;
}

}  // namespace ep

using namespace ep;

namespace {
constexpr size_t kTicketBytes = 256;     // of the workspace, ahead of the partial sums
}

extern "C" size_t ep_grad_norm_workspace_bytes(int32_t count) {
    if (count < 0) return 0;
    return kTicketBytes + (size_t)kGradGrid * 8 * (1 + (size_t)count / kTable);
}

extern "C" int ep_grad_norm(int32_t count, const ep_tensor_t* tensors, double* sum_squares,
                            float* norm, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    const int v = check_tensors(count, tensors);
    if (v != EP_OK) return v;
    if (!sum_squares || ((uintptr_t)sum_squares & 7) || ((uintptr_t)norm & 3) || !workspace ||
        ((uintptr_t)workspace & 15) || workspace_bytes < ep_grad_norm_workspace_bytes(count))
        return EP_ERR_INVALID_ARG;
    GradArgs a{};
    a.ticket = reinterpret_cast<uint32_t*>(workspace);
    double* const partials =
        reinterpret_cast<double*>(reinterpret_cast<uint8_t*>(workspace) + kTicketBytes);
    a.partials = partials;
    a.sum_squares = sum_squares;
    a.norm = norm;
    int32_t left = 0;        // tensors with elements
    for (int32_t i = 0; i < count; ++i) left += tensors[i].n > 0;
    int32_t at = 0;
    int64_t done = 0;
    do {
        fill_table(a, count, tensors, nullptr, &at);
        left -= a.t.count;
        // without a unit one workgroup still writes the sum, zero
        const uint32_t grid =
            a.units < (uint32_t)kGradGrid ? (a.units ? a.units : 1u) : (uint32_t)kGradGrid;
        a.partial = partials + done;
        done += grid;
        a.n_partials = left == 0 ? (int32_t)done : 0;
        clear_hip_error();
        hipLaunchKernelGGL(grad_norm_kernel, dim3(grid), dim3(kGradThreads), 0, stream, a);
        EP_HIP_CHECK(hipGetLastError());
    } while (left > 0);
    return EP_OK;
}

extern "C" int ep_grad_clip(int32_t count, const ep_tensor_t* tensors, const ep_tensor_t* into,
                            const double* sum_squares, double max_norm, hipStream_t stream) {
    int v = check_tensors(count, tensors);
    if (v != EP_OK) return v;
    if (into && (v = check_tensors(count, into)) != EP_OK) return v;
    if (!sum_squares || ((uintptr_t)sum_squares & 7) || !(max_norm >= 0.0)) return EP_ERR_INVALID_ARG;
    for (int32_t i = 0; into && i < count; ++i)
        if (into[i].n != tensors[i].n) return EP_ERR_INVALID_ARG;
    GradArgs a{};
    a.sum_squares = const_cast<double*>(sum_squares);
    a.max_norm = max_norm;
    a.in_place = !into;
    for (int32_t at = 0;;) {
        fill_table(a, count, tensors, into ? into : tensors, &at);
        if (a.units == 0) return EP_OK;
        clear_hip_error();
        hipLaunchKernelGGL(grad_clip_kernel,
                           dim3(a.units < (uint32_t)kGradGrid ? a.units : (uint32_t)kGradGrid),
                           dim3(kGradThreads), 0, stream, a);
        EP_HIP_CHECK(hipGetLastError());
    }
}
