// ep_grad_norm.hip — the norm of all gradients together, and their clipping.
//
// The tensors come as a table in device memory, made once on the host.  A tensor
// is cut into units of kUnit elements (one pass of a workgroup's loads), which the
// workgroups take in turn, a few at a time.  Units begin on a 128-byte line (a line
// written in two parts costs as two); the elements before a tensor's first line
// belong to its first unit.
//
// The norm: squares and their sums in double (a float's square leaves float's
// range from 1.8e19 up and, towards zero, 1e-19 down); a partial sum a workgroup;
// the last workgroup that ends adds them in their order.
//
// The clip: v * m * 2^e with max_norm / norm = m * 2^e, so a ratio below float's
// range still scales what float holds.
//
// Bound by memory.  40 tensors of 622 MB, nearly all bf16: norm 111 us (5.6 TB/s), clip
// into other buffers 241 us (5.2), both in a row 337: the clip finds the last 200 MB in the
// last-level cache.  1000 tensors of 156 MB: norm 37 us.  The same bytes all in float: norm
// 113 and 40 us, clip of the 622 MB 260 us; all in bf16 126, 42 and 233.

#include <string.h>

#include "ep_rows8.h"

namespace ep {

constexpr int kGradThreads = 1024;
constexpr int kGradGrid = 512;            // two workgroups a CU
constexpr int kUnitVecs = 2;              // groups of 8 elements a thread
constexpr int kUnit = kGradThreads * 8 * kUnitVecs;
constexpr int kHeld = 1024;               // tensors whose entries a workgroup holds in LDS
constexpr int kMostChunk = 2;             // units that a workgroup takes at a time: with 1 the
                                          // 622 MB's norm and clip take 377 us, 2 340, 4 352, 8 369
constexpr int64_t kMaxTensor = (int64_t)1 << 38;   // elements
constexpr int64_t kMaxUnits = (int64_t)1 << 31;

// One tensor of the table; the entry behind the last one has `first` alone.
struct GradEntry {
    uint64_t data;      // bit 0: float (an address of either type has it clear)
    int64_t n;
    uint32_t first;     // its first unit; without elements it has none
    uint32_t pad;
    uint64_t pad2;
};
static_assert(sizeof(GradEntry) == 32, "entries stay 16-byte aligned");

struct GradArgs {
    const GradEntry* src;
    const GradEntry* dst;       // clip
    double* partial;            // norm: a partial sum a workgroup
    double* sum_squares;
    float* norm;
    uint32_t* ticket;           // norm: workgroups that are done
    double max_norm;            // clip
    uint32_t units;
    int32_t count, chunk;
    bool in_place;              // clip
};

// Elements before the first line.
__host__ __device__ inline int64_t head_of(uint64_t p, int64_t n, bool wide) {
    const int64_t h = (int64_t)((128 - (p & 127)) & 127) / (wide ? 4 : 2);
    return h < n ? h : n;
}

__device__ inline float load1(uint64_t p, int64_t i) {
    return p & 1 ? reinterpret_cast<const float*>(p & ~1ull)[i]
                 : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// Eight elements from an aligned address.
__device__ inline void load8(uint64_t p, int64_t i, float* f) {
    if (p & 1) {
        const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p & ~1ull) + i);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = a[j];
            f[4 + j] = b[j];
        }
    } else {
        unpack8(*reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i), f);
    }
}

// Walks a workgroup's units.  `eight(from, to, i)` gets a tensor's addresses and the
// first of eight aligned elements, `one(from, to, i)` a single one.  The clip goes
// through them from the end: what the norm read last is in cache first.
template <bool CLIP, typename EIGHT, typename ONE>
__device__ inline void walk(const GradArgs& a, EIGHT eight, ONE one) {
    __shared__ uint32_t s_first[kHeld + 1];
    __shared__ uint64_t s_from[kHeld], s_to[CLIP ? kHeld : 1];
    __shared__ int64_t s_n[kHeld];
    if (a.units == 0) return;      // there may be no table
    const bool held = a.count <= kHeld;
    const int tid = (int)threadIdx.x;
    for (int i = tid; held && i <= a.count; i += kGradThreads) {
        const GradEntry e = a.src[i];
        s_first[i] = e.first;
        if (i < a.count) {
            s_from[i] = e.data;
            s_n[i] = e.n;
            if (CLIP) s_to[i] = a.dst[i].data;
        }
    }
    __syncthreads();
    const auto first = [&](int i) { return held ? s_first[i] : a.src[i].first; };
    const uint32_t chunks = (a.units + a.chunk - 1) / a.chunk;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        uint32_t u = (CLIP ? chunks - 1 - c : c) * a.chunk;
        const uint32_t end = u + a.chunk < a.units ? u + a.chunk : a.units;
        int t = 0;      // the last tensor whose first unit is not behind u
        for (int hi = a.count - 1; t < hi;) {
            const int mid = (t + hi + 1) / 2;
            if (first(mid) <= u)
                t = mid;
            else
                hi = mid - 1;
        }
        while (u < end) {
            while (u >= first(t + 1)) ++t;
            const uint64_t p = held ? s_from[t] : a.src[t].data;
            const uint64_t d = !CLIP ? 0 : held ? s_to[t] : a.dst[t].data;
            const int64_t n = held ? s_n[t] : a.src[t].n, head = head_of(p & ~1ull, n, p & 1);
            const uint32_t at = first(t), stop = first(t + 1) < end ? first(t + 1) : end;
            if (u == at && tid < head) one(p, d, (int64_t)tid);
            for (; u < stop; ++u) {
                const int64_t from = head + (int64_t)(u - at) * kUnit;
                if (from + kUnit <= n) {
#pragma unroll
                    for (int v = 0; v < kUnitVecs; ++v)
                        eight(p, d, from + (int64_t)(v * kGradThreads + tid) * 8);
                } else {
#pragma unroll
                    for (int v = 0; v < kUnitVecs; ++v) {
                        const int64_t i = from + (int64_t)(v * kGradThreads + tid) * 8;
                        if (i + 8 <= n)
                            eight(p, d, i);
                        else
                            for (int64_t j = i; j < n; ++j) one(p, d, j);
                    }
                }
            }
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
    walk<false>(
        a,
        [&](uint64_t p, uint64_t, int64_t i) {
            float f[8];
            load8(p, i, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) add(f[q]);
        },
        [&](uint64_t p, uint64_t, int64_t i) { add(load1(p, i)); });
    sum = block_sum(sum);
    __shared__ bool s_last;
    if (threadIdx.x == 0) {
        // The partial sum goes past the XCD's L2 and is waited for before the ticket; the
        // last one's loads go past it too.  (Fences would have every workgroup write its
        // L2 back and clear it: 22 us in place of 16 for 40 MB in 100 tensors.)
        __hip_atomic_store(a.partial + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::: "memory");
        wait_vm();
        asm volatile("" ::: "memory");
        s_last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    sum = 0.0;
    for (int i = (int)threadIdx.x; i < (int)gridDim.x; i += kGradThreads)
        sum += __hip_atomic_load(a.partial + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
    walk<true>(
        a,
        [&](uint64_t p, uint64_t d, int64_t i) {
            float f[8];
            load8(p, i, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = ldexpf(f[q] * m, e);
            if (d & 1) {
                float* o = reinterpret_cast<float*>(d & ~1ull) + i;
                if (((uintptr_t)o & 15) == 0) {
                    // (not streaming: the two halves of 32 bytes meet in cache)
                    reinterpret_cast<f32x4*>(o)[0] = f32x4{f[0], f[1], f[2], f[3]};
                    reinterpret_cast<f32x4*>(o)[1] = f32x4{f[4], f[5], f[6], f[7]};
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
        [&](uint64_t p, uint64_t d, int64_t i) {
            const float f = ldexpf(load1(p, i) * m, e);
            if (d & 1)
                reinterpret_cast<float*>(d & ~1ull)[i] = f;
            else
                reinterpret_cast<uint16_t*>(d)[i] = (uint16_t)bf16_pack(f, 0.0f);
        });
}

// Its data may be NULL only where a tensor has no elements.
bool tensor_fits(const ep_tensor_t& t) {
    return t.n >= 0 && t.n < kMaxTensor && (t.dtype == EP_BF16 || t.dtype == EP_F32) &&
           (t.n == 0 || t.data) && ((uintptr_t)t.data & (t.dtype == EP_F32 ? 3 : 1)) == 0;
}

}  // namespace ep

using namespace ep;

namespace {
constexpr size_t kTicketBytes = 256;     // of the workspace, ahead of the partial sums

int list_fits(const ep_tensor_list_t* l) {
    return l && l->count >= 0 && l->units >= 0 && l->units < kMaxUnits &&
           (l->units == 0 || (l->table && ((uintptr_t)l->table & 15) == 0));
}

// Launch shape: a few turns of the workgroups where there is enough, so that none
// has much more than the others.
unsigned grad_grid(GradArgs& a) {
    const int64_t chunk = a.units / (4 * kGradGrid);
    a.chunk = (int32_t)(chunk < 1 ? 1 : chunk < kMostChunk ? chunk : kMostChunk);
    return a.units < 1 ? 1u : a.units < (uint32_t)kGradGrid ? a.units : (uint32_t)kGradGrid;
}
}  // namespace

extern "C" size_t ep_tensor_table_bytes(int32_t count) {
    return count < 0 ? 0 : ((size_t)count + 1) * sizeof(GradEntry);
}

extern "C" int ep_tensor_table(int32_t count, const ep_tensor_t* tensors, void* table,
                               ep_tensor_list_t* list) {
    if (count < 0 || (count > 0 && !tensors) || !table || ((uintptr_t)table & 7) || !list)
        return EP_ERR_INVALID_ARG;
    GradEntry* e = reinterpret_cast<GradEntry*>(table);
    memset(e, 0, ep_tensor_table_bytes(count));
    int64_t units = 0;
    uint64_t sizes = 1469598103934665603ull;
    for (int32_t i = 0; i < count; ++i) {
        const ep_tensor_t& t = tensors[i];
        if (!tensor_fits(t)) return EP_ERR_INVALID_ARG;
        const bool wide = t.dtype == EP_F32;
        e[i].data = (uint64_t)(uintptr_t)t.data | (wide ? 1 : 0);
        e[i].n = t.n;
        e[i].first = (uint32_t)units;
        const int64_t rest = t.n - head_of((uint64_t)(uintptr_t)t.data, t.n, wide);
        units += t.n == 0 ? 0 : rest ? ceil_div(rest, kUnit) : 1;
        if (units >= kMaxUnits) {
            record_error("tensor table: more than 2^31 units of elements");
            return EP_ERR_INVALID_ARG;
        }
        sizes = (sizes ^ (uint64_t)t.n) * 1099511628211ull;
        sizes ^= sizes >> 29;
    }
    e[count].first = (uint32_t)units;
    list->table = nullptr;
    list->units = units;
    list->sizes = sizes;
    list->count = count;
    list->pad_ = 0;
    return EP_OK;
}

extern "C" size_t ep_grad_norm_workspace_bytes(void) {
    return kTicketBytes + (size_t)kGradGrid * sizeof(double);
}

extern "C" int ep_grad_norm(const ep_tensor_list_t* tensors, double* sum_squares, float* norm,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!list_fits(tensors)) return EP_ERR_INVALID_ARG;
    if (!sum_squares || ((uintptr_t)sum_squares & 7) || ((uintptr_t)norm & 3) || !workspace ||
        ((uintptr_t)workspace & 15) || workspace_bytes < ep_grad_norm_workspace_bytes())
        return EP_ERR_INVALID_ARG;
    GradArgs a{};
    a.src = reinterpret_cast<const GradEntry*>(tensors->table);
    a.ticket = reinterpret_cast<uint32_t*>(workspace);
    a.partial = reinterpret_cast<double*>(reinterpret_cast<uint8_t*>(workspace) + kTicketBytes);
    a.sum_squares = sum_squares;
    a.norm = norm;
    a.units = (uint32_t)tensors->units;
    a.count = tensors->count;
    clear_hip_error();
    // without a unit one workgroup still writes the sum, zero
    hipLaunchKernelGGL(grad_norm_kernel, dim3(grad_grid(a)), dim3(kGradThreads), 0,
                       stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

extern "C" int ep_grad_clip(const ep_tensor_list_t* tensors, const ep_tensor_list_t* into,
                            const double* sum_squares, double max_norm, hipStream_t stream) {
    if (!list_fits(tensors)) return EP_ERR_INVALID_ARG;
    if (into && (!list_fits(into) || into->count != tensors->count || into->sizes != tensors->sizes))
        return EP_ERR_INVALID_ARG;
    if (!sum_squares || ((uintptr_t)sum_squares & 7) || !(max_norm >= 0.0)) return EP_ERR_INVALID_ARG;
    if (tensors->units == 0) return EP_OK;
    GradArgs a{};
    a.src = reinterpret_cast<const GradEntry*>(tensors->table);
    a.dst = into ? reinterpret_cast<const GradEntry*>(into->table) : a.src;
    a.sum_squares = const_cast<double*>(sum_squares);
    a.max_norm = max_norm;
    a.in_place = !into;
    a.units = (uint32_t)tensors->units;
    a.count = tensors->count;
    clear_hip_error();
    hipLaunchKernelGGL(grad_clip_kernel, dim3(grad_grid(a)), dim3(kGradThreads), 0,
                       stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}
