// ep_gate.hip — the router: each token's k experts and gate weights from its
// logits, the experts' counts and the balance loss, and the gradient of the
// logits.
//
//   p[t,:]   = softmax(logits[t,:])
//   topk_idx = the k largest logits, descending, ties to the lowest expert
//   topk_w   = p of the chosen, or that divided by its sum over the chosen
//   f_e = (choices of e) / (n k),  P_e = (sum over kept t of p[t,e]) / n
//   balance_loss = E * sum_e f_e P_e       (n kept tokens)
// Backward, with d_e = grad_balance_loss * E * count_e / (n^2 k), z_j =
// grad_topk_w_j * topk_w_j and S = sum_j z_j:
//   grad_logits_e = p_e (d_e - sum_i p_i d_i) + sum_{j: e_j = e} z_j
//                   - (renormalised: sum_{j: e_j = e} topk_w_j S; else p_e S)
// (the counts are constants of the gradient, as in the loss's definition).
//
// A token is a group of L lanes (16 for E <= 256, else a wavefront), each with V
// logits in registers, four neighbours of every 4 L; one pass over the logits.
// The choices are k rounds of a maximum over the group (exact in float), then
// of the lowest expert that has it.
//
// 16384 tokens of 256 experts, k = 8, are 16.8 MB of logits, 3.4 us at a copy's
// rate; the k rounds cost about 90 instructions for four tokens each, 6 us.
// With counts and loss: 16 us and 6 of the second kernel (one logit a load: 36 and
// 22).  Backward: 33 MB, 7 us at a copy's rate, 11 us (37 with one logit a load;
// 16 while the choices' parts went over all registers in k rounds, 13 while the
// counts were awaited before the first logits were asked for).

#include "ep_rows8.h"

namespace ep {

constexpr int kGateBlocks = 256;    // workgroups, and partial sums, of a call with counts
constexpr int kGateCols = 64;       // experts that a workgroup of the second kernel sums

struct GateArgs {
    const void* logits;
    const uint8_t* mask;
    int32_t* topk_idx;
    float* topk_w;
    float* lse;
    float* part_p;        // [blocks, E]
    int32_t* part_n;      // [blocks, E]
    int32_t* part_kept;   // [blocks]
    int32_t T, E, k, renorm;
};

// Expert of register i of lane `sub` of a group of L lanes.
template <int L>
__device__ inline int expert_of(int sub, int i) {
    return i / 4 * (4 * L) + sub * 4 + i % 4;
}

template <typename F>
struct Logits;
template <>
struct Logits<float> {
    __device__ static float one(const void* p, int64_t i) {
        return reinterpret_cast<const float*>(p)[i];
    }
    __device__ static void four(const void* p, int64_t i, float* v) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = q[k];
    }
    __device__ static void put(void* p, int64_t i, float v) { reinterpret_cast<float*>(p)[i] = v; }
    __device__ static void put4(void* p, int64_t i, const float* v) {
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
    }
};
template <>
struct Logits<uint16_t> {
    __device__ static float one(const void* p, int64_t i) {
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
    }
    __device__ static void four(const void* p, int64_t i, float* v) {
        const u32x2 q = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(p) + i);
        v[0] = bf16_lo(q[0]);
        v[1] = bf16_hi(q[0]);
        v[2] = bf16_lo(q[1]);
        v[3] = bf16_hi(q[1]);
    }
    __device__ static void put(void* p, int64_t i, float v) {
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)bf16_pack(v, 0.0f);
    }
    __device__ static void put4(void* p, int64_t i, const float* v) {
        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p) + i) =
            u32x2{bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3])};
    }
};

// A lane's logits of the token whose logits start at `base`; -inf behind the
// last expert.  WIDE: four at a time (E % 4 == 0, four logits' alignment).
template <typename F, int L, int V, bool WIDE>
__device__ inline void load_logits(const void* p, int64_t base, int sub, int E, float* v) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const int e = expert_of<L>(sub, i);
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i + k] = -__builtin_inff();
            if (e < E) Logits<F>::four(p, base + e, v + i);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[i + k] = e + k < E ? Logits<F>::one(p, base + e + k) : -__builtin_inff();
        }
    }
}

// Threads of a workgroup of a call with counts, which leaves one partial sum a
// workgroup: as many wavefronts, up to 16, as have room for their sums in 32 KB
// of LDS (joining them there in turn took 14 of 23 us at 4096 tokens of 256
// experts).
constexpr int gate_threads(int E) {
    return E <= 512 ? 1024 : E <= 1024 ? 512 : E <= 2048 ? 256 : 128;
}

template <typename F, int L, int V, bool WIDE, bool STATS>
__global__ __launch_bounds__(STATS ? gate_threads(L * V) : 256) void gate_kernel(GateArgs a) {
    // STATS: [E, rounded up to 4] counts, then as many float sums a wavefront
    extern __shared__ __attribute__((aligned(16))) int32_t s_gate[];
    constexpr int kThreads = STATS ? gate_threads(L * V) : 256;
    constexpr int kGroups = kThreads / L;
    constexpr int kHold = L == 16 ? 2 : 1;     // lane j of a group holds choices j and j + L
    const int sub = (int)threadIdx.x % L;
    float sum_p[V], v[V];
    int kept = 0;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t t = (int64_t)blockIdx.x * kGroups + (int)threadIdx.x / L;
    const auto load = [&]() {
        if (t < a.T) load_logits<F, L, V, WIDE>(a.logits, t * a.E, sub, a.E, v);
    };
    load();    // under way with the mask, ahead of the barrier
    if constexpr (STATS) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum_p[i] = 0.0f;
        for (int e = (int)threadIdx.x; e < a.E; e += kThreads) s_gate[e] = 0;
        __syncthreads();
    }
    for (; t < a.T; t += step, load()) {
        if (a.mask && !a.mask[t]) {
            for (int j = sub; j < a.k; j += L) {
                a.topk_idx[t * a.k + j] = -1;
                a.topk_w[t * a.k + j] = 0.0f;
            }
            if (a.lse && sub == 0) a.lse[t] = 0.0f;
            continue;
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
        top = group_max<L>(top);
        // a row without a finite logit: every exponential is zero, not NaN
        const float shift = top == -__builtin_inff() ? 0.0f : top;
        float total = 0.0f;
        {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = expf(v[i] - shift);
                total += x[i];
            }
            total = group_sum<L>(total);
            if constexpr (STATS) {
                const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) sum_p[i] = fmaf(x[i], inv, sum_p[i]);
                kept += sub == 0;
            }
        }
        if (a.lse && sub == 0) a.lse[t] = top + logf(total);

        float my_v[kHold];
        int my_e[kHold];
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            my_v[q] = -__builtin_inff();
            my_e[q] = -1;
        }
        for (int j = 0; j < a.k; ++j) {
            float m = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < V; ++i) m = fmaxf(m, v[i]);
            const float best = group_max<L>(m);
            if (!(best > -__builtin_inff())) break;   // only -inf and NaN are left
            int at = V;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) at = v[i] == best ? i : at;
            const int mine = at < V ? expert_of<L>(sub, at) : 0x7FFFFFFF;
            const int e = group_min<L>(mine);
            at = mine == e ? at : V;
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i == at ? -__builtin_inff() : v[i];
#pragma unroll
            for (int q = 0; q < kHold; ++q)
                if (j == sub + q * L) {
                    my_v[q] = best;
                    my_e[q] = e;
                }
        }
        float my_w[kHold], chosen = 0.0f;
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            my_w[q] = expf(my_v[q] - shift);
            chosen += my_w[q];
        }
        chosen = group_sum<L>(chosen);
        float scale = 1.0f / (a.renorm ? chosen : total);
        if (total != total) scale = total;   // a NaN logit makes every weight NaN
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            const int j = sub + q * L;
            if (j < a.k) {
                a.topk_idx[t * a.k + j] = my_e[q];
                a.topk_w[t * a.k + j] = my_e[q] < 0 ? 0.0f : my_w[q] * scale;
                if constexpr (STATS)
                    if (my_e[q] >= 0) atomicAdd(&s_gate[my_e[q]], 1);
            }
        }
    }
    if constexpr (STATS) {
        // the groups of a wavefront, then the wavefronts, in a fixed order
        const int E4 = (a.E + 3) / 4 * 4;
        float* const s_sum = reinterpret_cast<float*>(s_gate + E4);
        __shared__ int s_kept[kThreads / kWave];
#pragma unroll
        for (int o = 1; o < 64; o *= 2) kept += __shfl_xor(kept, o);
        if (lane_id() == 0) s_kept[threadIdx.x / kWave] = kept;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int o = L; o < 64; o *= 2) sum_p[i] += __shfl_xor(sum_p[i], o);
        }
        if (lane_id() < L) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int e = expert_of<L>(sub, i);
                if (e < E4)
                    *reinterpret_cast<f32x4*>(&s_sum[(int)threadIdx.x / kWave * E4 + e]) =
                        f32x4{sum_p[i], sum_p[i + 1], sum_p[i + 2], sum_p[i + 3]};
            }
        }
        __syncthreads();
        for (int e = (int)threadIdx.x; e < a.E; e += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / kWave; ++w) sum += s_sum[w * E4 + e];
            a.part_p[(int64_t)blockIdx.x * a.E + e] = sum;
            a.part_n[(int64_t)blockIdx.x * a.E + e] = s_gate[e];
        }
        if (threadIdx.x == kThreads - 1) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kThreads / kWave; ++w) sum += s_kept[w];
            a.part_kept[blockIdx.x] = sum;
        }
    }
}

struct GateSumArgs {
    const float* part_p;
    const int32_t* part_n;
    const int32_t* part_kept;
    int32_t* num_tokens_per_expert;
    int32_t* num_tokens;
    float* balance_loss;
    double* part_loss;      // [workgroups]
    uint32_t* arrive;       // zero between calls
    int32_t blocks, E, k;
};

// Sums the first kernel's partials over its workgroups, kGateCols experts a
// workgroup; the last workgroup to arrive adds the experts' shares of the loss
// in their order.
__global__ __launch_bounds__(1024) void gate_sum_kernel(GateSumArgs a) {
    __shared__ double s_p[16][kGateCols];
    __shared__ int32_t s_n[16][kGateCols];
    __shared__ int s_last;
    const int c = lane_id(), g = (int)threadIdx.x / kWave;
    const int e = (int)blockIdx.x * kGateCols + c;
    double p = 0.0;
    int32_t n = 0;
    if (e < a.E)
#pragma unroll 8
        for (int b = g; b < a.blocks; b += 16) {
            p += (double)a.part_p[(int64_t)b * a.E + e];
            n += a.part_n[(int64_t)b * a.E + e];
        }
    s_p[g][c] = p;
    s_n[g][c] = n;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < 16; ++i) {
            p += s_p[i][c];
            n += s_n[i][c];
        }
        if (e < a.E) a.num_tokens_per_expert[e] = n;
        double share = e < a.E ? p * (double)n : 0.0;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) share += __shfl_xor(share, o);
        if (c == 0) {
            __hip_atomic_store(&a.part_loss[blockIdx.x], share, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            s_last = __hip_atomic_fetch_add(a.arrive, 1u, __ATOMIC_ACQ_REL,
                                            __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last || g != 0) return;
    int32_t kept = 0;
    for (int b = c; b < a.blocks; b += 64) kept += a.part_kept[b];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) kept += __shfl_xor(kept, o);
    double loss = 0.0;
    for (int b = 0; b < (int)gridDim.x; ++b)
        loss += __hip_atomic_load(&a.part_loss[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (c == 0) {
        const double m = kept > 0 ? (double)kept : 1.0;
        a.balance_loss[0] = (float)((double)a.E * loss / (m * m * (double)a.k));
        a.num_tokens[0] = kept;
        __hip_atomic_store(a.arrive, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

struct GateBackArgs {
    const void* logits;
    const uint8_t* mask;
    const int32_t* topk_idx;
    const float* topk_w;
    const float* lse;
    const int32_t* num_tokens_per_expert;
    const int32_t* num_tokens;
    const float* grad_topk_w;
    const float* grad_balance_loss;
    void* grad_logits;
    int32_t T, E, k, renorm;
};

template <typename F, int L, int V, bool WIDE>
__device__ inline void store_logits(void* p, int64_t base, int sub, int E, const float* v) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const int e = expert_of<L>(sub, i);
        if constexpr (WIDE) {
            if (e < E) Logits<F>::put4(p, base + e, v + i);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < E) Logits<F>::put(p, base + e + k, v[i + k]);
        }
    }
}

// Between LDS operations of lanes of one wavefront.
__device__ inline void lanes_meet() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename F, int L, int V, bool WIDE>
__global__ __launch_bounds__(256) void gate_back_kernel(GateBackArgs a) {
    constexpr int kGroups = 256 / L;
    constexpr int kHold = L == 16 ? 2 : 1;     // lane j of a group holds choices j and j + L
    const int sub = (int)threadIdx.x % L;
    // the parts of the group's token that belong to its chosen experts
    __shared__ __attribute__((aligned(16))) float s_parts[kGroups][L * V];
    float* const s_place = s_parts[threadIdx.x / L];
    int count[V];
#pragma unroll
    for (int i = 0; i < V; ++i) count[i] = 0;
    float n = 1.0f, grad_loss = 0.0f;
    if (a.grad_balance_loss) {
        n = fmaxf((float)a.num_tokens[0], 1.0f);
        grad_loss = a.grad_balance_loss[0];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_of<L>(sub, i);
            if (e < a.E) count[i] = a.num_tokens_per_expert[e];
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * kGroups + (int)threadIdx.x / L; t < a.T;
         t += (int64_t)gridDim.x * kGroups) {
        float p[V];
        load_logits<F, L, V, WIDE>(a.logits, t * a.E, sub, a.E, p);   // under way with the mask
        if (a.mask && !a.mask[t]) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = 0.0f;
            store_logits<F, L, V, WIDE>(a.grad_logits, t * a.E, sub, a.E, p);
            continue;
        }
        const float lse = a.lse[t];
        float z[kHold], w[kHold];   // of choices sub and sub + L
        int e[kHold];
        float S = 0.0f;
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            const int j = sub + q * L;
            z[q] = w[q] = 0.0f;
            e[q] = -1;
            if (j < a.k && a.grad_topk_w) {
                e[q] = a.topk_idx[t * a.k + j];
                w[q] = e[q] < 0 ? 0.0f : a.topk_w[t * a.k + j];
                z[q] = e[q] < 0 ? 0.0f : a.grad_topk_w[t * a.k + j] * w[q];
            }
            S += z[q];
        }
        S = group_sum<L>(S);
        const float shift = lse == -__builtin_inff() ? 0.0f : lse;
        // d_e here, not ahead of the loop: there it would wait for the counts
        // before the first logits are asked for
        float g = grad_loss;
        asm volatile("" : "+v"(g));
        const float c = g * (float)a.E / n / (n * (float)a.k);
        float pd = 0.0f, total = 0.0f, d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = c * (float)count[i];
            p[i] = expf(p[i] - shift);
            total += p[i];
            pd = fmaf(p[i], d[i], pd);
        }
        // lse is a float: far from zero it is off by more than p may be (by log E
        // where the logits are the type's lowest value), alike for all of the
        // token's p, so their sum, one but for that, takes it out
        total = group_sum<L>(total);
        const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
        pd = group_sum<L>(pd) * inv;
        if (a.renorm)
#pragma unroll
            for (int q = 0; q < kHold; ++q) z[q] = fmaf(-w[q], S, z[q]);
        else
            pd += S;
        // p (d - pd), then each choice's part at its expert
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] *= inv * (d[i] - pd);
        if (a.grad_topk_w) {
            // through the group's LDS: its lanes are of one wavefront, whose LDS
            // operations run in order, so the fences hold back the compiler only
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<f32x4*>(&s_place[expert_of<L>(sub, i)]) =
                    f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            lanes_meet();
#pragma unroll
            for (int q = 0; q < kHold; ++q)
                if ((uint32_t)e[q] < (uint32_t)a.E) atomicAdd(&s_place[e[q]], z[q]);
            lanes_meet();
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const f32x4 at = *reinterpret_cast<const f32x4*>(&s_place[expert_of<L>(sub, i)]);
#pragma unroll
                for (int c = 0; c < 4; ++c) p[i + c] += at[c];
            }
            lanes_meet();
        }
        store_logits<F, L, V, WIDE>(a.grad_logits, t * a.E, sub, a.E, p);
    }
}

int check_gate(int32_t T, int32_t E, int32_t k) {
    if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E) return EP_ERR_INVALID_ARG;
    if ((int64_t)T * k >= ((int64_t)1 << 31)) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// tokens that a workgroup of the call with counts has at once
inline int gate_groups(int E) { return gate_threads(E) / (E <= 256 ? 16 : 64); }

inline int64_t gate_blocks(int32_t T, int32_t E) {
    const int64_t b = ceil_div(T, gate_groups(E));
    return b < 1 ? 1 : b > kGateBlocks ? kGateBlocks : b;
}

inline int64_t sum_blocks(int32_t E) { return ceil_div(E, kGateCols); }

// Workspace: the arrival counter (zero between calls) in a 256-byte line, the
// experts' shares of the loss, then the first kernel's partials.
inline size_t gate_workspace(int32_t T, int32_t E) {
    const size_t b = (size_t)gate_blocks(T, E);
    return 256 + (size_t)sum_blocks(E) * 8 + b * E * 8 + b * 4;
}

}  // namespace ep

using namespace ep;

namespace {
// f(kernel of <float or bf16 bits, lanes, logits a lane>) for E experts.
#define EP_GATE_SIZES(CALL)                                      \
    if (E <= 64) return CALL(16, 4);                             \
    if (E <= 128) return CALL(16, 8);                            \
    if (E <= 256) return CALL(16, 16);                           \
    if (E <= 512) return CALL(64, 8);                            \
    if (E <= 1024) return CALL(64, 16);                          \
    if (E <= 2048) return CALL(64, 32);                          \
    return CALL(64, 64)

// Whether every token's logits can be read four at a time.
template <typename F>
bool wide_logits(const void* p, const void* q, int E) {
    return E % 4 == 0 && (((uintptr_t)p | (uintptr_t)q) & (4 * sizeof(F) - 1)) == 0;
}

template <typename F, int L, int V, bool WIDE>
int launch_gate_lv(const GateArgs& a, bool stats, hipStream_t stream) {
    clear_hip_error();
    if (stats)
        hipLaunchKernelGGL((gate_kernel<F, L, V, WIDE, true>),
                           dim3((unsigned)gate_blocks(a.T, a.E)), dim3(gate_threads(a.E)),
                           (size_t)(a.E + 3) / 4 * 16 * (1 + gate_threads(a.E) / kWave), stream, a);
    else
        hipLaunchKernelGGL((gate_kernel<F, L, V, WIDE, false>),
                           dim3(loop_grid(ceil_div(a.T, 256 / L), 256)), dim3(256), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

template <typename F>
int launch_gate(const GateArgs& a, bool stats, hipStream_t stream) {
    const int E = a.E;
    const bool wide = wide_logits<F>(a.logits, nullptr, E);
#define EP_CALL(L, V)                                                  \
    (wide ? launch_gate_lv<F, L, V, true>(a, stats, stream)            \
          : launch_gate_lv<F, L, V, false>(a, stats, stream))
    EP_GATE_SIZES(EP_CALL);
#undef EP_CALL
}

template <typename F, int L, int V, bool WIDE>
int launch_gate_back_lv(const GateBackArgs& a, hipStream_t stream) {
    clear_hip_error();
    hipLaunchKernelGGL((gate_back_kernel<F, L, V, WIDE>),
                       dim3(loop_grid(ceil_div(a.T, 256 / L), 256)), dim3(256), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

template <typename F>
int launch_gate_back(const GateBackArgs& a, hipStream_t stream) {
    const int E = a.E;
    const bool wide = wide_logits<F>(a.logits, a.grad_logits, E);
#define EP_CALL(L, V)                                                  \
    (wide ? launch_gate_back_lv<F, L, V, true>(a, stream)              \
          : launch_gate_back_lv<F, L, V, false>(a, stream))
    EP_GATE_SIZES(EP_CALL);
#undef EP_CALL
}
}  // namespace

extern "C" size_t ep_route_workspace_bytes(int32_t T, int32_t E) {
    if (check_gate(T, E, 1) != EP_OK) return 0;
    return gate_workspace(T, E);
}

extern "C" int ep_route(int32_t T, int32_t E, int32_t k, int32_t dtype, int32_t mode,
                        const void* logits, const uint8_t* token_mask, int32_t* topk_idx,
                        float* topk_w, int32_t* num_tokens_per_expert, int32_t* num_tokens,
                        float* lse, float* balance_loss, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    int v = check_gate(T, E, k);
    if (v != EP_OK) return v;
    if (dtype != EP_BF16 && dtype != EP_F32) return EP_ERR_INVALID_ARG;
    if (mode != EP_GATE_SOFTMAX && mode != EP_GATE_SOFTMAX_RENORM) return EP_ERR_INVALID_ARG;
    const bool stats = num_tokens_per_expert || num_tokens || balance_loss;
    if (stats && (!num_tokens_per_expert || !num_tokens || !balance_loss || !workspace))
        return EP_ERR_INVALID_ARG;
    if (stats && (workspace_bytes < gate_workspace(T, E) || ((uintptr_t)workspace & 15)))
        return EP_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !topk_idx || !topk_w)) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)topk_idx | (uintptr_t)topk_w | (uintptr_t)lse |
         (uintptr_t)num_tokens_per_expert | (uintptr_t)num_tokens | (uintptr_t)balance_loss) & 3)
        return EP_ERR_INVALID_ARG;
    if ((uintptr_t)logits & (dtype == EP_F32 ? 3 : 1)) return EP_ERR_INVALID_ARG;
    if (T == 0 && !stats) return EP_OK;
    const int64_t blocks = gate_blocks(T, E);
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    GateArgs a{};
    a.logits = logits;
    a.mask = token_mask;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.lse = lse;
    a.T = T;
    a.E = E;
    a.k = k;
    a.renorm = mode == EP_GATE_SOFTMAX_RENORM;
    if (stats) {
        a.part_p = reinterpret_cast<float*>(ws + 256 + sum_blocks(E) * 8);
        a.part_n = reinterpret_cast<int32_t*>(a.part_p + blocks * E);
        a.part_kept = a.part_n + blocks * E;
    }
    v = dtype == EP_F32 ? launch_gate<float>(a, stats, stream)
                        : launch_gate<uint16_t>(a, stats, stream);
    if (v != EP_OK || !stats) return v;
    GateSumArgs b{};
    b.part_p = a.part_p;
    b.part_n = a.part_n;
    b.part_kept = a.part_kept;
    b.num_tokens_per_expert = num_tokens_per_expert;
    b.num_tokens = num_tokens;
    b.balance_loss = balance_loss;
    b.part_loss = reinterpret_cast<double*>(ws + 256);
    b.arrive = reinterpret_cast<uint32_t*>(ws);
    b.blocks = (int32_t)blocks;
    b.E = E;
    b.k = k;
    hipLaunchKernelGGL(gate_sum_kernel, dim3((unsigned)sum_blocks(E)), dim3(1024), 0, stream, b);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

extern "C" int ep_route_backward(int32_t T, int32_t E, int32_t k, int32_t dtype, int32_t mode,
                                 const void* logits, const uint8_t* token_mask,
                                 const int32_t* topk_idx, const float* topk_w,
                                 const int32_t* num_tokens_per_expert, const int32_t* num_tokens,
                                 const float* lse, const float* grad_topk_w,
                                 const float* grad_balance_loss, void* grad_logits,
                                 hipStream_t stream) {
    int v = check_gate(T, E, k);
    if (v != EP_OK) return v;
    if (dtype != EP_BF16 && dtype != EP_F32) return EP_ERR_INVALID_ARG;
    if (mode != EP_GATE_SOFTMAX && mode != EP_GATE_SOFTMAX_RENORM) return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (!logits || !lse || !grad_logits) return EP_ERR_INVALID_ARG;
    if (grad_topk_w && (!topk_idx || !topk_w)) return EP_ERR_INVALID_ARG;
    if (grad_balance_loss && (!num_tokens_per_expert || !num_tokens)) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)topk_idx | (uintptr_t)topk_w | (uintptr_t)lse | (uintptr_t)grad_topk_w |
         (uintptr_t)num_tokens_per_expert | (uintptr_t)num_tokens |
         (uintptr_t)grad_balance_loss) & 3)
        return EP_ERR_INVALID_ARG;
    if (((uintptr_t)logits | (uintptr_t)grad_logits) & (dtype == EP_F32 ? 3 : 1))
        return EP_ERR_INVALID_ARG;
    GateBackArgs a{};
    a.logits = logits;
    a.mask = token_mask;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.lse = lse;
    a.num_tokens_per_expert = num_tokens_per_expert;
    a.num_tokens = num_tokens;
    a.grad_topk_w = grad_topk_w;
    a.grad_balance_loss = grad_balance_loss;
    a.grad_logits = grad_logits;
    a.T = T;
    a.E = E;
    a.k = k;
    a.renorm = mode == EP_GATE_SOFTMAX_RENORM;
    return dtype == EP_F32 ? launch_gate_back<float>(a, stream)
                           : launch_gate_back<uint16_t>(a, stream);
}
