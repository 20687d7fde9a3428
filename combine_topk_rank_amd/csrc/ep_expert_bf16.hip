// ep_expert_bf16.hip — the experts' products in bf16, and their gradients: the
// training form of ep_expert.hip's.
//
// Three products over rows grouped by expert, of the same shape: out[q, p] is the
// sum over c of P and Q.
//   forward          out[m,n]  = sum_k w[n,k] * rows[m,k]        P = w,    Q = rows
//   rows' gradient   out[m,k]  = sum_n w[n,k] * grad_out[m,n]    P = w,    Q = grad_out
//   weights'         out[n,k]  = sum_m rows[m,k] * grad_out[m,n] P = rows, Q = grad_out
// P is the matrix instruction's first operand and Q its second, so a lane's four
// results are four neighbouring columns of one row of the output.
//
// An operand lies in memory along c (P and Q of the forward, Q of the rows'
// gradient) or across it (the others).  Either way it is copied as it lies, 16
// bytes a lane, straight to LDS.  What lies along c is read from LDS 16 bytes a
// lane; what lies across it is read by the transposing LDS read, which hands each
// lane four consecutive c of one column.
//
// The gate's forward has an output's gate and up in one wavefront and stores
// silu(gate) * up; its backward makes the gradient of both first, in bf16, and
// goes on as the plain one.

#include <type_traits>

#include "ep_tiles.h"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* LdsS16x4;

enum Product { kForward, kGate, kRowsBack, kWeightBack };

struct Bf16Args {
    const uint16_t* p;
    const uint16_t* q;
    const int32_t* group_offset;   // [G+1]
    void* out;
    uint16_t* pre;                 // gate
    int32_t* st;
    int64_t M;
    int64_t tiles;                 // of the launch
    int64_t places;                // small tiles: with what fills the runs up
    int32_t G;
    int32_t W;                     // P's extent outside c (gate: 2F)
    int32_t V;                     // weights' gradient: Q's extent outside c
    int32_t C;                     // extent of c (weights' gradient: the group's rows)
    int32_t pitch_p, pitch_q;      // elements
    int32_t tiles_w, tiles_v;      // tiles along W, along V
    int32_t splits;                // weights' gradient: parts of c, each a float output
    bool wide;                     // weights' gradient: float output
};

constexpr int kDepth = 64;         // c of a block: 128 bytes of an operand along c

// 1 / (1 + exp(-g)); far below zero exp(g), which is the same there: exp(-g) leaves
// float's range at -88.7, where times a large up the product is still a number.
__device__ inline float sigmoid(float g) {
    const bool far = g < -80.0f;
    const float e = expf(far ? g : -g);
    return far ? e : 1.0f / (1.0f + e);
}

// g * sigmoid(g), for the forward: through exp(-|g|), which never leaves float's range
// upwards (nor, below -200, zero), by the hardware's exp2 and reciprocal (off by a unit in the last place each;
// log2(e) in two parts, and scaled where the result is below float's normal range, which
// that exp2 makes zero).  Half of sigmoid()'s instructions: a big tile's 128 results a lane,
// with one wavefront on a SIMD, took 6 us with it.
__device__ inline float silu(float g) {
    const float x = fmaxf(-fabsf(g), -200.0f), t = x * 1.44269504f;
    const float rest = fmaf(x, 1.44269504f, -t) + x * 1.92596300e-8f;
    const bool low = t < -126.0f;
    const float e = __builtin_amdgcn_exp2f(low ? t + 64.0f : t) * fmaf(rest, 0.693147181f, 1.0f) *
                    (low ? 0x1p-64f : 1.0f);
    return g * (g < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}

__device__ inline f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ inline bf16x8 lds16(const uint8_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// Two transposing reads: lane l of 16 gets column l of the 4 x 16 elements that
// its 16 lanes point at (8 bytes each), from `p` and from `p` + `next`.  (`p` is
// restrict so that the reads carry alias information: without any the compiler
// waits for all copies to LDS under way before each.)
__device__ inline __attribute__((always_inline)) bf16x8 lds_across(const uint8_t* __restrict__ p,
                                                                   int next) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(p + next));
    return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// ---- Small tiles ------------------------------------------------------------------
// 64 x 64 outputs a workgroup of four wavefronts, 32 x 32 each; four blocks of c
// of both operands in LDS, 16 KB each, three under way.  For few rows: bound by the
// weights' way from memory (one row at each of 8 experts, 7168 x 1792, 206 MB: 39 us,
// 5.3 TB/s).
//
// Rows along c that do not begin on 128-byte lines are copied by lines all the same: a
// row's chunk comes with block b's copies where it lies in the same line as the block's
// first chunk, else with block b + 1's, and is read from there.  That takes a fifth block
// in LDS.  Copies of 128 bytes across two lines would ask for both, for each of them
// twice (24 experts of 1808 x 2184, 1436 rows falling off as 1 / rank: forward 56 us, by
// blocks 71; of 1808 x 2208, on half lines, 56 : 62).  Where all rows begin on lines,
// four blocks with nothing to look up: 39 us for the one row an expert above, against 40.
constexpr int kSmall = 64;
constexpr int kSmallBytes = 2 * kSmall * 128;
constexpr int kSmallThreads = 256;
// Across, the tiles beside each other share lines at their border where rows do not
// begin on lines.  Workgroups go to the eight XCDs in turn: each gets runs of this many
// tiles, so that such a line comes to its L2 once (rows' gradient, 8 experts of 7168 x
// 1800, one row each: 59 us one by one, 44 in eights; 16384 rows of 32 experts of 512 x
// 1032, weights' gradient: 66 and 57; where rows begin on lines mostly within 3 %, 4 experts
// of 5120 x 5120, 300 rows falling off, 86 and 78).
constexpr int kRun = 8;

template <int MODE, bool LINES>
__global__ __launch_bounds__(kSmallThreads, 2) void bf16_small_kernel(Bf16Args a) {
    constexpr bool kPAcross = MODE == kRowsBack || MODE == kWeightBack;
    constexpr bool kQAcross = MODE == kWeightBack;
    constexpr int kStages = LINES ? 4 : 5, kNeeded = LINES ? 1 : 2;
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[kStages * kSmallBytes];
    if (blockIdx.x == 0) check_groups(a.group_offset, a.G, a.M, a.st);
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int wp = wave % 2, wq = wave / 2, r = lane % 16, g = lane / 16;

    for (int64_t place = blockIdx.x; place < a.places; place += gridDim.x) {
        int64_t id = place;
        if constexpr (kPAcross) {
            id = (place / (8 * kRun) * 8 + place % 8) * kRun + place / 8 % kRun;
            if (id >= a.tiles) continue;
        }
        // where the tile lies: P from p0 on, Q from q0 on (for the weights'
        // gradient of expert e, else rows of e), c the `depth` values from c0 on
        const int p0 = (int)(id % a.tiles_w) * (MODE == kGate ? kSmall / 2 : kSmall);
        int64_t rest = id / a.tiles_w;
        int e, q_count;
        int64_t q0, c0 = 0, depth = a.C;
        if constexpr (MODE == kWeightBack) {
            q0 = (rest % a.tiles_v) * kSmall;
            e = (int)(rest / a.tiles_v);
            c0 = clamp_row(a.group_offset[e], a.M);
            depth = clamp_row(a.group_offset[e + 1], a.M) - c0;
            depth = depth < 0 ? 0 : depth;
            q_count = a.V - (int)q0 < kSmall ? a.V - (int)q0 : kSmall;
        } else {
            const RowTile tile = find_tile(a.group_offset, a.G, a.M, rest, kSmall);
            if (tile.g < 0) continue;
            e = tile.g;
            q0 = tile.first;
            q_count = tile.count;
        }
        const int blocks = (int)((depth + kDepth - 1) / kDepth);

        // Copies: lane's 16 bytes are chunk `lane % 8` of row 8 (2 wave + i) + lane / 8
        // of 128 bytes in LDS, i = 0, 1.  Along c: the row is an index of P (Q), and
        // its chunk c sits at c ^ (row / 2 % 8), so that 16 rows' reads of one chunk
        // meet all 64 banks once.  Across: the row is a c, and the pairs of chunks that
        // a 16-column tile takes sit at pair ^ f, f = (c / 2) % 2 + 2 (c / 8 % 2), so
        // that the 8 rows which half a wavefront reads meet all banks once.
        // Buffers end behind the last valid row: the rest reads as zero.  Columns
        // behind a row's last value read the next row's, for outputs that are not
        // stored; c behind the last is masked.
        const int row = wave * 16 + lane / 8;
        const int prow = MODE == kGate ? lane / 8 : row;
        const int along = (lane % 8) ^ (lane / 16), across = (lane % 8) ^ (lane / 16 % 2 * 2);
        __amdgpu_buffer_rsrc_t pbuf, qbuf;
        // Chunks of 16 bytes from the beginning of a line to that of a row along c
        const auto behind_line = [](const uint16_t* x, int64_t row, int pitch) {
            return LINES ? 0 : (int)(((uintptr_t)(x + row * pitch) >> 4) & 7);
        };
        int p_from[2] = {0, 0}, q_from[2] = {0, 0};   // the copied row's chunk, in block 0
        const auto from = [](int c, int behind) { return c + behind < 8 ? c : c - 8; };
        if constexpr (!kPAcross) {
            int first = p0, extent = a.W, most = kSmall;
            if constexpr (MODE == kGate) {    // a wavefront copies 16 gates or 16 ups
                first = p0 + wave / 2 * 16 + wave % 2 * (a.W / 2);
                extent = (wave % 2 + 1) * (a.W / 2);
                most = 16;
            }
            first = first < extent ? first : extent - 1;
            const int rows = extent - first < most ? extent - first : most;
            pbuf = buffer_rsrc(const_cast<uint16_t*>(a.p) + ((int64_t)e * a.W + first) * a.pitch_p,
                               rows * a.pitch_p * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p_from[i] = from(along ^ (4 * i),
                                 behind_line(a.p, (int64_t)e * a.W + first + prow + 8 * i, a.pitch_p));
        }
        if constexpr (!kQAcross) {
            qbuf = buffer_rsrc(const_cast<uint16_t*>(a.q) + q0 * a.pitch_q, q_count * a.pitch_q * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                q_from[i] = from(along ^ (4 * i), behind_line(a.q, q0 + row + 8 * i, a.pitch_q));
        }
        const auto fetch = [&](int b, int stage) {
            uint8_t* l = s_mem + stage * kSmallBytes + wave * 2048;
            const int chunk = b * 8, chunks = (int)(depth / 8);   // depth: a multiple of 8, or across
            b = b < blocks ? b : blocks - 1;  // across: repeated behind the last block
            const int64_t left = depth - (int64_t)b * kDepth;
            const int rows = left < kDepth ? (int)left : kDepth;
            if constexpr (kPAcross) {
                const int64_t from = MODE == kRowsBack ? (int64_t)e * a.C : c0;
                pbuf = buffer_rsrc(const_cast<uint16_t*>(a.p) +
                                       (from + (int64_t)b * kDepth) * a.pitch_p + p0,
                                   (rows * a.pitch_p - p0) * 2);
            }
            if constexpr (kQAcross)
                qbuf = buffer_rsrc(const_cast<uint16_t*>(a.q) +
                                       (c0 + (int64_t)b * kDepth) * a.pitch_q + q0,
                                   (rows * a.pitch_q - (int)q0) * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t at = (uint32_t)((prow + 8 * i) * a.pitch_p * 2);
                if constexpr (kPAcross)
                    to_lds(pbuf, at + (across ^ (4 * i)) * 16, 0, l + i * 1024);
                else
                    to_lds(pbuf, (uint32_t)(chunk + p_from[i]) < (uint32_t)chunks
                                     ? at + (chunk + p_from[i]) * 16 : 0x80000000u, 0, l + i * 1024);
                at = (uint32_t)((row + 8 * i) * a.pitch_q * 2);
                if constexpr (kQAcross)
                    to_lds(qbuf, at + (across ^ (4 * i)) * 16, 0, l + kSmall * 128 + i * 1024);
                else
                    to_lds(qbuf, (uint32_t)(chunk + q_from[i]) < (uint32_t)chunks
                                     ? at + (chunk + q_from[i]) * 16 : 0x80000000u, 0,
                           l + kSmall * 128 + i * 1024);
            }
        };

        f32x4 acc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int at0 = r * 128 + (g ^ (r / 2)) * 16;
        const int f = r / 8 + g % 2 * 2, at_across = (8 * g + r / 4) * 128 + r % 4 * 8;
        // how far behind its line's beginning each row of the lane's tiles begins
        int p_behind[2], q_behind[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tp = wp * 2 + i, tq = wq * 2 + i;
            const int64_t prow0 = MODE == kGate ? p0 + tp / 2 * 16 + tp % 2 * (a.W / 2) : p0 + tp * 16;
            p_behind[i] = behind_line(a.p, (int64_t)e * a.W + prow0 + r, a.pitch_p);
            q_behind[i] = behind_line(a.q, q0 + tq * 16 + r, a.pitch_q);
        }
        if (blocks > 0) {
#pragma unroll
            for (int s = 0; s < kStages - 1; ++s) {
                fetch(s, s);
                __builtin_amdgcn_sched_barrier(0);   // the meetings count on this order
            }
            int stage = 0;
            for (int b = 0; b < blocks; ++b) {
                // block b, and the next copies, which may hold the last of it, are here
                // when all but the two behind are; everyone is then done with block
                // b - 1, whose place the next copies take
                meet<4 * (kStages - 1 - kNeeded), 0>();
                fetch(b + kStages - 1, (stage + kStages - 1) % kStages);
                __builtin_amdgcn_sched_barrier(0);
                const int next = (stage + 1) % kStages;
                const uint8_t* lp = s_mem + stage * kSmallBytes;
                const uint8_t* lq = lp + kSmall * 128;
                const int later = (next - stage) * kSmallBytes;
                bf16x8 p[2][2], q[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int tp = wp * 2 + i, tq = wq * 2 + i;
                        if constexpr (kPAcross)
                            p[h][i] = lds_across(lp + h * 4096 + at_across + (tp ^ f) * 32, 512);
                        else
                            p[h][i] = lds16(lp + tp * 2048 + (at0 ^ (h * 64)) +
                                            (4 * h + g + p_behind[i] < 8 ? 0 : later));
                        if constexpr (kQAcross)
                            q[h][i] = lds_across(lq + h * 4096 + at_across + (tq ^ f) * 32, 512);
                        else
                            q[h][i] = lds16(lq + tq * 2048 + (at0 ^ (h * 64)) +
                                            (4 * h + g + q_behind[i] < 8 ? 0 : later));
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(p[h][i], q[h][j], acc[i][j]);
                stage = next;
            }
            meet<0, 0>();   // the copies behind the last block are in, its reads done
        }

#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int qi = wq * 32 + j * 16 + r;
            if (qi >= q_count) continue;
            const int64_t qrow = q0 + qi;
            if constexpr (MODE == kGate) {
                const int F = a.W / 2, c = p0 + wp * 16 + g * 4;
                if (c >= F) continue;
                const f32x4 gate = acc[0][j], up = acc[1][j];
                float h[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) h[v] = silu(gate[v]) * up[v];
                *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + qrow * F + c) =
                    u32x2{bf16_pack(h[0], h[1]), bf16_pack(h[2], h[3])};
                if (a.pre) {
                    uint16_t* pre = a.pre + qrow * a.W + c;
                    *reinterpret_cast<u32x2*>(pre) =
                        u32x2{bf16_pack(gate[0], gate[1]), bf16_pack(gate[2], gate[3])};
                    *reinterpret_cast<u32x2*>(pre + F) =
                        u32x2{bf16_pack(up[0], up[1]), bf16_pack(up[2], up[3])};
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = p0 + wp * 32 + i * 16 + g * 4;
                    if (c >= a.W) continue;
                    const f32x4 v = acc[i][j];
                    const int64_t at =
                        (MODE == kWeightBack ? (int64_t)e * a.V + qrow : qrow) * a.W + c;
                    if (MODE == kWeightBack && a.wide) {
                        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at) = v;
                    } else {
                        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
                            u32x2{bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3])};
                    }
                }
            }
        }
    }
}

// ---- Big tiles --------------------------------------------------------------------
// 256 x 256 outputs a workgroup of four wavefronts, one workgroup a CU, which works
// through its share of tiles.  The blocks of c of both operands, 32 KB each, go from
// memory to LDS ahead of their use, two blocks ahead and on into the next tile: three
// blocks of P and two of Q fill the 160 KB.  A wavefront, one on a SIMD, has 128 x 128
// results in all 256 accumulation registers: eight wavefronts of 128 x 64 read half as
// much again from LDS and took 5 % longer.
//
// Bound by the card's power: with random numbers in the operands a block takes 1.38 us
// (clock lowered to about 1.7 GHz), with zeros 1.06; a bare loop of these MFMAs (16 x 16 x
// 32; 32 x 32 x 16 draw more) reaches 2.0 PFLOP/s with random numbers.  8192 x 8192 x
// 7168, the card warm: forward 1.46 PFLOP/s, rows' gradient 1.33, weights' 1.33; the
// library's product of the same operands 1.6, 1.2, 0.9.  About 8 us a tile go to its
// beginning and end, 4 of them to stores, which all CUs have at once: 7680 rows of 8
// experts, 7168 x 1792, 184 to 192 us (1.03 to 1.07 PFLOP/s; 34 row tiles for 30 tiles' rows,
// and 3.7 rounds of the CUs run as four).
constexpr int kBig = 256;
constexpr int kBigThreads = 256;
constexpr int kBigCopies = 8;                   // a wavefront's copies of a block of an operand
constexpr int kBigTiles = 8;                    // its tiles of 16 along P, and along Q
constexpr int kBigGrid = 256;                   // CUs of the GPU: one workgroup fills a CU's LDS
constexpr int kOperandBytes = kBig * kDepth * 2;
constexpr int kQAt = 3 * kOperandBytes;         // LDS: three blocks of P, two of Q

// A value that all lanes have, in scalar registers whatever it was made from: what
// a buffer is made of has to be.
__device__ inline int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline bool uniform(bool v) { return __builtin_amdgcn_readfirstlane((int)v); }
__device__ inline int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int32_t)(v >> 32)) << 32 |
                     (uint32_t)uniform((int32_t)v));
}

// A workgroup's share of the weights' gradient's tiles, whose depths differ: the
// experts with most rows first, dealt to the workgroups there and back, so that
// who had the larger of one round has the smaller of the next.  Neighbours in a
// round are 32 workgroups of one XCD, bands of 5 tiles along V.  (Up to 64 experts
// are ordered, a lane each; with more, every workgroup has many.)
struct WeightShare {
    int64_t all, per_expert;      // per_expert: with its parts
    int32_t count, tiles_w, tiles_v, at;
    int32_t order;     // lane r: the expert with the r-th most rows

    __device__ WeightShare(const Bf16Args& a) {
        const int lane = lane_id();
        order = lane;
        if (a.G <= kWave) {
            int n = -1;
            if (lane < a.G) {
                const int64_t rows =
                    clamp_row(a.group_offset[lane + 1], a.M) - clamp_row(a.group_offset[lane], a.M);
                n = rows < 0 ? 0 : (int)rows;
            }
            int rank = 0;
            for (int g = 0; g < kWave; ++g) {
                const int m = bcast(n, g);
                rank += m > n || (m == n && g < lane);
            }
            order = __builtin_amdgcn_ds_permute(rank * 4, lane);
        }
        tiles_w = a.tiles_w;
        tiles_v = a.tiles_v;
        per_expert = (int64_t)tiles_w * tiles_v * a.splits;
        all = per_expert * a.G;
        at = (int)(blockIdx.x % 8u * (gridDim.x / 8u) + blockIdx.x / 8u);
        const int64_t rounds = all / gridDim.x;
        count = (int)rounds + (index((int)rounds) < all);
    }
    __device__ int64_t index(int i) const {
        return (int64_t)i * gridDim.x + (i % 2 ? (int)gridDim.x - 1 - at : at);
    }
    __device__ void place(const Bf16Args& a, int i, int* e, int* part, int* v, int* w) const {
        const int64_t id = index(i), r = id / per_expert;
        const int64_t one = (int64_t)tiles_w * tiles_v;
        *part = (int)((id - r * per_expert) / one);
        const int in = (int)((id - r * per_expert) % one), wide = kBand * tiles_w, band = in / wide;
        const int left = tiles_v - band * kBand, rows = left < kBand ? left : kBand;
        *e = a.G <= kWave ? bcast(order, (int)r) : (int)r;
        *v = band * kBand + (in - band * wide) % rows;
        *w = (in - band * wide) / rows;
    }
};

// A tile: P from p0 on, Q from q0 on (q_count of them), `depth` values of c, the
// first at c0.
struct BigTile {
    int64_t q0, c0, depth;
    int32_t e, part, p0, q_count, blocks;
};

template <int MODE, bool WIDE>
__global__ __launch_bounds__(kBigThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void bf16_big_kernel(Bf16Args a) {
    constexpr bool kPAcross = MODE == kRowsBack || MODE == kWeightBack;
    constexpr bool kQAcross = MODE == kWeightBack;
    constexpr bool kGateUp = MODE == kGate, kWeights = MODE == kWeightBack;
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[5 * kOperandBytes];
    if (blockIdx.x == 0) check_groups(a.group_offset, a.G, a.M, a.st);
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int wp = wave % 2, wq = wave / 2;
    const auto share = [&]() {
        if constexpr (kWeights) {
            return WeightShare(a);
        } else {
            // offsets that decrease can count rows many times: no more than M's tiles
            const int64_t counted = count_tiles(a.group_offset, a.G, a.M, kBig),
                          most = max_tiles(a.M, a.G, kBig);
            return TileShare(uniform(counted < most ? counted : most), a.tiles_w);
        }
    }();
    // the first 64 groups' offsets, a lane each: a tile's start costs no load then (its
    // wait would be a wait for the copies)
    int64_t lo = 0, rows_here = 0;
    if (lane < a.G) {
        lo = clamp_row(a.group_offset[lane], a.M);
        rows_here = clamp_row(a.group_offset[lane + 1], a.M) - lo;
        rows_here = rows_here < 0 ? 0 : rows_here;
    }
    const auto tile_at = [&](int i) {
        BigTile t;
        if constexpr (kWeights) {
            int v, w;
            share.place(a, i, &t.e, &t.part, &v, &w);
            t.p0 = w * kBig;
            t.q0 = (int64_t)v * kBig;
            t.q_count = a.V - v * kBig < kBig ? a.V - v * kBig : kBig;
            if (t.e < kWave) {
                t.c0 = bcast((int32_t)lo, t.e);
                t.depth = bcast((int32_t)rows_here, t.e);
            } else {
                t.c0 = clamp_row(a.group_offset[t.e], a.M);
                t.depth = clamp_row(a.group_offset[t.e + 1], a.M) - t.c0;
                if (t.depth < 0) t.depth = 0;
            }
            if (a.splits > 1) {     // whole blocks
                const int64_t blocks = (t.depth + kDepth - 1) / kDepth;
                const int64_t b0 = blocks * t.part / a.splits, b1 = blocks * (t.part + 1) / a.splits;
                const int64_t end = b1 * kDepth < t.depth ? b1 * kDepth : t.depth;
                t.depth = b0 < b1 ? end - b0 * kDepth : 0;
                t.c0 += b0 * kDepth;
            }
        } else {
            t.part = 0;
            int64_t m;
            int n;
            share.place(i, &m, &n);
            RowTile r{-1, 0, 0};
            int64_t before = 0;
            if (!find_in(lo, rows_here, 0, &before, m, kBig, &r) && a.G > kWave)
                r = find_tile(a.group_offset, a.G, a.M, m, kBig);
            t.e = r.g < 0 ? 0 : r.g;
            t.p0 = n * (kGateUp ? kBig / 2 : kBig);
            t.q0 = r.g < 0 ? 0 : r.first;
            t.q_count = r.g < 0 ? 0 : r.count;
            t.c0 = 0;
            t.depth = a.C;
        }
        t.q0 = uniform(t.q0);
        t.c0 = uniform(t.c0);
        t.depth = uniform(t.depth);
        t.e = uniform(t.e);
        t.part = uniform(t.part);
        t.p0 = uniform(t.p0);
        t.q_count = uniform(t.q_count);
        t.blocks = (int)((t.depth + kDepth - 1) / kDepth);
        return t;
    };

    // Where the copies stand: block `fb` of tile `ft`.  Along c a wavefront copies
    // rows 64 wave + 8 i + lane / 8 of an operand, chunk c of row q to chunk
    // c ^ (q / 2 % 8) of its 128 bytes.  Across, c's of a block are rows of 512 bytes,
    // two an instruction, 16 wave + 2 i + lane / 32; the 32 bytes of row c which a
    // tile of 16 columns takes sit at ^ f, f = c % 4 + 4 (c / 8 % 2), so that the
    // eight rows which half a wavefront reads meet all banks once.  The buffers' ends
    // and what lies behind them are as in the small tiles.
    int ft = 0, fb = 0;
    BigTile to{};
    __amdgpu_buffer_rsrc_t pbuf, qbuf;
    uint32_t op[4], oq[4];         // this lane's offsets, by i % 2 and, across, also i / 4 % 2
    const uint32_t pitch_p = (uint32_t)a.pitch_p * 2, pitch_q = (uint32_t)a.pitch_q * 2;
    const uint16_t *pb = nullptr, *qb = nullptr;    // across: where block fb begins
    const auto aim_block = [&]() {
        const int64_t left = to.depth - (int64_t)fb * kDepth;
        const int rows = left < kDepth ? (int)left : kDepth;
        if constexpr (kPAcross) {
            const int64_t from = kWeights ? to.c0 : (int64_t)to.e * a.C;
            pb = a.p + (from + (int64_t)fb * kDepth) * a.pitch_p + to.p0;
            pbuf = buffer_rsrc(const_cast<uint16_t*>(pb), (rows * a.pitch_p - to.p0) * 2);
        }
        if constexpr (kQAcross) {
            qb = a.q + (to.c0 + (int64_t)fb * kDepth) * a.pitch_q + to.q0;
            qbuf = buffer_rsrc(const_cast<uint16_t*>(qb), (rows * a.pitch_q - (int)to.q0) * 2);
        }
        if (!kQAcross && a.C % kDepth != 0 && (fb == 0 || fb == to.blocks - 1)) {
            // c behind the last is masked: only in a last block, undone in a first
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = (lane % 8) ^ (lane / 16) ^ (4 * i);
                // (the sign, not a choice: that becomes a branch, and what follows divergent)
                const uint32_t past = (uint32_t)(rows / 8 - 1 - c) & 0x80000000u;
                if constexpr (!kPAcross) op[i] = ((uint32_t)(lane / 8) * pitch_p + c * 16) | past;
                oq[i] = ((uint32_t)(wave * 8 * kBigCopies + lane / 8) * pitch_q + c * 16) | past;
            }
        }
    };
    const auto aim = [&]() {
        if constexpr (!kPAcross) {
            // this wavefront's rows of P: for the gate some of the 64 gates or 64 ups that 128
            // rows have
            constexpr int kRows = 8 * kBigCopies;
            const int at = wave * kRows, half = kGateUp ? at % 128 / 64 : 0, F = a.W / 2;
            const int first = kGateUp ? half * F + to.p0 + at / 128 * 64 + at % 64 : to.p0 + at;
            const int extent = kGateUp ? (half + 1) * F : a.W;
            const int base = first < extent ? first : extent - 1;
            const int rows = extent - base < kRows ? extent - base : kRows;
            pbuf = buffer_rsrc(const_cast<uint16_t*>(a.p) + ((int64_t)to.e * a.W + base) * a.pitch_p,
                               rows * a.pitch_p * 2);
        }
        if constexpr (!kQAcross)
            qbuf = buffer_rsrc(const_cast<uint16_t*>(a.q) + to.q0 * a.pitch_q,
                               (to.q_count < 1 ? 1 : to.q_count) * a.pitch_q * 2);
        aim_block();
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = (lane % 8) ^ (lane / 16) ^ (i % 2 * 4);
        op[i] = (uint32_t)(lane / 8) * pitch_p + c * 16;
        oq[i] = (uint32_t)(wave * 8 * kBigCopies + lane / 8) * pitch_q + c * 16;
        if constexpr (kPAcross)
            op[i] = (uint32_t)(wave * 2 * kBigCopies + lane / 32) * pitch_p +
                    ((lane % 32) ^ (lane / 32 * 2) ^ (i % 2 * 4) ^
                     (i / 2 * 8)) * 16;
        if constexpr (kQAcross)
            oq[i] = (uint32_t)(wave * 2 * kBigCopies + lane / 32) * pitch_q +
                    ((lane % 32) ^ (lane / 32 * 2) ^ (i % 2 * 4) ^
                     (i / 2 * 8)) * 16;
    }
    // behind the last tile the copies repeat its last block
    const auto advance = [&]() {
        if (uniform(++fb < to.blocks)) return aim_block();
        int next = ft + 1;
        BigTile t{};
        for (; next < share.count; ++next) {
            t = tile_at(next);
            if (!kWeights || t.blocks > 0) break;
        }
        if (uniform(next < share.count)) {
            ft = next;
            to = t;
            fb = 0;
            aim();
        } else {
            fb = to.blocks - 1;
            aim_block();
        }
    };
    // The same for a block that is neither its tile's first nor its last, without a branch:
    // nothing changes but where it begins.  on: 1, or 0 to stay.
    const auto step = [&](int on) {
        fb += on;
        if constexpr (kPAcross) {
            pb += (int64_t)(on * kDepth) * a.pitch_p;
            pbuf = buffer_rsrc(const_cast<uint16_t*>(pb), (kDepth * a.pitch_p - to.p0) * 2);
        }
        if constexpr (kQAcross) {
            qb += (int64_t)(on * kDepth) * a.pitch_q;
            qbuf = buffer_rsrc(const_cast<uint16_t*>(qb), (kDepth * a.pitch_q - (int)to.q0) * 2);
        }
    };
    const auto fetch_p = [&](uint32_t at, int i) {
        to_lds(pbuf, op[kPAcross ? i % 2 + i / 4 * 2 : i % 2] + (uint32_t)i * (kPAcross ? 2 : 8) * pitch_p,
               kPAcross ? 0 : fb * 128, s_mem + at + (wave * kBigCopies + i) * 1024);
    };
    const auto fetch_q = [&](uint32_t at, int i) {
        to_lds(qbuf, oq[kQAcross ? i % 2 + i / 4 * 2 : i % 2] + (uint32_t)i * (kQAcross ? 2 : 8) * pitch_q,
               kQAcross ? 0 : fb * 128, s_mem + at + (wave * kBigCopies + i) * 1024);
    };

    // Reads: lane's column of P (Q) is r = lane % 16 of a tile of 16, its c's are 8 g on,
    // g = lane / 16, in each half of a block.
    const int r = lane % 16, g = lane / 16;
    const int along = r * 128 + (g ^ (r / 2)) * 16;
    const int fold = r / 4 + g % 2 * 4, across = (8 * g + r / 4) * 512 + r % 4 * 8;
    const int across_p = across + ((wp * 8) ^ fold) * 32, across_q = across + ((wq * kBigTiles) ^ fold) * 32;
    const auto ptile = [&](uint32_t at, int i, int h) {
        if constexpr (kPAcross)
            return lds_across(s_mem + at + (across_p ^ (i * 32)) + h * 16384, 2048);
        else
            return lds16(s_mem + at + wp * 16384 + i * 2048 + (along ^ (h * 64)));
    };
    const auto qtile = [&](uint32_t at, int j, int h) {
        if constexpr (kQAcross)
            return lds_across(s_mem + at + (across_q ^ (j * 32)) + h * 16384, 2048);
        else
            return lds16(s_mem + at + (wq * kBigTiles + j) * 2048 + (along ^ (h * 64)));
    };

    // the first tile with a block
    bool any = false;
    for (; ft < share.count && !any; ft += !any) {
        to = tile_at(ft);
        any = to.blocks > 0;
    }

    // places of this, the next and the over-next block
    uint32_t p_at[3] = {0, kOperandBytes, 2 * kOperandBytes};
    uint32_t q_at[2] = {kQAt, kQAt + kOperandBytes};
    f32x4 acc[8][kBigTiles];
    bf16x8 p[4][2], q[2][kBigTiles];
    if (any) {
        aim();
#pragma unroll
        for (int i = 0; i < kBigCopies; ++i) {
            fetch_p(p_at[0], i);
            fetch_q(q_at[0], i);
        }
        advance();
#pragma unroll
        for (int i = 0; i < kBigCopies; ++i) {
            fetch_p(p_at[1], i);
            fetch_q(q_at[1], i);
        }
        meet<0, 0>();
        advance();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < kBigTiles; ++j) q[h][j] = qtile(q_at[0], j, h);
            p[0][h] = ptile(p_at[0], 0, h);
            p[1][h] = ptile(p_at[0], 1, h);
        }
    }

    // One block: eight P tiles i, sixteen MFMAs n each.  There is one wavefront on a SIMD:
    // what else it has to issue goes between the MFMAs, a little at a time.  P is read
    // two tiles ahead.  The copies of the block two ahead go out at an even pace, two a
    // row, P's and then Q's (all sixteen in rows 0 to 5: 7 % slower where the operands do
    // not fit the last-level cache, in rows 0 to 3: 18 %).  Two meetings: at i = 1 every
    // wavefront has its Q in registers, and their place may take the next copies; at i = 6
    // every wavefront has read its P and the next block has arrived (all but the twelve
    // copies that this block has sent out so far).  The last two rows go by columns, so
    // that Q of the next block can replace this one's over 32 MFMAs, each tile after its
    // last use.
    // A tile's first block begins from zero, and finds its next block there already: it
    // was waited for ahead of the last tile's stores, which need not end before.
    const auto block = [&](auto first) {
        const auto add = [&](int i, int h, int j) {
            const bool zero = first.value && h == 0;
            acc[i][j] = mfma_bf16(p[i % 4][h], q[h][j], zero ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j]);
        };
        constexpr int kReads = kPAcross ? 4 : 2;    // LDS reads of a tile of P
        const bool inner = uniform(fb + 2 < to.blocks);      // the copies go on within their tile
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            // the reads of P tile 2 may be under way, not Q's
            if (i == 1) meet<63, kReads>();
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                const int h = n / 8, j = n % 8;
                __builtin_amdgcn_sched_barrier(0);
                add(i, h, j);
                __builtin_amdgcn_sched_barrier(0);
                if (n == 1 || n == 4) p[(i + 2) % 4][n / 4] = ptile(p_at[0], i + 2, n / 4);
                if (n % 8 == 6 && i < 4) fetch_p(p_at[2], 2 * i + n / 8);
                if (n % 8 == 6 && i >= 4) fetch_q(q_at[0], 2 * i - 8 + n / 8);
            }
        }
        meet<first.value ? 63 : 12, 0>();
#pragma unroll
        for (int n = 0; n < 32; ++n) {
            const int j = n / 4, h = n / 2 % 2, i = 6 + n % 2;
            __builtin_amdgcn_sched_barrier(0);
            add(i, h, j);
            __builtin_amdgcn_sched_barrier(0);
            if (n == 1 || n == 4) p[0][n / 4] = ptile(p_at[1], 0, n / 4);
            if (n == 8 || n == 12) p[1][n / 4 - 2] = ptile(p_at[1], 1, n / 4 - 2);
            if (n % 8 == 6) fetch_q(q_at[0], 4 + n / 8);
            if (n == 31) step(inner);
            if (n >= 5 && n % 2 == 1) q[n / 2 % 2][n / 4 - 1] = qtile(q_at[1], n / 4 - 1, n / 2 % 2);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) q[h][7] = qtile(q_at[1], 7, h);
        if (!inner) advance();
        const uint32_t p0 = p_at[0], q0 = q_at[0];
        p_at[0] = p_at[1];
        p_at[1] = p_at[2];
        p_at[2] = p0;
        q_at[0] = q_at[1];
        q_at[1] = q0;
    };

    for (int ti = 0; ti < share.count; ++ti) {
        const BigTile t = tile_at(ti);
        if (kWeights && t.blocks == 0) {      // an expert without rows
            const int vecs = (a.W - t.p0 < kBig ? a.W - t.p0 : kBig) / 8;
            for (int i = (int)threadIdx.x; i < t.q_count * (kBig / 8); i += kBigThreads) {
                const int c = i % (kBig / 8);
                if (c >= vecs) continue;
                const int64_t at =
                    (((int64_t)t.part * a.G + t.e) * a.V + t.q0 + i / (kBig / 8)) * a.W + t.p0 +
                    c * 8;
                u32x4* out = reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(a.out) +
                                                      at * (WIDE ? 4 : 2));
                out[0] = u32x4{0, 0, 0, 0};
                if (WIDE) out[1] = u32x4{0, 0, 0, 0};
            }
            continue;
        }
        block(std::true_type{});
        for (int b = 1; b < t.blocks; ++b) block(std::false_type{});
        wait_vm();    // the next tile's first two blocks
        {
            // (opaque: addresses made from them are not worth registers in the loop.  The
            // empty statements below keep the results in the accumulation registers until
            // their turn: all of them at once do not fit the others.)
            int row = lane % 16, group = lane / 16;
            asm volatile("" : "+v"(row), "+v"(group));
#pragma unroll
            for (int j = 0; j < kBigTiles; ++j) {
                const int qi = (wq * kBigTiles + j) * 16 + row;
                const int64_t qrow = t.q0 + qi;
                const bool in = qi < t.q_count;
                // A lane has columns 4 group .. 4 group + 3 of each 16: two neighbouring
                // tiles' halves change hands, so that it has 8 of one of them.
                const auto store8 = [&](const f32x4& v, const f32x4& w, uint16_t* out, int first,
                                        int end) {
                    __builtin_amdgcn_sched_barrier(0);   // few results at a time
                    const u32x2 lo = __builtin_amdgcn_permlane16_swap(
                        bf16_pack(v[0], v[1]), bf16_pack(w[0], w[1]), false, false);
                    const u32x2 hi = __builtin_amdgcn_permlane16_swap(
                        bf16_pack(v[2], v[3]), bf16_pack(w[2], w[3]), false, false);
                    const int c = first + group % 2 * 16 + group / 2 * 8;
                    if (in && c < end)
                        *reinterpret_cast<u32x4*>(out + c) = u32x4{lo[0], hi[0], lo[1], hi[1]};
                };
                if constexpr (kGateUp) {
                    const int F = a.W / 2;
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const int first = t.p0 + wp * 64 + i * 16;
                        asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i + 1][j]),
                                     "+a"(acc[i + 4][j]), "+a"(acc[i + 5][j]));
                        if (a.pre) {
                            uint16_t* pre = a.pre + qrow * a.W;
                            store8(acc[i][j], acc[i + 1][j], pre, first, F);
                            store8(acc[i + 4][j], acc[i + 5][j], pre + F, first, F);
                        }
                        f32x4 h[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                h[k][v] = silu(acc[i + k][j][v]) * acc[i + k + 4][j][v];
                        store8(h[0], h[1], reinterpret_cast<uint16_t*>(a.out) + qrow * F, first, F);
                    }
                } else {
                    const int64_t at =
                        (kWeights ? ((int64_t)t.part * a.G + t.e) * a.V + qrow : qrow) * a.W;
                    const int first = t.p0 + wp * 128;
                    if constexpr (WIDE) {
                        float* out = reinterpret_cast<float*>(a.out) + at;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            asm volatile("" : "+a"(acc[i][j]));
                            const int c = first + i * 16 + group * 4;
                            if (in && c < a.W) *reinterpret_cast<f32x4*>(out + c) = acc[i][j];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i + 1][j]));
                            store8(acc[i][j], acc[i + 1][j], reinterpret_cast<uint16_t*>(a.out) + at,
                                   first + i * 16, a.W);
                        }
                    }
                }
            }
        }
    }
    wait_vm();   // no copy may reach the LDS after the workgroup's end
}

// The parts of a weights' gradient, added in their order.
struct JoinArgs {
    const f32x4* parts;
    void* out;
    int64_t n;        // vectors of 4
    int32_t splits;
    bool wide;
};

__global__ __launch_bounds__(256) void weight_join_kernel(JoinArgs a) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n; i += (int64_t)gridDim.x * 256) {
        f32x4 v = a.parts[i];
        for (int s = 1; s < a.splits; ++s) v += a.parts[s * a.n + i];
        if (a.wide)
            reinterpret_cast<f32x4*>(a.out)[i] = v;
        else
            reinterpret_cast<u32x2*>(a.out)[i] =
                u32x2{bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3])};
    }
}

// ---- The gate's backward ------------------------------------------------------------
// grad_gate = d * u * s * (1 + g * (1 - s)), grad_up = d * g * s, s = sigmoid(g).
// A thread has eight outputs of a row at a time, 2^tpr_log threads a row.  Bound by memory.
// d's products come first: of two bf16 values they are exact in float.  Each
// operation is rounded by itself (no fused multiply-add), as elementary float
// operations are.
__device__ inline void gate_back(float& gate, float& up, float d) {
#pragma clang fp contract(off)
    const float s = sigmoid(gate), g = gate;
    gate = d * up * s * (1.0f + g * (1.0f - s));
    up = d * g * s;
}

struct GateBackArgs {
    const u32x4* pre;        // [M, 2F/8]
    const u32x4* grad_out;   // [M, F/8]
    u32x4* grad_pre;
    const int32_t* group_offset;
    int32_t* st;
    int64_t M;
    int32_t G, nv, tpr_log;
};

__global__ __launch_bounds__(256) void gate_back_kernel(GateBackArgs a) {
    if (blockIdx.x == 0) check_groups(a.group_offset, a.G, a.M, a.st);
    const int64_t lo = clamp_row(a.group_offset[0], a.M), end = clamp_row(a.group_offset[a.G], a.M);
    const int tpr = 1 << a.tpr_log, rpb = 256 >> a.tpr_log;
    for (int64_t m = lo + (int64_t)blockIdx.x * rpb + ((int)threadIdx.x >> a.tpr_log); m < end;
         m += (int64_t)gridDim.x * rpb) {
        for (int c = (int)threadIdx.x & (tpr - 1); c < a.nv; c += tpr) {
            float gate[8], up[8], d[8];
            unpack8(a.pre[m * 2 * a.nv + c], gate);
            unpack8(a.pre[m * 2 * a.nv + a.nv + c], up);
            unpack8(a.grad_out[m * a.nv + c], d);
#pragma unroll
            for (int q = 0; q < 8; ++q) gate_back(gate[q], up[q], d[q]);
            a.grad_pre[m * 2 * a.nv + c] = pack8(gate);
            a.grad_pre[m * 2 * a.nv + a.nv + c] = pack8(up);
        }
    }
}

constexpr int kMaxDim = 1 << 20;   // K and N: a tile's rows stay within 32-bit offsets

int check_bf16(int32_t G, int64_t M, int32_t N, int32_t K) {
    if (G < 1 || G > kMaxE || M < 0 || M >= ((int64_t)1 << 31)) return EP_ERR_INVALID_ARG;
    if (K < 8 || K % 8 != 0 || K > kMaxDim || N < 8 || N % 8 != 0 || N > kMaxDim)
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Parts of c that a weights' gradient is cut into: as many as give every CU a big tile,
// but at least eight blocks of the average expert's rows each.
int32_t weight_splits(int32_t G, int64_t M, int32_t N, int32_t K) {
    const int64_t tiles = (int64_t)G * ceil_div(N, kBig) * ceil_div(K, kBig);
    const int64_t most = ceil_div(ceil_div(M, G), 8 * kDepth);
    const int64_t want = kBigGrid / tiles;
    return (int32_t)(want < most ? (want < 1 ? 1 : want) : (most < 1 ? 1 : most));
}

}  // namespace ep

using namespace ep;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

int common_args(Bf16Args& a, int32_t G, int64_t M, const int32_t* group_offset, int32_t* st) {
    if (!group_offset || !st || (((uintptr_t)group_offset | (uintptr_t)st) & 3))
        return EP_ERR_INVALID_ARG;
    a.group_offset = group_offset;
    a.st = st;
    a.M = M;
    a.G = G;
    a.splits = 1;
    return EP_OK;
}

template <int MODE>
int launch_small(Bf16Args& a, hipStream_t stream) {
    a.tiles_w = (int32_t)(MODE == kGate ? ceil_div(a.W / 2, kSmall / 2) : ceil_div(a.W, kSmall));
    if (MODE == kWeightBack) {
        a.tiles_v = (int32_t)ceil_div(a.V, kSmall);
        a.tiles = (int64_t)a.G * a.tiles_v * a.tiles_w;
    } else {
        a.tiles = max_tiles(a.M, a.G, kSmall) * a.tiles_w;
    }
    clear_hip_error();
    a.places = MODE == kRowsBack || MODE == kWeightBack ? ceil_div(a.tiles, 8 * kRun) * 8 * kRun : a.tiles;
    const dim3 grid(loop_grid(a.places, kSmallThreads));
    const uint64_t lines = (uintptr_t)a.p | (uintptr_t)a.q | (uint64_t)a.pitch_p * 2 | (uint64_t)a.pitch_q * 2;
    if constexpr (MODE == kForward || MODE == kGate) {
        if (lines % 128 != 0) {
            hipLaunchKernelGGL((bf16_small_kernel<MODE, false>), grid, dim3(kSmallThreads), 0, stream, a);
            EP_HIP_CHECK(hipGetLastError());
            return EP_OK;
        }
    }
    hipLaunchKernelGGL((bf16_small_kernel<MODE, true>), grid, dim3(kSmallThreads), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

// A workgroup a CU, or, for fewer tiles, one each, in whole eights for the XCDs
// that share them out.
template <int MODE, bool WIDE>
int launch_big(Bf16Args& a, hipStream_t stream) {
    a.tiles_w = (int32_t)(MODE == kGate ? ceil_div(a.W / 2, kBig / 2) : ceil_div(a.W, kBig));
    if (MODE == kWeightBack) {
        a.tiles_v = (int32_t)ceil_div(a.V, kBig);
        a.tiles = (int64_t)a.G * a.splits * a.tiles_v * a.tiles_w;
    } else {
        a.tiles = max_tiles(a.M, a.G, kBig) * a.tiles_w;
    }
    if (a.tiles >= ((int64_t)1 << 31)) {
        record_error("expert product: more than 2^31 tiles");
        return EP_ERR_INVALID_ARG;
    }
    clear_hip_error();
    hipLaunchKernelGGL((bf16_big_kernel<MODE, WIDE>),
                       dim3((unsigned)(a.tiles < kBigGrid ? ceil_div(a.tiles, 8) * 8 : kBigGrid)),
                       dim3(kBigThreads), 0, stream, a);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

// Which tiles take less time, from what each kind costs (ns):
//   small  the weights once from memory (5.4 TB/s) or once for every 64 rows from cache
//          (7.5 TB/s), for the rows' gradient a third more where the weights' rows do not
//          begin on lines; 4 us
//   big    rounds of tiles over the CUs, 1.25 us a block of c; 10 us, for the gate 20; no
//          less than the weights at 4.4 TB/s
// Small : big, us, as measured (rows an expert; e: even, s: falling off as 1 / rank):
//   forward, 8 experts of 7168 x 1792   1  39 : 47   32 e  43 : 46   64 e 50 : 46   256 e 118 : 55
//   forward, 8 of 3584 x 7168          64 e  91 : 139  128 e 144 : 143  192 s 198 : 146
//   forward, 24 of 1808 x 2184         16 e  41 : 62    64 s  62 : 72   256 e 139 : 78
//   forward, 1 of 7168 x 1792         512  29 : 44    32 of 512 x 1024  128 e 18 : 27  512 s 50 : 32
//   rows, 8 of 7168 x 1792             64 e  49 : 133  256 e 138 : 156  512 s 247 : 156
//   rows, 8 of 3584 x 7168              1  83 : 79   128 e 155 : 86
//   rows, 8 of 7168 x 1800              1  44 : 141  256 e 166 : 142   64 e of 24 of 1808 x 2184 63 : 47
// (The bound by the weights is too high for the rows' gradient of 3584 x 7168: 98 us for the
// 79 that big tiles take with one row an expert.  The small ones it takes there are 5 % slower.)
template <int MODE>
bool big_takes_less(const Bf16Args& a) {
    const double experts = a.G < a.M ? a.G : (double)a.M;     // that can have rows
    const double weights = 2.0 * a.W * a.C;
    const double per64 = (double)(a.M / kSmall) + 0.5 * experts;
    double small = fmax(experts * weights / 5400.0, per64 * weights / 7500.0);
    if (MODE == kRowsBack && a.pitch_p % kDepth != 0) small *= 4.0 / 3.0;
    const double row_tiles = fmax(experts, (double)(a.M / kBig) + 0.5 * experts);
    const double columns = MODE == kGate ? ceil_div(a.W / 2, kBig / 2) : ceil_div(a.W, kBig);
    const double rounds = ceil(row_tiles * columns / kBigGrid);
    const double big = rounds * ceil_div(a.C, kDepth) * 1250.0 + (MODE == kGate ? 20000.0 : 10000.0);
    return fmax(big, experts * weights / 4400.0 + 5000.0) <= small + 4000.0;
}

template <int MODE>
bool takes_big(const Bf16Args& a) {
    return big_takes_less<MODE>(a);
}

// The weights' gradient: big tiles write it faster (8 rows of 8 experts, 7168 x 1792:
// 52 : 145 us) and, in parts, take a long sum apart.  Only where an expert's few tiles may
// have many of the rows, no tile can be dealt against them: small ones there (32 experts of
// 512 x 1024, 256 rows each, falling off as 1 / rank 37 : 50 us, even 36 : 20; 512 each 51 :
// 87 and 50 : 26).
template <>
bool takes_big<kWeightBack>(const Bf16Args& a) {
    const int64_t tiles = (int64_t)a.G * a.splits * ceil_div(a.V, kBig) * ceil_div(a.W, kBig);
    return a.G == 1 || a.splits > 1 || tiles >= 2 * kBigGrid || a.M < 32 * kBig;
}

template <int MODE>
int launch(Bf16Args& a, hipStream_t stream) {
    if (!takes_big<MODE>(a)) return launch_small<MODE>(a, stream);
    if constexpr (MODE == kWeightBack)
        if (a.wide) return launch_big<MODE, true>(a, stream);
    return launch_big<MODE, false>(a, stream);
}

// What the rules look at, of the products from rows [M, K] and weights [G, N, K].
void forward_sizes(Bf16Args& a, int32_t N, int32_t K) {
    a.W = N;
    a.C = a.pitch_p = a.pitch_q = K;
}
void rows_back_sizes(Bf16Args& a, int32_t N, int32_t K) {
    a.W = a.pitch_p = K;
    a.C = a.pitch_q = N;
}
void weight_back_sizes(Bf16Args& a, int32_t N, int32_t K) {
    a.W = a.pitch_p = K;
    a.V = a.pitch_q = N;
    a.splits = weight_splits(a.G, a.M, N, K);
}

int forward(int32_t G, int64_t M, int32_t N, int32_t K, const void* rows,
            const int32_t* group_offset, const void* w, void* pre, void* out, int32_t* dev_status,
            bool gate, hipStream_t stream) {
    int v = check_bf16(G, M, N, K);
    if (v != EP_OK) return v;
    Bf16Args a{};
    v = common_args(a, G, M, group_offset, dev_status);
    if (v != EP_OK) return v;
    if (!w || (M > 0 && (!rows || !out))) return EP_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(rows) || !aligned16(out) || !aligned16(pre))
        return EP_ERR_INVALID_ARG;
    if (M == 0) return EP_OK;
    a.p = reinterpret_cast<const uint16_t*>(w);
    a.q = reinterpret_cast<const uint16_t*>(rows);
    a.out = out;
    a.pre = reinterpret_cast<uint16_t*>(pre);
    forward_sizes(a, N, K);
    return gate ? launch<kGate>(a, stream) : launch<kForward>(a, stream);
}

int check_backward(bool any, int32_t dtype, const void* rows, const void* w, const void* grad_rows,
                   const void* grad_w) {
    if (dtype != EP_BF16 && dtype != EP_F32) return EP_ERR_INVALID_ARG;
    if (grad_rows && !w) return EP_ERR_INVALID_ARG;
    if (grad_w && any && !rows) return EP_ERR_INVALID_ARG;
    if (!aligned16(rows) || !aligned16(w) || !aligned16(grad_rows) || !aligned16(grad_w))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Both gradients, the arguments checked.
int backward(Bf16Args a, int32_t N, int32_t K, int32_t dtype, const void* rows, const void* w,
             const void* grad_out, void* grad_rows, void* grad_w, void* workspace,
             hipStream_t stream) {
    a.q = reinterpret_cast<const uint16_t*>(grad_out);
    if (grad_rows && a.M > 0) {
        rows_back_sizes(a, N, K);
        a.p = reinterpret_cast<const uint16_t*>(w);
        a.out = grad_rows;
        const int v = launch<kRowsBack>(a, stream);
        if (v != EP_OK) return v;
    }
    if (!grad_w) return EP_OK;
    weight_back_sizes(a, N, K);
    a.p = reinterpret_cast<const uint16_t*>(rows);
    a.wide = dtype == EP_F32 || a.splits > 1;
    a.out = a.splits > 1 ? workspace : grad_w;
    const int v = launch<kWeightBack>(a, stream);
    if (v != EP_OK || a.splits == 1) return v;
    JoinArgs j{};
    j.parts = reinterpret_cast<const f32x4*>(workspace);
    j.out = grad_w;
    j.n = (int64_t)a.G * N * K / 4;
    j.splits = a.splits;
    j.wide = dtype == EP_F32;
    const int64_t blocks = ceil_div(j.n, 256);
    clear_hip_error();
    hipLaunchKernelGGL(weight_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                       0, stream, j);
    EP_HIP_CHECK(hipGetLastError());
    return EP_OK;
}

int check_workspace(int32_t G, int64_t M, int32_t N, int32_t K, const void* workspace,
                    size_t workspace_bytes) {
    const size_t need = ep_expert_backward_workspace_bytes(G, M, N, K);
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}
}  // namespace

extern "C" int ep_expert_product_bf16(int32_t G, int64_t M, int32_t N, int32_t K, const void* rows,
                                      const int32_t* group_offset, const void* w, void* out,
                                      int32_t* dev_status, hipStream_t stream) {
    return forward(G, M, N, K, rows, group_offset, w, nullptr, out, dev_status, false, stream);
}

extern "C" int ep_expert_gate_up_bf16(int32_t G, int64_t M, int32_t F, int32_t K, const void* rows,
                                      const int32_t* group_offset, const void* w, void* pre,
                                      void* out, int32_t* dev_status, hipStream_t stream) {
    if (F < 8 || F % 8 != 0 || F > kMaxDim / 2) return EP_ERR_INVALID_ARG;
    return forward(G, M, 2 * F, K, rows, group_offset, w, pre, out, dev_status, true, stream);
}

extern "C" int ep_expert_bf16_plan(int32_t product, int32_t G, int64_t M, int32_t N, int32_t K) {
    if (check_bf16(G, M, N, K) != EP_OK || (product == EP_PRODUCT_GATE_UP && N % 16 != 0))
        return EP_ERR_INVALID_ARG;
    Bf16Args a{};
    a.G = G;
    a.M = M;
    a.splits = 1;
    bool big = false;
    switch (product) {
        case EP_PRODUCT_FORWARD:
            forward_sizes(a, N, K);
            big = takes_big<kForward>(a);
            break;
        case EP_PRODUCT_GATE_UP:
            forward_sizes(a, N, K);
            big = takes_big<kGate>(a);
            break;
        case EP_PRODUCT_ROWS_BACKWARD:
            rows_back_sizes(a, N, K);
            big = takes_big<kRowsBack>(a);
            break;
        case EP_PRODUCT_WEIGHTS_BACKWARD:
            weight_back_sizes(a, N, K);
            big = takes_big<kWeightBack>(a);
            break;
        default: return EP_ERR_INVALID_ARG;
    }
    return big ? EP_TILES_BIG : EP_TILES_SMALL;
}

extern "C" size_t ep_expert_backward_workspace_bytes(int32_t G, int64_t M, int32_t N, int32_t K) {
    if (check_bf16(G, M, N, K) != EP_OK) return 0;
    const int32_t splits = weight_splits(G, M, N, K);
    return splits > 1 ? (size_t)splits * G * N * K * 4 : 0;
}

extern "C" int ep_expert_product_bf16_backward(int32_t G, int64_t M, int32_t N, int32_t K,
                                               int32_t dtype, const void* rows,
                                               const int32_t* group_offset, const void* w,
                                               const void* grad_out, void* grad_rows, void* grad_w,
                                               int32_t* dev_status, void* workspace,
                                               size_t workspace_bytes, hipStream_t stream) {
    int v = check_bf16(G, M, N, K);
    if (v != EP_OK) return v;
    Bf16Args a{};
    v = common_args(a, G, M, group_offset, dev_status);
    if (v != EP_OK) return v;
    v = check_backward(M > 0, dtype, rows, w, grad_rows, grad_w);
    if (v != EP_OK) return v;
    if (!aligned16(grad_out) || (M > 0 && !grad_out)) return EP_ERR_INVALID_ARG;
    if (!grad_rows && !grad_w && M > 0) return EP_ERR_INVALID_ARG;
    if (grad_w && (v = check_workspace(G, M, N, K, workspace, workspace_bytes)) != EP_OK) return v;
    return backward(a, N, K, dtype, rows, w, grad_out, grad_rows, grad_w, workspace, stream);
}

extern "C" int ep_expert_gate_up_bf16_backward(int32_t G, int64_t M, int32_t F, int32_t K,
                                               int32_t dtype, const void* rows,
                                               const int32_t* group_offset, const void* w,
                                               const void* pre, const void* grad_out,
                                               void* grad_pre, void* grad_rows, void* grad_w,
                                               int32_t* dev_status, void* workspace,
                                               size_t workspace_bytes, hipStream_t stream) {
    if (F < 8 || F % 8 != 0 || F > kMaxDim / 2) return EP_ERR_INVALID_ARG;
    int v = check_bf16(G, M, 2 * F, K);
    if (v != EP_OK) return v;
    Bf16Args a{};
    v = common_args(a, G, M, group_offset, dev_status);
    if (v != EP_OK) return v;
    v = check_backward(M > 0, dtype, rows, w, grad_rows, grad_w);
    if (v != EP_OK) return v;
    if (!aligned16(pre) || !aligned16(grad_out) || !aligned16(grad_pre)) return EP_ERR_INVALID_ARG;
    if (M > 0 && (!pre || !grad_out || !grad_pre)) return EP_ERR_INVALID_ARG;
    if (grad_w && (v = check_workspace(G, M, 2 * F, K, workspace, workspace_bytes)) != EP_OK) return v;
    if (M > 0) {
        GateBackArgs b{};
        b.pre = reinterpret_cast<const u32x4*>(pre);
        b.grad_out = reinterpret_cast<const u32x4*>(grad_out);
        b.grad_pre = reinterpret_cast<u32x4*>(grad_pre);
        b.group_offset = group_offset;
        b.st = dev_status;
        b.M = M;
        b.G = G;
        b.nv = F / 8;
        while (b.tpr_log < 8 && (1 << b.tpr_log) < b.nv) ++b.tpr_log;
        clear_hip_error();
        hipLaunchKernelGGL(gate_back_kernel, dim3(loop_grid(ceil_div(M, 256 >> b.tpr_log), 256)),
                           dim3(256), 0, stream, b);
        EP_HIP_CHECK(hipGetLastError());
    }
    return backward(a, 2 * F, K, dtype, rows, w, grad_pre, grad_rows, grad_w, workspace, stream);
}
