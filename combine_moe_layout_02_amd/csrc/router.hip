// Router (top-k gate), load-balance loss and their gradients.
//
// A wave owns one token: its E logits lie in registers, lane l holding experts
// l*V .. l*V+V-1 (V = E/64 rounded up to a power of two), so the lowest index
// among equal logits is the lowest lane, then the lowest register.  Softmax is
// one maximum and one sum across the wave (DPP); a pick is the wave's maximum,
// one ballot for its lane, and the owner's register struck out, K times.
// Arithmetic within a token is fp32, sums over tokens are fp64.
//
// Loss = sum over tokens and experts of coef[sequence][e] * p[t][e], where coef
// comes from the counts alone.  A workgroup adds up its own tokens'
// probabilities (registers, then LDS in wave order) and counts and writes one
// row of partial sums; a second launch adds the rows of a sequence in order,
// so no result depends on which workgroup ran first, and nothing has to be
// cleared before a call.
//
// Bound: at path sizes (4 MB of logits) launch and latency; beyond, reading
// the logits.  4096 x 256, K = 8 of 4 of 8 groups: picks and sums 9.6 us, the
// finish 7.2, the gradient 6.3; 128 tokens to serve 4.9 us.
#include <algorithm>

#include "router.h"

namespace moe {
namespace {

constexpr int kRouterWaves = 4;              // tokens of a workgroup without the loss, and of the backward pass
constexpr int kMaxGroups = 64;
constexpr int kFinishThreads = 1024;
constexpr int kMaxParts = 256;               // workgroups per sequence
constexpr int kMaxLastParts = 1024;          // workgroups whose last one adds up the loss
constexpr int kMaxCountedSeqs = 1024;        // sequences that k_router_finish counts itself,
constexpr int64_t kMaxCounting = 1 << 23;    // and the partial rows that its workgroups read for it in all

// Wave-wide reductions: DPP shifts inside rows of 16, then across rows; lane
// 63 ends with the result and every lane reads it from there.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float fill, float v) {
    return __uint_as_float(static_cast<unsigned int>(__builtin_amdgcn_update_dpp(
        static_cast<int>(__float_as_uint(fill)), static_cast<int>(__float_as_uint(v)), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float lane63(float v) {
    return __uint_as_float(static_cast<unsigned int>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), 63)));
}
__device__ __forceinline__ float wave_max(float v) {
    const float low = -__builtin_inff();
    v = fmaxf(v, dpp_or<0x111, 0xf>(low, v));
    v = fmaxf(v, dpp_or<0x112, 0xf>(low, v));
    v = fmaxf(v, dpp_or<0x114, 0xf>(low, v));
    v = fmaxf(v, dpp_or<0x118, 0xf>(low, v));
    v = fmaxf(v, dpp_or<0x142, 0xa>(low, v));
    v = fmaxf(v, dpp_or<0x143, 0xc>(low, v));
    return lane63(v);
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_or<0x111, 0xf>(0.0f, v);
    v += dpp_or<0x112, 0xf>(0.0f, v);
    v += dpp_or<0x114, 0xf>(0.0f, v);
    v += dpp_or<0x118, 0xf>(0.0f, v);
    v += dpp_or<0x142, 0xa>(0.0f, v);
    v += dpp_or<0x143, 0xc>(0.0f, v);
    return lane63(v);
}

// One token's logits: lane l gets experts l*V + j, -inf past E.  A row is read
// in whole vectors where E and the row's address allow it (V*size bytes, at
// most 16 at a time).
template <int V, bool BF16, bool VEC>
__device__ __forceinline__ void load_logits(const void *logits, int64_t t, int E, float (&z)[V]) {
    const int e0 = (threadIdx.x & (kWave - 1)) * V;
    const float none = -__builtin_inff();
    if constexpr (BF16) {
        const unsigned short *row = static_cast<const unsigned short *>(logits) + t * E;
        if constexpr (VEC) {
            unsigned short h[V];
            if (e0 < E) {
                __builtin_memcpy(h, __builtin_assume_aligned(row + e0, V * 2 < 16 ? V * 2 : 16), sizeof(h));
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = __uint_as_float(static_cast<unsigned int>(h[j]) << 16);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = none;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                z[j] = e0 + j < E ? __uint_as_float(static_cast<unsigned int>(row[e0 + j]) << 16) : none;
        }
    } else {
        const float *row = static_cast<const float *>(logits) + t * E;
        if constexpr (VEC) {
            if (e0 < E) {
                __builtin_memcpy(z, __builtin_assume_aligned(row + e0, V * 4 < 16 ? V * 4 : 16), sizeof(z));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = none;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = e0 + j < E ? row[e0 + j] : none;
        }
    }
}

// What a token's logits say: top = the highest; counts = some logit is above
// -inf (and the mask, checked by the caller); broken = a NaN or +inf among
// them.  Lanes past E hold -inf.
template <int V>
__device__ __forceinline__ void inspect(const float (&z)[V], float &top, bool &broken) {
    float m = -__builtin_inff();
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bad = bad || !(z[j] < __builtin_inff());
        m = fmaxf(m, z[j]);
    }
    broken = __ballot(bad) != 0;
    top = wave_max(m);
}

// Softmax over the wave's logits (top = their maximum, finite).  The product
// with the rounded reciprocal has two roundings; its remainder, exact in a fused
// step, times the reciprocal makes it the quotient with one, as the route
// weights are (the division itself takes 10 instructions per logit).
template <int V>
__device__ __forceinline__ void softmax(const float (&z)[V], float top, float (&p)[V]) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        p[j] = expf(z[j] - top);
        sum += p[j];
    }
    const float total = wave_sum(sum), inv = 1.0f / total;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float q = p[j] * inv;
        p[j] = __builtin_fmaf(__builtin_fmaf(-q, total, p[j]), inv, q);
    }
}

// Bits that order like the floats (no NaN; -0 was added to +0 before).
__device__ __forceinline__ unsigned int order_bits(float v) {
    const unsigned int b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Strikes out the logits outside the token's topk_groups best groups.  Group
// scores meet in LDS (`best`, kMaxGroups words of the wave's own).
template <int V>
__device__ __forceinline__ void keep_groups(float (&z)[V], int E, int n_groups, int topk_groups, unsigned int *best) {
    const int lane = threadIdx.x & (kWave - 1), size = E / n_groups;
    best[lane] = 0u;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (lane * V + j < E) atomicMax(best + (lane * V + j) / size, order_bits(z[j]));
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    // a lane below n_groups holds its group's score; a group's rank is the
    // number of groups ahead of it, so the best are those of rank < topk_groups
    const unsigned int mine = best[lane];
    int rank = 0;
    for (int g = 0; g < n_groups; ++g) {
        const unsigned int other = static_cast<unsigned int>(__builtin_amdgcn_readlane(static_cast<int>(mine), g));
        rank += (other > mine || (other == mine && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < n_groups && rank < topk_groups);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int g = min((lane * V + j) / size, kMaxGroups - 1);
        if (!((kept >> g) & 1u)) z[j] = -__builtin_inff();
    }
    __builtin_amdgcn_wave_barrier();
}

// The K highest of the wave's logits, descending, ties to the lower expert:
// lane k < K gets pick k and its logit, -1 and -inf once none is left.
template <int V>
__device__ __forceinline__ void pick_top(float (&z)[V], int K, int &my_idx, float &my_z) {
    const int lane = threadIdx.x & (kWave - 1);
    const float none = -__builtin_inff();
    my_idx = -1;
    my_z = none;
    for (int k = 0; k < K; ++k) {
        float m = z[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < V; ++j) {
            at = z[j] > m ? j : at;
            m = fmaxf(m, z[j]);
        }
        const float top = wave_max(m);
        if (top == none) break;
        const int owner = __builtin_ctzll(__ballot(m == top));
        const int e = __builtin_amdgcn_readlane(lane * V + at, owner);
        if (lane == k) {
            my_idx = e;
            my_z = top;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = (lane == owner && at == j) ? none : z[j];
    }
}

// Waves of a workgroup that sums for the loss: as many as keep a SIMD busy (a
// token's picks are one long chain of dependent steps: with 4 waves per
// workgroup and 4 tokens per wave the 4096 x 256 batch took 16.0 us, with 16
// waves and one token each 9.4), with LDS for a row of E sums each.
template <int V>
constexpr int loss_waves() {
    return V <= 4 ? 16 : 64 / V;
}

// What the finishing launch reads, per workgroup and expert: the sum of the
// probabilities and the picks.
struct Partial {
    float p;
    int32_t c;
};

struct LossShape {
    int per_seq;   // workgroups per sequence
    int tokens;    // tokens per workgroup
};

// GIVEN: the routing is the caller's; else the router picks.  LOSS: the
// workgroup's tokens are a run of one sequence and it writes partial sums.
template <int V, bool BF16, bool VEC, bool GIVEN, bool LOSS, int WAVES = LOSS ? loss_waves<V>() : kRouterWaves>
__global__ __launch_bounds__(WAVES * kWave) void k_router(RouterArgs a, LossShape sh, Partial *part, int32_t *part_n,
                                                         int32_t *counter) {
    static_assert(LOSS || !GIVEN, "without the loss the router makes the routing");
    __shared__ float s_p[LOSS ? WAVES * V * kWave : 1];       // [waves][E] probabilities
    __shared__ int32_t s_c[LOSS ? V * kWave : 1];             // [E] picks
    __shared__ unsigned int best[GIVEN ? 1 : WAVES][kMaxGroups];
    __shared__ int s_n;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int E = a.E, K = a.K;
    int64_t t0, t1;
    if constexpr (LOSS) {
        const int64_t g = blockIdx.x / sh.per_seq, at = blockIdx.x % sh.per_seq;
        t0 = g * a.seq + at * sh.tokens;
        t1 = min(t0 + sh.tokens, (g + 1) * static_cast<int64_t>(a.seq));
        for (int e = threadIdx.x; e < E; e += WAVES * kWave) s_c[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
    } else {
        t0 = static_cast<int64_t>(blockIdx.x) * WAVES;
        t1 = min(t0 + WAVES, static_cast<int64_t>(a.S));
    }
    // 64 bits: a wave of a long sequence adds thousands of tokens.  Its sum is
    // rounded to fp32 where it passes to LDS, and the workgroup's in its partial
    // row: half a unit each, however long the sequence.
    double sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0;
    int n = 0;
    for (int64_t t = t0 + wave; t < t1; t += WAVES) {
        float z[V];
        load_logits<V, BF16, VEC>(a.logits, t, E, z);
        const bool masked = a.mask != nullptr && a.mask[t] == 0;
        int given = -1;
        if (GIVEN && lane < K) given = a.given_idx[t * K + lane];
        float top;
        bool broken;
        inspect<V>(z, top, broken);
        const bool counts = !masked && (broken || top > -__builtin_inff());
        float p[V];
        if constexpr (LOSS) {
            if (counts) {
                n += 1;
                if (broken) {
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] = __builtin_nan("");
                } else {
                    softmax<V>(z, top, p);
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] += p[j];
                }
            }
        }
        int my = -1;
        if constexpr (GIVEN) {
            if (counts && given >= 0 && given < E) my = given;
        } else {
            float my_z = -__builtin_inff(), w = 0.0f;
            if (counts && !broken) {
                float total = 0.0f;
                if (!a.renorm) {
#pragma unroll
                    for (int j = 0; j < V; ++j) total += expf(z[j] - top);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] += 0.0f;   // -0 and +0 are equal logits
                if (a.topk_groups < a.n_groups) keep_groups<V>(z, E, a.n_groups, a.topk_groups, best[wave]);
                pick_top<V>(z, K, my, my_z);
                // renorm: the first pick is the highest logit of all, so both
                // forms subtract the same maximum
                const float e = my >= 0 ? expf(my_z - top) : 0.0f;
                w = e / wave_sum(a.renorm ? e : total);
            }
            if (lane < K) {
                a.idx[t * K + lane] = my;
                a.w[t * K + lane] = w;
            }
        }
        if constexpr (LOSS) {
            if (my >= 0) atomicAdd(s_c + my, 1);
        }
    }
    if constexpr (LOSS) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (lane * V + j < E) s_p[wave * E + lane * V + j] = static_cast<float>(sum[j]);
        if (lane == 0) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t base = static_cast<size_t>(blockIdx.x) * E;
        for (int e = threadIdx.x; e < E; e += WAVES * kWave) {
            double v = 0.0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v += s_p[w * E + e];
            part[base + e] = Partial{static_cast<float>(v), s_c[e]};
        }
        if (threadIdx.x == 0) part_n[blockIdx.x] = s_n;
        if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;   // for k_router_finish, launched behind this
    }
}

// Sum of a double over the workgroup, in thread order per wave, then over
// waves; the result is valid in every thread.
__device__ __forceinline__ double block_sum(double v, double *s_tmp) {
    for (int d = kWave / 2; d > 0; d /= 2) v += __shfl_xor(v, d, kWave);
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) s_tmp[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kFinishThreads / kWave; ++w) s += s_tmp[w];
    return s;
}

// Sequences with a token that counts, where k_router_finish does not count them
// itself (one workgroup).
__global__ __launch_bounds__(kFinishThreads) void k_router_used(const int32_t *__restrict__ part_n, int G, int per_seq,
                                                               int32_t *used) {
    __shared__ double s_tmp[kFinishThreads / kWave];
    int mine = 0;
    for (int g = threadIdx.x; g < G; g += kFinishThreads) {
        int n = 0;
        for (int b = 0; b < per_seq; ++b) n |= part_n[static_cast<size_t>(g) * per_seq + b];
        mine += n != 0 ? 1 : 0;
    }
    const double total = block_sum(mine, s_tmp);
    if (threadIdx.x == 0) *used = static_cast<int32_t>(total);
}

// One workgroup per sequence and kFinishCols experts: adds the partial rows in
// order, writes counts and coefficients, and its part of the loss (the loss
// itself where it is alone).  used: the number of sequences that count, or null:
// then it is counted here, a bit in LDS for each.  The rows come from every
// XCD's workgroups, past this one's L2, so few columns per workgroup: all 256 of
// the 4096 x 256 batch in one took 23 us, 32 take 7.5.
constexpr int kFinishCols = 32;
__global__ __launch_bounds__(kFinishThreads) void k_router_finish(RouterArgs a, int per_seq, int col_blocks,
                                                                 const Partial *__restrict__ part,
                                                                 const int32_t *__restrict__ part_n,
                                                                 const int32_t *__restrict__ used, double *part_loss,
                                                                 int32_t *counter) {
    constexpr int kSlices = kFinishThreads / kFinishCols;
    constexpr int kBatch = kMaxParts / kSlices;   // a thread's rows, all in flight
    __shared__ int2 s_tmp[kFinishThreads / kWave];
    __shared__ double s_p[kSlices][kFinishCols];
    __shared__ int32_t s_c[kSlices][kFinishCols];
    __shared__ unsigned int s_bits[kMaxCountedSeqs / 32];
    const int tid = threadIdx.x, E = a.E, g = blockIdx.x / col_blocks;
    const int col = tid % kFinishCols, slice = tid / kFinishCols, e = (blockIdx.x % col_blocks) * kFinishCols + col;
    const size_t first = static_cast<size_t>(g) * per_seq;
    const bool count_here = a.G > 1 && used == nullptr;
    // slice s adds rows s, s + slices, ...
    Partial v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int b = slice + i * kSlices;
        v[i] = b < per_seq && e < E ? part[(first + b) * E + e] : Partial{0.0f, 0};
    }
    int2 mine = make_int2(tid < per_seq ? part_n[first + tid] : 0, 0);   // per_seq <= kMaxParts
    if (count_here) {
        for (int i = tid; i < (a.G + 31) / 32; i += kFinishThreads) s_bits[i] = 0u;
        __syncthreads();
        for (int i = tid; i < a.G * per_seq; i += kFinishThreads)
            if (part_n[i] != 0) atomicOr(&s_bits[i / per_seq / 32], 1u << (i / per_seq % 32));
        __syncthreads();
        for (int i = tid; i < (a.G + 31) / 32; i += kFinishThreads) mine.y += __popc(s_bits[i]);
    }
    double p = 0.0;
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        p += v[i].p;
        c += v[i].c;
    }
    s_p[slice][col] = p;
    s_c[slice][col] = c;
    int2 sums;
    block_exclusive_scan2<kFinishThreads / kWave>(mine, s_tmp, sums);
    if (tid >= kWave) return;
    const double n = sums.x, seqs = count_here ? sums.y : (a.G > 1 ? *used : 1);
    double loss = 0.0;
    if (slice == 0 && e < E) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) {
            p += s_p[i][col];
            c += s_c[i][col];
        }
        const size_t cell = static_cast<size_t>(g) * E + e;
        const double coef = n > 0.0 ? static_cast<double>(a.alpha) * E / (seqs * a.K * n * n) * c : 0.0;
        a.count[cell] = c;
        a.coef[cell] = static_cast<float>(coef);
        loss = coef * p;
    }
    for (int d = kWave / 2; d > 0; d /= 2) loss += __shfl_xor(loss, d, kWave);
    if (gridDim.x == 1) {
        if (tid == 0) *a.loss = static_cast<float>(loss);
        return;
    }
    // The workgroup that arrives last adds the parts, in their own order: a
    // launch less than k_router_loss.  Nobody waits.  (The counter is 0: k_router
    // cleared it.)
    int arrived = 0;
    if (tid == 0) {
        __hip_atomic_store(part_loss + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (gridDim.x <= kMaxLastParts)
            arrived = __hip_atomic_fetch_add(counter, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1;
    }
    if (__builtin_amdgcn_readfirstlane(arrived) != static_cast<int>(gridDim.x)) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    loss = 0.0;
    for (int i = tid; i < static_cast<int>(gridDim.x); i += kWave)
        loss += __hip_atomic_load(part_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int d = kWave / 2; d > 0; d /= 2) loss += __shfl_xor(loss, d, kWave);
    if (tid == 0) *a.loss = static_cast<float>(loss);
}

__global__ __launch_bounds__(kFinishThreads) void k_router_loss(const double *__restrict__ part_loss, int n, float *loss) {
    __shared__ double s_tmp[kFinishThreads / kWave];
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kFinishThreads) v += part_loss[i];
    v = block_sum(v, s_tmp);
    if (threadIdx.x == 0) *loss = static_cast<float>(v);
}

// One wave per token.
template <int V, bool BF16, bool VEC>
__global__ __launch_bounds__(kRouterWaves * kWave) void k_router_backward(RouterArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWaves + wave;
    if (t >= a.S) return;
    const int E = a.E, K = a.K, e0 = lane * V;
    float z[V], d[V];
    load_logits<V, BF16, VEC>(a.logits, t, E, z);
    const bool masked = a.mask != nullptr && a.mask[t] == 0;
    int my = -1;
    float w = 0.0f, dw = 0.0f;
    if (a.d_w != nullptr && lane < K) {
        my = a.picked[t * K + lane];
        if (my < 0 || my >= E) my = -1;
        if (my >= 0) {
            w = a.picked_w[t * K + lane];
            dw = a.d_w[t * K + lane];
        }
    }
    float top;
    bool broken;
    inspect<V>(z, top, broken);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = 0.0f;
    if (!masked && broken) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = __builtin_nanf("");
    } else if (!masked && top > -__builtin_inff()) {
        float p[V];
        softmax<V>(z, top, p);
        if (a.saved_coef != nullptr) {
            const float *coef = a.saved_coef + t / a.seq * E;
            const float dl = *a.d_loss;
            float inner = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = e0 + j < E ? coef[e0 + j] : 0.0f;
                inner = __builtin_fmaf(d[j], p[j], inner);
            }
            inner = wave_sum(inner);
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = dl * (p[j] * (d[j] - inner));
        }
        if (a.d_w != nullptr) {
            const float inner = wave_sum(w * dw);
            // what pick k adds: to its own logit (renorm), or to the
            // probability's factor
            const float add = a.renorm ? w * (dw - inner) : dw;
            float pk[V];
#pragma unroll
            for (int j = 0; j < V; ++j) pk[j] = 0.0f;
            for (int k = 0; k < K; ++k) {
                const int e = __builtin_amdgcn_readlane(my, k);
                const float v = __uint_as_float(static_cast<unsigned int>(
                    __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(add)), k)));
#pragma unroll
                for (int j = 0; j < V; ++j) pk[j] += e == e0 + j ? v : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] += a.renorm ? pk[j] : p[j] * (pk[j] - inner);
        }
    }
    if constexpr (BF16) {
        unsigned short *row = static_cast<unsigned short *>(a.d_logits) + t * E;
        unsigned short h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = __builtin_bit_cast(unsigned short, static_cast<__bf16>(d[j]));
        if constexpr (VEC) {
            if (e0 < E) __builtin_memcpy(__builtin_assume_aligned(row + e0, V * 2 < 16 ? V * 2 : 16), h, sizeof(h));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e0 + j < E) row[e0 + j] = h[j];
        }
    } else {
        float *row = static_cast<float *>(a.d_logits) + t * E;
        if constexpr (VEC) {
            if (e0 < E) __builtin_memcpy(__builtin_assume_aligned(row + e0, V * 4 < 16 ? V * 4 : 16), d, sizeof(d));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e0 + j < E) row[e0 + j] = d[j];
        }
    }
}

// Lanes' experts: the power of two that covers E.
int lane_experts(int E) { return E <= 64 ? 1 : (E <= 128 ? 2 : (E <= 256 ? 4 : (E <= 512 ? 8 : 16))); }

// Workgroups of the loss form: a token per wave, more once that would make more
// than kMaxParts partial rows in a sequence, whose sum is one workgroup's work.
LossShape loss_shape(const RouterArgs &a) {
    const int v = lane_experts(a.E), waves = v <= 4 ? 16 : 64 / v;
    LossShape sh;
    sh.tokens = static_cast<int>(std::max<int64_t>(waves, (a.seq + int64_t(kMaxParts) - 1) / kMaxParts));
    sh.per_seq = std::max(1, static_cast<int>((static_cast<int64_t>(a.seq) + sh.tokens - 1) / sh.tokens));
    return sh;
}

int finish_blocks(const RouterArgs &a) { return (a.E + kFinishCols - 1) / kFinishCols; }

size_t up16(size_t x) { return (x + 15) & ~size_t(15); }

struct LossWorkspace {
    size_t part, n, used, loss, bytes;
};
LossWorkspace loss_workspace(const RouterArgs &a, const LossShape &sh) {
    LossWorkspace w{};
    const size_t parts = static_cast<size_t>(a.G) * sh.per_seq;
    w.part = 0;
    w.n = up16(parts * a.E * sizeof(Partial));
    w.used = up16(w.n + parts * 4);
    w.loss = w.used + 16;
    w.bytes = up16(w.loss + static_cast<size_t>(a.G) * finish_blocks(a) * 8);
    return w;
}

// Whole vectors: rows and the array start on a lane's vector.
template <int V>
bool whole_vectors(const RouterArgs &a, const void *p) {
    const int bytes = std::min(16, V * (a.bf16 ? 2 : 4));
    return a.E % V == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

template <int V, bool BF16, bool GIVEN>
hipError_t launch_v(const RouterArgs &a, void *workspace, hipStream_t s) {
    const bool vec = whole_vectors<V>(a, a.logits);
    if constexpr (!GIVEN) {
        if (a.loss == nullptr) {
            const dim3 block(kRouterWaves * kWave), grid((static_cast<unsigned>(a.S) + kRouterWaves - 1) / kRouterWaves);
            if (vec)
                hipLaunchKernelGGL((k_router<V, BF16, true, false, false>), grid, block, 0, s, a, LossShape{}, nullptr, nullptr, nullptr);
            else
                hipLaunchKernelGGL((k_router<V, BF16, false, false, false>), grid, block, 0, s, a, LossShape{}, nullptr, nullptr, nullptr);
            return hipGetLastError();
        }
    }
    if (a.G == 0) {   // no sequence: the loss is 0
        hipLaunchKernelGGL(k_router_loss, dim3(1), dim3(kFinishThreads), 0, s, nullptr, 0, a.loss);
        return hipGetLastError();
    }
    const LossShape sh = loss_shape(a);
    const LossWorkspace w = loss_workspace(a, sh);
    char *ws = static_cast<char *>(workspace);
    Partial *part = reinterpret_cast<Partial *>(ws + w.part);
    int32_t *pn = reinterpret_cast<int32_t *>(ws + w.n), *used = reinterpret_cast<int32_t *>(ws + w.used);
    double *pl = reinterpret_cast<double *>(ws + w.loss);
    const int64_t parts = static_cast<int64_t>(a.G) * sh.per_seq;
    const dim3 grid(static_cast<unsigned>(parts)), wide(loss_waves<V>() * kWave);
    if (vec)
        hipLaunchKernelGGL((k_router<V, BF16, true, GIVEN, true>), grid, wide, 0, s, a, sh, part, pn, used + 1);
    else
        hipLaunchKernelGGL((k_router<V, BF16, false, GIVEN, true>), grid, wide, 0, s, a, sh, part, pn, used + 1);
    // Which sequences count: every finishing workgroup finds out by itself, or one
    // more launch does for all of them.  The former grows as workgroups times
    // partial rows.  Measured in place / apart (us, the whole call): 64 workgroups
    // x 32 rows 10.8 / 12.6; 256 x 8192 105 / 119; 512 x 4096 53 / 51; 1024 x 128
    // 33 / 35; 1024 x 32768 515 / 432; 2048 x 1024 37 / 28; 16384 x 8192 616 / 162;
    // 65536 x 8192 2285 / 446.
    const int cols = finish_blocks(a), blocks = a.G * cols;
    const bool count_apart = blocks > kMaxCountedSeqs || blocks * parts > kMaxCounting;
    if (count_apart) hipLaunchKernelGGL(k_router_used, dim3(1), dim3(kFinishThreads), 0, s, pn, a.G, sh.per_seq, used);
    hipLaunchKernelGGL(k_router_finish, dim3(blocks), dim3(kFinishThreads), 0, s, a, sh.per_seq, cols, part, pn,
                       count_apart ? used : nullptr, pl, used + 1);
    if (blocks > kMaxLastParts) hipLaunchKernelGGL(k_router_loss, dim3(1), dim3(kFinishThreads), 0, s, pl, blocks, a.loss);
    return hipGetLastError();
}

template <int V>
hipError_t launch_type(const RouterArgs &a, void *workspace, hipStream_t s) {
    if (a.given)
        return a.bf16 ? launch_v<V, true, true>(a, workspace, s) : launch_v<V, false, true>(a, workspace, s);
    return a.bf16 ? launch_v<V, true, false>(a, workspace, s) : launch_v<V, false, false>(a, workspace, s);
}

template <int V>
hipError_t launch_backward_v(const RouterArgs &a, hipStream_t s) {
    const bool vec = whole_vectors<V>(a, a.logits) && whole_vectors<V>(a, a.d_logits);
    const dim3 grid((static_cast<unsigned>(a.S) + kRouterWaves - 1) / kRouterWaves), block(kRouterWaves * kWave);
    if (a.bf16) {
        if (vec)
            hipLaunchKernelGGL((k_router_backward<V, true, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_router_backward<V, true, false>), grid, block, 0, s, a);
    } else {
        if (vec)
            hipLaunchKernelGGL((k_router_backward<V, false, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_router_backward<V, false, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

size_t router_workspace_bytes(const RouterArgs &a) { return loss_workspace(a, loss_shape(a)).bytes; }

bool router_grid_ok(const RouterArgs &a, bool loss) {
    if (!loss) return static_cast<int64_t>(a.S) * kWave + kRouterWaves * kWave <= kMaxLaunchThreads;
    const LossShape sh = loss_shape(a);
    const int v = lane_experts(a.E), waves = v <= 4 ? 16 : 64 / v;
    return static_cast<int64_t>(a.G) * sh.per_seq * waves * kWave <= kMaxLaunchThreads &&
           static_cast<int64_t>(a.G) * finish_blocks(a) * kFinishThreads <= kMaxLaunchThreads;
}

hipError_t launch_router(const RouterArgs &a, void *workspace, hipStream_t s) {
    if (a.E <= 64) return launch_type<1>(a, workspace, s);
    if (a.E <= 128) return launch_type<2>(a, workspace, s);
    if (a.E <= 256) return launch_type<4>(a, workspace, s);
    if (a.E <= 512) return launch_type<8>(a, workspace, s);
    return launch_type<16>(a, workspace, s);
}

hipError_t launch_router_backward(const RouterArgs &a, hipStream_t s) {
    if (a.E <= 64) return launch_backward_v<1>(a, s);
    if (a.E <= 128) return launch_backward_v<2>(a, s);
    if (a.E <= 256) return launch_backward_v<4>(a, s);
    if (a.E <= 512) return launch_backward_v<8>(a, s);
    return launch_backward_v<16>(a, s);
}

}  // namespace moe
